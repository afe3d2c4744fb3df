"""Plain implementations, in 64 bits on the CPU, of beam selection, state
reordering, path commit, attention-weight accumulation and eviction, written
from the definitions in include/specverify.h.  No code of the package."""
import numpy as np


def beam_select(logits, scores, vocab, keep, temperature=1.0, finished=None, end_token=-1):
    """logits [B][W][stride], scores [B][W]: float arrays.  Returns (scores
    float64, parents, tokens, finished); bad requests (NaN, +inf) have parents
    and tokens -1 and scores -inf."""
    B, W, _ = logits.shape
    out_s = np.full((B, keep), -np.inf)
    out_p = np.full((B, keep), -1, np.int32)
    out_t = np.full((B, keep), -1, np.int32)
    out_f = np.zeros((B, keep), np.int32)
    bad = np.zeros(B, bool)
    for b in range(B):
        cs, cw, ct = [], [], []
        for w in range(W):
            sc = float(scores[b, w])
            if np.isnan(sc) or sc == np.inf:
                bad[b] = True
                continue
            if sc == -np.inf:
                continue
            if finished is not None and finished[b, w]:
                cs.append(np.array([sc]))
                cw.append(np.array([w]))
                ct.append(np.array([end_token]))
                continue
            x = logits[b, w, :vocab].astype(np.float64)
            m = x.max()
            if np.isnan(m) or m == np.inf:
                bad[b] = True
                continue
            if m == -np.inf:
                continue
            with np.errstate(under="ignore"):
                lse = np.log(np.sum(np.exp((x - m) / temperature)))
            t = np.nonzero(x > -np.inf)[0]
            cs.append(sc + (x[t] - m) / temperature - lse)
            cw.append(np.full(len(t), w))
            ct.append(t)
        if bad[b] or not cs:
            continue
        cs, cw, ct = np.concatenate(cs), np.concatenate(cw), np.concatenate(ct)
        if len(cs) > 4 * keep + 64:  # only what can be among the best is sorted
            least = np.partition(cs, len(cs) - keep)[len(cs) - keep]
            near = cs >= least
            cs, cw, ct = cs[near], cw[near], ct[near]
        order = np.lexsort((ct, cw, -cs))[:keep]
        n = len(order)
        out_s[b, :n], out_p[b, :n], out_t[b, :n] = cs[order], cw[order], ct[order]
        out_f[b, :n] = (ct[order] == end_token) & (end_token >= 0)
    return out_s, out_p, out_t, out_f, bad


def reorder_beams(state, parents, axis=None, begin=None, end=None):
    """state [B][W][...]; returns the new state."""
    new = state.copy()
    for b in range(parents.shape[0]):
        for j, p in enumerate(parents[b]):
            if p < 0:
                continue
            if axis is None:
                new[b, j] = state[b, p]
            else:
                at = [slice(None)] * (state.ndim - 2)
                at[axis - 2] = slice(int(begin[b]) if begin is not None else 0,
                                     int(end[b]) if end is not None else state.shape[axis])
                new[b, j][tuple(at)] = state[b, p][tuple(at)]
    return new


def commit_path(state, base, path, axis):
    """state [B][...]; returns the new state and the new lengths."""
    new = state.copy()
    lens = np.zeros(path.shape[0], np.int32)
    for b in range(path.shape[0]):
        old, dst = np.moveaxis(state[b], axis - 1, 0), np.moveaxis(new[b], axis - 1, 0)
        n = 0
        while n < path.shape[1] and path[b, n] >= 0:
            dst[base[b] + n] = old[base[b] + path[b, n]]
            n += 1
        lens[b] = base[b] + n
    return new, lens


def cache_score(q, k, begin, end, scores, scale, unit):
    """q [B][Q][Hq][D], k [B][H][C][D], scores [B][H][C], float64 arrays (values
    of the tensors' type).  Returns (out, bound): the sums, and how far an
    fp32 computation may be off: a product of D terms accumulated in fp32 is
    off by at most E = (D + 8) unit scale sum |q_d k_d| (`unit` per addition),
    a row's log-sum-exp by the largest E of its slots, so a weight by a factor
    exp(2 max E + 2^-18) at most (2^-18: the exponentials, of 2^-22 each, and
    a sum of positive terms over a chunk tree); adding up rows and the old
    value rounds to 2^-24 of the partial sums, at most R + 2 times."""
    B, Q, Hq, D = q.shape
    H, C = k.shape[1], k.shape[2]
    G = Hq // H
    out, bound = scores.copy(), np.zeros_like(scores)
    for b in range(B):
        b0, b1 = int(begin[b]), int(end[b])
        out[b, :, b0:b1] = 0.0
        for h in range(H):
            for i in range(b1 - b0):
                n = b0 + i + 1
                kk = k[b, h, :n]
                for g in range(G):
                    row = q[b, i, h * G + g]
                    s = scale * (kk @ row)
                    e = (D + 8) * unit * abs(scale) * (np.abs(kk) @ np.abs(row))
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, h, :n] += w
                    bound[b, h, :n] += w * np.expm1(2 * e.max() + 2.0 ** -18)
        rows = (b1 - b0) * G
        bound[b, :, :b1] += (rows + 2) * 2.0 ** -24 * np.abs(out[b, :, :b1]) + 1e-37
    return out, bound


def evict(k, v, scores, positions, lens, budget, sinks, recent):
    """k, v [B][H][C][D], scores, positions [B][H][C].  Returns the new k, v,
    scores, positions (below the new length) and lens."""
    k, v, scores, positions, lens = k.copy(), v.copy(), scores.copy(), positions.copy(), lens.copy()
    B, H, C = scores.shape
    for b in range(B):
        n = int(lens[b])
        if n <= budget:
            continue
        for h in range(H):
            s, p = scores[b, h, :n].copy(), positions[b, h, :n].astype(np.int64)
            safe = (p < sinks) | (p > p.max() - recent)
            nan = np.isnan(s)
            s[nan] = 0.0
            kind = np.where(safe, 2, np.where(nan, 0, 1))
            s[kind != 1] = 0.0
            order = np.lexsort((np.arange(n), -s, -kind))
            stays = np.zeros(n, bool)
            stays[order[:budget]] = True
            src = [t for t in range(budget, n) if stays[t]]
            dst = [t for t in range(budget) if not stays[t]]
            assert len(src) == len(dst)
            for a in (k, v, scores, positions):
                a[b, h, dst] = a[b, h, src]
        lens[b] = budget
    return k, v, scores, positions, lens
