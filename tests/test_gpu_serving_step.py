"""The calls as a serving loop chains them, on the device, against the plain
implementations chained the same way: a draft tree grown by beam selection,
verified, its accepted path committed in the cache, the path's queries
weighed and the cache cut to its budget; and a beam search whose caches
follow the beams."""
import numpy as np
import pytest
import torch

import oracle
import state_ref as ref
from test_gpu_cache import UNIT, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from speculative_decoding_verification_87_b200 import binding, build
    build.build()
    binding.load_library()
    return binding


def bits(t):
    """bf16 CPU tensor -> its uint16 bits, as the oracle takes them."""
    return t.view(torch.int16).numpy().view(np.uint16)


def test_tree_step(sv):
    B, widths, V, T, D, G, H = 3, (1, 3, 4, 2), 2000, 0.8, 64, 2, 2
    N, depth = sum(widths), len(widths) - 1
    C, budget, sinks, recent = 140, 96, 2, 16
    g = torch.Generator().manual_seed(5)
    draft = torch.randn((B, N, V), generator=g) * 3
    target = (draft + 0.3 * torch.randn((B, N, V), generator=g)).to(torch.bfloat16)
    draft = draft.to(torch.bfloat16)
    dd, td = draft.cuda(), target.cuda()

    # grow the tree level by level: the first level's one beam is the root
    tokens = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    parents = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    scores = torch.zeros((B, 1), device="cuda")
    ref_scores, start = np.zeros((B, 1)), 0
    for level in range(depth):
        W, K = widths[level], widths[level + 1]
        rows = dd[:, start:start + W].contiguous()
        scores, par, tok, _ = sv.spec_beam_select(rows, scores, V, K, T)
        rs, rp, rt, _, _ = ref.beam_select(rows.double().cpu().numpy(), ref_scores, V, K, float(np.float32(T)))
        assert np.array_equal(par.cpu().numpy(), rp) and np.array_equal(tok.cpu().numpy(), rt)
        ref_scores = scores.double().cpu().numpy()
        tokens[:, start + W:start + W + K] = tok
        parents[:, start + W:start + W + K] = par + start
        start += W

    path = torch.zeros((B, depth + 1), dtype=torch.int32, device="cuda")
    out, acc, _ = sv.spec_verify_tree(td, dd, tokens, parents, depth, V, 0, out_path_nodes=path)
    o = oracle.verify_tree(bits(target), bits(draft), tokens.cpu().numpy(), parents.cpu().numpy(), depth, V,
                           False, 1.0, 0, 0)
    assert np.array_equal(out.cpu().numpy(), o["out"]) and np.array_equal(acc.cpu().numpy(), o["acc"])
    assert int(acc.max()) >= 1  # something was accepted

    # the forward over the tree left its rows behind the cache
    base = ints([90, 30, 120])
    k, v = (torch.randn((B, H, C, D), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((B, N, H * G, D), generator=g).to(torch.bfloat16)
    kd, vd, qd = k.cuda(), v.cuda(), q.cuda()
    score = torch.rand((B, H, C), generator=g)
    pos = torch.arange(C, dtype=torch.int32).expand(B, H, C).contiguous()
    sd, pd = score.cuda(), pos.cuda()
    lens = sv.spec_commit_path([kd, vd], base, path, N, 2)
    sv.spec_commit_path([qd], None, path, N, 1)
    sv.spec_cache_score(qd, kd, base, lens, sd)
    sv.spec_cache_evict(kd, vd, sd, pd, lens, budget, sinks, recent, out_lens=lens)

    bn, pn = base.cpu().numpy(), path.cpu().numpy()
    rk, rl = ref.commit_path(k.float().numpy(), bn, pn, 2)
    rv, _ = ref.commit_path(v.float().numpy(), bn, pn, 2)
    rq, _ = ref.commit_path(q.float().numpy(), np.zeros(B, int), pn, 1)
    want, bound = ref.cache_score(rq.astype(np.float64), rk.astype(np.float64), bn, rl, score.double().numpy(),
                                  D ** -0.5, UNIT)
    # the sums at the budget's border lie further apart than their bounds: every
    # slot that stays for its sum against every one that goes
    before = rl.copy()
    rk, rv, rs, rp, rl = ref.evict(rk, rv, want, pos.numpy(), rl, budget, sinks, recent)
    for b in np.nonzero(before > budget)[0]:
        for h in range(H):
            n = before[b]
            stays = np.isin(np.arange(n), rp[b, h, :budget])
            weighed = stays & (np.arange(n) >= sinks) & (np.arange(n) <= n - 1 - recent)
            lo, hi = (want - bound)[b, h, :n], (want + bound)[b, h, :n]
            assert lo[weighed].min() > hi[~stays].max()
    assert np.array_equal(lens.cpu().numpy(), rl) and rl.max() == budget
    assert np.array_equal(kd.float().cpu().numpy(), rk) and np.array_equal(vd.float().cpu().numpy(), rv)
    for b in range(B):
        n = rl[b]
        assert np.array_equal(pd.cpu().numpy()[b, :, :n], rp[b, :, :n])
        assert np.abs(sd.cpu().numpy()[b, :, :n] - rs[b, :, :n]).max() <= bound[b].max()


def test_beam_search_with_caches(sv):
    B, W, V, H, C, D = 2, 4, 500, 2, 24, 8
    g = torch.Generator().manual_seed(9)
    k, pos = torch.zeros((B, W, H, C, D)), torch.zeros((B, W, C), dtype=torch.int32)
    kd, posd = k.cuda(), pos.cuda()
    kn, pn = k.numpy().copy(), pos.numpy().copy()
    scores = torch.full((B, W), -float("inf"))
    scores[:, 0] = 0
    sd, prompt = scores.cuda(), 6
    rs = scores.double().numpy()
    begin = ints([prompt] * B)
    for step in range(10):
        at = prompt + step
        new = torch.randint(-9, 9, (B, W, H, D), generator=g).float()
        kd[:, :, :, at], kn[:, :, :, at] = new.cuda(), new.numpy()
        posd[:, :, at], pn[:, :, at] = at, at
        x = torch.randn((B, W, V + 4), generator=g) * 2
        sd, par, tok, _ = sv.spec_beam_select(x.cuda(), sd, V, W)
        end = ints([at + 1] * B)
        sv.spec_reorder_beams([kd], par, 3, begin, end)
        sv.spec_reorder_beams([posd], par, 2, begin, end)
        _, rp, rt, _, _ = ref.beam_select(x.double().numpy(), rs, V, W)
        assert np.array_equal(par.cpu().numpy(), rp) and np.array_equal(tok.cpu().numpy(), rt)
        rs = sd.double().cpu().numpy()
        w = np.array([prompt] * B), np.array([at + 1] * B)
        kn, pn = ref.reorder_beams(kn, rp, 3, *w), ref.reorder_beams(pn, rp, 2, *w)
        assert np.array_equal(kd.cpu().numpy(), kn) and np.array_equal(posd.cpu().numpy(), pn)
