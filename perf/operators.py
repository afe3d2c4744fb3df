"""Measured cases of the operators around verification: beam selection, reordering of states, commit of an accepted tree path,
accumulation of attention weight and eviction from a cache.

A case is a dict of plain values whose "op" names the operator.  `prepare` makes what a serving loop holds before the call, `run` makes
one call: the plain form in elementary torch operations, or the library's kernels where `own` is set.  Lengths follow from the case
alone, contents from the seed.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's beam search with four beams: launch latency counts
        dict(name="select-one", op="select", batch=1, beams=4, keep=4, vocab=128256, dtype="bf16",
             temperature=1.0, masked=False, finished=False),
        # a level of 16 nodes of the 60-node draft trees of a batch of 32
        dict(name="select-tree-level", op="select", batch=32, beams=16, keep=16, vocab=128256,
             dtype="bf16", temperature=1.0, masked=False, finished=False),
        # constrained decoding in fp32: most of an odd vocabulary masked, finished beams, twice as many kept as held
        dict(name="select-constrained", op="select", batch=5, beams=7, keep=14, vocab=50257,
             dtype="f32", temperature=0.7, masked=True, finished=True),
        # the caches of four layers follow four beams of one request, short window after the shared prompt
        dict(name="beams-one", op="beams", states=8, batch=1, beams=4, heads=8, capacity=640, dim=128,
             prompt=500, layout="htd", dtype="bf16"),
        # the same for eight beams of four requests, long generated windows, positions outermost
        dict(name="beams-batch", op="beams", states=8, batch=4, beams=8, heads=8, capacity=2048, dim=128,
             prompt=1000, layout="thd", dtype="bf16"),
        # a verified tree of 21 nodes, one request, fp32 cache
        dict(name="path-one", op="path", states=4, batch=1, nodes=21, depth=4, heads=5, capacity=333, dim=80,
             layout="thd", dtype="f32"),
        # the 60-node trees of a batch of 32 in eight layers' keys and values
        dict(name="path-batch", op="path", states=16, batch=32, nodes=60, depth=6, heads=8, capacity=1024,
             dim=128, layout="htd", dtype="bf16"),
        # plain decoding: one query a request, ragged caches
        dict(name="weight-decode", op="weight", batch=32, queries=1, group=4, kv_heads=8, dim=128,
             capacity=4096, dtype="bf16"),
        # the accepted queries of a verification with eight drafts
        dict(name="weight-verify", op="weight", batch=16, queries=9, group=8, kv_heads=4, dim=64,
             capacity=2100, dtype="bf16"),
        # the last 32 queries of a long prompt weigh all of it
        dict(name="weight-prompt", op="weight", batch=1, queries=32, group=4, kv_heads=8, dim=128,
             capacity=65536, dtype="bf16"),
        # a step of serving: the few slots past the budget are given up in every head
        dict(name="evict-step", op="evict", batch=32, heads=8, dim=128, capacity=2057, budget=2048, sinks=4,
             recent=256, dtype="bf16"),
        # a prompt of 32768 cut down to 4096 slots a head
        dict(name="evict-prompt", op="evict", batch=2, heads=8, dim=128, capacity=32768, budget=4096, sinks=16,
             recent=64, dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("select", "beams", "path", "weight", "evict"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "select":
        batch, beams = _spread(rng, 1, 64), _spread(rng, 1, 32)
        most = 32 * 16 * 128256 // (2 if dtype == "f32" else 1)
        vocab = _spread(rng, 40, min(130000, most // (batch * beams)))
        return dict(op=op, batch=batch, beams=beams, keep=_spread(rng, 1, 2 * beams), vocab=vocab,
                    dtype=dtype, temperature=rng.choice((0.5, 1.0, 1.3)), masked=rng.random() < 0.3,
                    finished=rng.random() < 0.3)
    if op == "beams":
        batch, beams, heads = _spread(rng, 1, 8), _spread(rng, 2, 16), rng.choice((1, 3, 8))
        capacity = _spread(rng, 40, max(41, min(2048, 4 * 8 * 2048 // (batch * beams))))
        return dict(op=op, states=rng.randint(1, 8), batch=batch, beams=beams, heads=heads, capacity=capacity,
                    dim=rng.choice((16, 40, 64, 128)), prompt=rng.randint(0, capacity - 16),
                    layout=rng.choice(("htd", "thd")), dtype=dtype)
    if op == "path":
        depth = rng.randint(1, 8)
        nodes = rng.randint(2 * depth + 2, 64)
        return dict(op=op, states=rng.randint(1, 16), batch=_spread(rng, 1, 32), nodes=nodes, depth=depth,
                    heads=rng.choice((1, 3, 8)), capacity=nodes + _spread(rng, 10, 900),
                    dim=rng.choice((16, 40, 64, 128)), layout=rng.choice(("htd", "thd")), dtype=dtype)
    if op == "weight":
        queries, group, kv_heads = _spread(rng, 1, 32), rng.choice((1, 2, 4, 7, 8)), rng.choice((1, 2, 5, 8))
        dim = rng.choice((64, 80, 128, 256))
        most = 65536 * 8 * 32 * 4 * 128 // (queries * group * kv_heads * dim * (8 if dtype == "f32" else 1))
        batch = _spread(rng, 1, 32)
        capacity = queries + _spread(rng, 30, max(40, min(65536, most // batch, 33554432 // (batch * kv_heads * dim))))
        return dict(op=op, batch=batch, queries=queries, group=group, kv_heads=kv_heads, dim=dim,
                    capacity=capacity, dtype=dtype)
    batch, heads = _spread(rng, 1, 32), rng.choice((1, 3, 8))
    capacity = _spread(rng, 64, min(32768, 2 * 8 * 32768 // (batch * heads)))
    budget = rng.choice((capacity - rng.randint(1, 9), _spread(rng, 32, capacity - 1)))
    return dict(op=op, batch=batch, heads=heads, dim=rng.choice((64, 80, 128)), capacity=capacity, budget=budget,
                sinks=rng.randint(0, 8), recent=rng.randint(0, budget // 4), dtype=dtype)


# ------------------------------------------------- what follows from a case
def _lengths(case):
    """Filled slots of each request: from about half of the capacity up to all of it."""
    c, n = case["capacity"], case["batch"]
    return [c - (c // 2 * i) // n for i in range(n)]


def _windows(case):
    """The generated positions of each request of a beam search: [prompt, end)."""
    c, p, n = case["capacity"], case["prompt"], case["batch"]
    return [(p, c - (c - p) // 2 * i // n) for i in range(n)]


def _weighed(case):
    """Slots before and after the step of each request whose attention weight is added up: all queries, or fewer of them."""
    q = case["queries"]
    return [(n - max(1, q - i % q), n) if case["batch"] > 1 else (n - q, n)
            for i, n in enumerate(max(n, q) for n in _lengths(case))]


def _depths(case):
    """Accepted depth of each request's tree."""
    return [case["depth"] - i % (case["depth"] + 1) for i in range(case["batch"])]


def _cache_lens(case):
    """Filled slots before an eviction: a little past the budget or up to the capacity; every fifth request is within its budget."""
    c, g = case["capacity"], case["budget"]
    return [max(1, g - i) if i % 5 == 4 else c - (c - g - 1) * (i % 3) // 3 for i in range(case["batch"])]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "select":
        rows = case["batch"] * case["beams"]
        if case["finished"]:
            rows = case["batch"] * (case["beams"] - case["beams"] // 4)
        n = rows * case["vocab"]
        return {"bytes": n * e + 4 * case["batch"] * (case["beams"] + 3 * case["keep"]), "flops": 4 * n}
    if op == "beams":
        w = case["beams"]
        unit = case["heads"] * case["dim"] * e * case["states"]
        rows = w - 1 + w * (1 - (1 - 1 / w) ** (w - 1))  # rows written, and distinct rows read, in the mean
        return {"bytes": sum(b - a for a, b in _windows(case)) * unit * rows, "flops": 0}
    if op == "path":
        return {"bytes": 2 * sum(_depths(case)) * case["heads"] * case["dim"] * e * case["states"] + 4 * case["batch"], "flops": 0}
    if op == "weight":
        slots = sum(n for _, n in _weighed(case)) * case["kv_heads"]
        rows = sum((b - a) * b for a, b in _weighed(case)) * case["kv_heads"] * case["group"]
        return {"bytes": slots * (case["dim"] * e + 8) + case["batch"] * case["queries"] * case["kv_heads"] * case["group"] * case["dim"] * e,
                "flops": rows * (2 * case["dim"] + 4)}
    moved, slots = 0.0, 0
    for n in _cache_lens(case):
        m = min(n, case["budget"])
        slots += n + m
        moved += max(0.0, (n - m) * m / n)  # slots past the budget that stay, in the mean
    return {"bytes": case["heads"] * (8 * slots + 4 * moved * case["dim"] * e), "flops": 0}


# ---------------------------------------------------------------- the inputs
def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    b = case["batch"]
    s = dict(case)
    if case["op"] == "select":
        w, v, k = case["beams"], case["vocab"], case["keep"]
        stride = -(-v // 8) * 8
        x = torch.randn((b, w, stride), generator=g, device="cuda") * 3
        x.scatter_add_(2, torch.randint(0, v, (b, w, 20), generator=g, device="cuda"),
                       torch.full((b, w, 20), 8.0, device="cuda"))
        if case["masked"]:
            x[torch.rand((b, w, stride), generator=g, device="cuda") < 0.9] = -math.inf
            x[:, 0, :1] = 0.0
            if w > 1:
                x[0, 1] = -math.inf  # a beam that may not go on
        s["logits"] = x.to(dtype)
        s["scores"] = torch.sort(torch.randn((b, w), generator=g, device="cuda") * 2 - 12, descending=True)[0]
        done = torch.zeros((b, w), dtype=torch.int32, device="cuda")
        done[:, w - w // 4:] = 1
        s["finished"] = done if case["finished"] else None
        s["end"] = 2 if case["finished"] else -1
        s["out"] = (torch.zeros((b, k), device="cuda"), torch.zeros((b, k), dtype=torch.int32, device="cuda"),
                    torch.zeros((b, k), dtype=torch.int32, device="cuda"))
        return s
    if case["op"] in ("beams", "path"):
        mid = (case["heads"], case["capacity"]) if case["layout"] == "htd" else (case["capacity"], case["heads"])
        lead = (b, case["beams"]) if case["op"] == "beams" else (b,)
        x = _randn(g, (case["states"], *lead, *mid, case["dim"]), dtype)
        s["all"], s["list"] = x, list(x.unbind(0))
        s["axis"] = len(lead) + (1 if case["layout"] == "htd" else 0)
        if case["op"] == "beams":
            at = _windows(case)
            s["begin"], s["end"] = _ints([a for a, _ in at]), _ints([z for _, z in at])
            w = case["beams"]
            s["parents"] = torch.randint(0, w, (b, w), generator=g, device="cuda", dtype=torch.int32)
        else:
            n, d = case["nodes"], case["depth"]
            s["base"] = _ints([(case["capacity"] - n) * (b - i) // b for i in range(b)])
            # a path: node 0, then rising nodes with at least one other between
            # the root and the first, so that every row past the root moves
            key = torch.rand((b, n - 2), generator=g, device="cuda")
            later = torch.sort(torch.topk(key, d, dim=1)[1], dim=1)[0] + 2
            path = torch.cat([torch.zeros((b, 1), dtype=torch.int64, device="cuda"), later], 1)
            keep = torch.arange(d + 1, device="cuda")[None] <= _ints(_depths(case))[:, None]
            s["path"] = torch.where(keep, path, -1).to(torch.int32)
            s["lens"] = torch.zeros(b, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "weight":
        hk, c, d, q = case["kv_heads"], case["capacity"], case["dim"], case["queries"]
        s["q"] = _randn(g, (b, q, hk * case["group"], d), dtype)
        k = torch.randn((b, hk, c, d), generator=g, device="cuda")
        k += 0.5 * torch.randn((b, hk, c, 1), generator=g, device="cuda") * s["q"][:, :1, ::case["group"]].float().transpose(1, 2)
        s["k"] = k.to(dtype)
        at = _weighed(case)
        s["begin"], s["end"] = _ints([a for a, _ in at]), _ints([z for _, z in at])
        # a few steps' weight, on the scale of what this step adds
        s["scores"] = torch.rand((b, hk, c), generator=g, device="cuda") * (4 * q * case["group"] / c)
        s["out"] = torch.zeros((b, hk, c), device="cuda")
        return s
    h, c, d, n = case["heads"], case["capacity"], case["dim"], case["budget"]
    s["k"], s["v"] = _randn(g, (b, h, c, d), dtype), _randn(g, (b, h, c, d), dtype)
    s["scores"] = torch.exp(2 * torch.randn((b, h, c), generator=g, device="cuda"))
    # a cache that has been cut before: old positions out of order, the newest at the end
    old = torch.argsort(torch.rand((b, h, n), generator=g, device="cuda"), 2) * 2
    new = torch.arange(c - n, device="cuda").expand(b, h, c - n) + 2 * n
    s["positions"] = torch.cat([old, new], 2).to(torch.int32)
    s["lens"] = _ints(_cache_lens(case))
    s["out"] = (torch.zeros((b, h, c), device="cuda"), torch.zeros((b, h, c), dtype=torch.int32, device="cuda"),
                torch.zeros(b, dtype=torch.int32, device="cuda"))
    return s


# ----------------------------------------------------------- the plain forms
def _select(s):
    """Sums of log probabilities in 64 bits (near-equal ones decide), the best of them with ties to the lowest index."""
    b, w, v, k = s["batch"], s["beams"], s["vocab"], s["keep"]
    x = s["logits"][:, :, :v].double() / s["temperature"]
    top = x.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x - top
    x = x - x.exp().sum(2, keepdim=True).log()
    x = torch.where(x.isnan(), -math.inf, x) + s["scores"].double()[:, :, None]
    if s["finished"] is not None:
        x = torch.where(s["finished"][:, :, None] != 0, -math.inf, x)
        x[:, :, s["end"]] = torch.where(s["finished"] != 0, s["scores"].double(), x[:, :, s["end"]])
    x = x.reshape(b, w * v)
    least = torch.topk(x, k, dim=1)[0][:, -1:]
    ties = x == least
    taken = (x > least) | (ties & (ties.cumsum(1, dtype=torch.int32) <= k - (x > least).sum(1, keepdim=True)))
    at = taken.nonzero()[:, 1].reshape(b, k)
    best, order = torch.sort(x.gather(1, at), dim=1, descending=True, stable=True)
    at = at.gather(1, order)
    none = best == -math.inf
    scores, parents, tokens = s["out"]
    scores.copy_(best)
    parents.copy_(torch.where(none, -1, at // v))
    tokens.copy_(torch.where(none, -1, at % v))
    return s["out"]


def _beams(s):
    x, axis = s["all"], s["axis"] + 1
    rows = torch.arange(s["batch"], device="cuda")[:, None]
    at = torch.arange(s["capacity"], device="cuda")
    inside = (at >= s["begin"][:, None]) & (at < s["end"][:, None])
    shape = [1, s["batch"], 1, 1, 1, 1]
    shape[axis] = s["capacity"]
    x.copy_(torch.where(inside.reshape(shape), x[:, rows, s["parents"].long()], x))
    return s["list"]


def _path(s):
    x = s["all"] if s["layout"] == "thd" else s["all"].transpose(2, 3)
    row, i = (s["path"] >= 0).nonzero(as_tuple=True)
    base = s["base"].long()[row]
    x[:, row, base + i] = x[:, row, base + s["path"].long()[row, i]]
    s["lens"].copy_(s["base"] + (s["path"] >= 0).sum(1))
    return s["list"], s["lens"]


def _weight(s):
    b, q, g, hk, d, c = (s[n] for n in ("batch", "queries", "group", "kv_heads", "dim", "capacity"))
    query = s["q"].float().reshape(b, q, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, q * g, d)
    x = torch.matmul(query, s["k"].float().transpose(2, 3)).reshape(b, hk, q, g, c) * d ** -0.5
    at, i = torch.arange(c, device="cuda"), torch.arange(q, device="cuda")
    last = s["begin"][:, None] + i
    seen = (at <= last[:, :, None]) & (last < s["end"][:, None])[:, :, None]
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    top = x.amax(4, keepdim=True)
    x = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = x.sum(4, keepdim=True)
    x = (x / torch.where(total == 0, 1.0, total)).sum((2, 3))
    old = torch.where((at < s["begin"][:, None])[:, None], s["scores"], 0.0)
    s["out"].copy_(torch.where((at < s["end"][:, None])[:, None], old + x, s["out"]))
    return s["out"]


def _evict(s):
    c, budget = s["capacity"], s["budget"]
    scores, positions, lens = s["out"]
    at = torch.arange(c, device="cuda")
    n = s["lens"][:, None, None]
    filled, whole = at < n, n <= budget
    pos = s["positions"]
    newest = torch.where(filled, pos, -1).amax(2, keepdim=True)
    safe = (pos < s["sinks"]) | (pos > newest - s["recent"])
    order = torch.where(filled, torch.where(safe, math.inf, s["scores"]), -1.0)
    best = torch.sort(order, dim=2, descending=True, stable=True)[1][:, :, :budget]
    kept = torch.zeros_like(filled.expand_as(pos)).scatter_(2, best, True) | whole
    source = (kept & (at >= budget) & filled).nonzero(as_tuple=True)
    target = (~kept & (at < budget)).nonzero(as_tuple=True)
    for x in (s["k"], s["v"]):
        x[target] = x[source]
    for x, old in ((scores, s["scores"]), (positions, pos)):
        x.copy_(torch.where(filled & (at < budget), old, x))
        x[target] = old[source]
    lens.copy_(s["lens"].clamp(max=budget))
    return s["k"], s["v"], scores, positions, lens


PLAIN = {"select": _select, "beams": _beams, "path": _path, "weight": _weight, "evict": _evict}


def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    from speculative_decoding_verification_87_b200 import binding as sv
    if s["op"] == "select":
        scores, parents, tokens = s["out"]
        sv.spec_beam_select(s["logits"], s["scores"], s["vocab"], s["keep"], temperature=s["temperature"],
                            finished=s["finished"], end_token=s["end"], out_scores=scores,
                            out_parents=parents, out_tokens=tokens)
        return s["out"]
    if s["op"] == "beams":
        sv.spec_reorder_beams(s["list"], s["parents"], axis=s["axis"], begin=s["begin"], end=s["end"])
        return s["list"]
    if s["op"] == "path":
        sv.spec_commit_path(s["list"], s["base"], s["path"], s["nodes"], axis=s["axis"], out_lens=s["lens"])
        return s["list"], s["lens"]
    if s["op"] == "weight":
        return sv.spec_cache_score(s["q"], s["k"], s["begin"], s["end"], s["scores"], out_scores=s["out"])
    scores, positions, lens = s["out"]
    sv.spec_cache_evict(s["k"], s["v"], s["scores"], s["positions"], s["lens"], s["budget"], sinks=s["sinks"],
                        recent=s["recent"], out_scores=scores, out_positions=positions, out_lens=lens)
    return s["k"], s["v"], scores, positions, lens


# ------------------------------------------------------ the values in 64 bits
def exact(case, seed):
    """Computed numbers from the definitions in 64 bits, request by request; moved rows are no computed numbers."""
    if case["op"] == "select":
        s = prepare(case, seed)
        k, v = case["keep"], case["vocab"]
        scores = []
        for b in range(case["batch"]):
            rows = []
            for w in range(case["beams"]):
                if case["finished"] and int(s["finished"][b, w]):
                    rows.append(s["scores"][b, w].double().reshape(1))
                else:
                    p = torch.log_softmax(s["logits"][b, w, :v].double() / case["temperature"], 0)
                    rows.append(torch.where(p.isnan(), -math.inf, p + s["scores"][b, w].double()))
            rows = torch.cat(rows + [torch.full((k,), -math.inf, dtype=torch.float64, device="cuda")])
            scores.append(torch.topk(rows, k)[0])
        return torch.stack(scores), None, None
    if case["op"] == "weight":
        s = prepare(case, seed)
        out = torch.zeros_like(s["scores"], dtype=torch.float64)
        for b, (begin, end) in enumerate(_weighed(case)):
            old = s["scores"][b, :, :end].double()
            old[:, begin:] = 0
            for h in range(case["kv_heads"]):
                k = s["k"][b, h, :end].double()
                for i in range(end - begin):
                    q = s["q"][b, i, h * case["group"]:(h + 1) * case["group"]].double()
                    x = q @ k[:begin + i + 1].T / math.sqrt(case["dim"])
                    old[h, :begin + i + 1] += torch.softmax(x, 1).sum(0)
            out[b, :, :end] = old
        return out
    return None
