"""spec_cache_score and spec_cache_evict against the plain 64-bit
implementations.  Score tolerances are the bounds that state_ref.cache_score
derives, with `unit` 2^-23 an addition (tensor-core sums may truncate: a
whole step, not half).  Eviction moves bytes: exact."""
import numpy as np
import pytest
import torch

import state_ref as ref

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -23


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from speculative_decoding_verification_87_b200 import binding, build
    build.build()
    binding.load_library()
    return binding


def ints(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def make(seed, B, Q, G, H, D, C, dtype):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Q, H * G, D), generator=g).to(dtype)
    k = torch.randn((B, H, C, D), generator=g).to(dtype)
    return q, k, torch.rand((B, H, C), generator=g)


def check_score(sv, q, k, begin, end, scores, scale=None, inplace=False, transpose=False):
    B, H, C, D = k.shape
    begin, end = np.asarray(begin), np.asarray(end)
    for b in range(B):  # rows behind the last slot may hold anything
        k[b, :, int(end[b]):] = float("nan")
        scores[b, :, int(begin[b]):] = float("nan")
        q[b, int(end[b] - begin[b]):] = float("nan")
    kd = k.cuda()
    if transpose:
        kd = kd.transpose(1, 2).contiguous().transpose(1, 2)
    sc = scores.cuda()
    out = sc if inplace else torch.full_like(sc, -7.0)
    status = ints([0])
    got = sv.spec_cache_score(q.cuda(), kd, ints(begin), ints(end), sc, scale, out, status)
    assert got is out and status.item() == 0
    want, bound = ref.cache_score(q.double().numpy(), k.double().numpy(), begin, end, scores.double().numpy(),
                                  D ** -0.5 if scale is None else scale, UNIT)
    got = got.cpu().numpy()
    for b in range(B):
        n = int(end[b])
        assert np.all(np.abs(got[b, :, :n] - want[b, :, :n]) <= bound[b, :, :n]), b
        rest = got[b, :, n:]
        assert np.all(np.isnan(rest)) if inplace else np.all(rest == -7.0)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, Q, G, H, D, C", [
    (1, 1, 1, 1, 8, 1), (2, 1, 4, 2, 64, 130), (3, 5, 1, 2, 128, 300), (2, 9, 8, 1, 64, 257), (1, 32, 4, 2, 128, 700),
    (2, 3, 7, 2, 80, 129), (2, 2, 2, 3, 40, 128), (1, 4, 3, 1, 256, 1000), (4, 1, 16, 2, 128, 2050), (1, 64, 2, 1, 16, 200),
    (1, 17, 5, 1, 96, 515), (1, 1, 1, 2, 128, 9000),
])
def test_score(sv, dtype, B, Q, G, H, D, C):
    q, k, s = make(B + 7 * Q + C, B, Q, G, H, D, C, dtype)
    r = np.random.RandomState(C)
    end = r.randint(min(Q, C), C + 1, B)
    end[0] = C
    count = np.array([min(e, r.randint(0, Q + 1)) for e in end])
    count[0] = min(Q, C)
    check_score(sv, q.clone(), k.clone(), end - count, end, s.clone())
    check_score(sv, q, k, end - count, end, s, inplace=True, transpose=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_score_from_an_empty_cache(sv, dtype):
    q, k, s = make(3, 3, 6, 2, 2, 64, 9, dtype)
    check_score(sv, q, k, [0, 0, 3], [6, 0, 3], s)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_score_scales(sv, dtype, scale):
    # scale 4: weights from 1 down to zero in fp32
    q, k, s = make(5, 2, 3, 4, 2, 64, 200, dtype)
    check_score(sv, q, k, [197, 100], [200, 102], s, scale)


@pytest.mark.parametrize("B, Q, G, H, D, C, scale", [
    (2, 40, 7, 1, 128, 1500, None), (3, 13, 4, 2, 112, 4000, None), (1, 128, 1, 2, 64, 1025, None),
    (9, 12, 8, 4, 128, 700, None), (1, 49, 1, 1, 8, 49, None), (2, 32, 4, 1, 72, 300, -0.3), (1, 64, 2, 1, 128, 260, 0.0),
    (1, 200, 2, 1, 32, 900, 2.0), (150, 16, 3, 1, 64, 40, None), (1, 6, 8, 1, 128, 20000, None),
])
def test_score_many_rows(sv, B, Q, G, H, D, C, scale):
    q, k, s = make(B + 3 * Q + C, B, Q, G, H, D, C, torch.bfloat16)
    r = np.random.RandomState(C + Q)
    end = r.randint(min(Q, C), C + 1, B)
    end[0] = C
    count = np.array([min(e, r.randint(0, Q + 1)) for e in end])
    count[0] = min(Q, C)
    check_score(sv, q, k, end - count, end, s, scale, inplace=bool(B % 2), transpose=bool(Q % 2))


@pytest.mark.parametrize("B, Q, G, H, D, C, scale", [
    (2, 40, 7, 1, 128, 900, None), (1, 13, 4, 2, 112, 3000, None), (1, 70, 1, 2, 64, 1025, None), (1, 33, 1, 1, 8, 49, None),
    (2, 32, 4, 1, 72, 300, -0.3), (1, 64, 2, 1, 256, 260, 0.0), (1, 100, 2, 1, 36, 500, 2.0), (60, 16, 3, 1, 64, 40, None),
])
def test_score_many_rows_f32(sv, B, Q, G, H, D, C, scale):
    q, k, s = make(B + 3 * Q + C, B, Q, G, H, D, C, torch.float32)
    r = np.random.RandomState(C + Q)
    end = r.randint(min(Q, C), C + 1, B)
    end[0] = C
    count = np.array([min(e, r.randint(0, Q + 1)) for e in end])
    count[0] = min(Q, C)
    check_score(sv, q, k, end - count, end, s, scale, inplace=bool(B % 2), transpose=bool(Q % 2))


@pytest.mark.parametrize("dtype, B, Q, G, H, D, C", [
    # rows and slots on either side of the choice between stored products and a second sweep
    (torch.bfloat16, 8, 5, 4, 8, 128, 4096), (torch.bfloat16, 8, 5, 4, 8, 128, 4095), (torch.bfloat16, 8, 2, 16, 8, 128, 4096),
    (torch.bfloat16, 2, 1, 17, 16, 64, 8192), (torch.bfloat16, 3, 2, 8, 2, 128, 515), (torch.bfloat16, 3, 17, 1, 2, 128, 515),
    (torch.bfloat16, 1, 16, 1, 2, 256, 700), (torch.float32, 1, 16, 2, 2, 64, 700), (torch.float32, 1, 11, 3, 2, 64, 700),
])
def test_score_between_few_and_many_rows(sv, dtype, B, Q, G, H, D, C):
    q, k, s = make(B + 5 * Q + C, B, Q, G, H, D, C, dtype)
    end = np.array([C - 700 * b // B * (C > 1000) for b in range(B)])
    check_score(sv, q, k, end - np.minimum(Q, end), end, s)


def test_score_many_rows_nan_inf(sv):
    q, k, s = make(8, 1, 20, 4, 3, 64, 400, torch.bfloat16)
    k[0, 1, 150, 3] = float("nan")
    q[0, 7, 9, 0] = float("inf")          # one row of head 2's group
    k[0, 0, :, 5] = float(torch.finfo(torch.bfloat16).min)   # the lowest value everywhere: equal products
    q[0, :, :4, 5] = 1.0
    out = sv.spec_cache_score(q.cuda(), k.cuda(), ints([380]), ints([400]), s.cuda()).cpu()
    assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1]).all()
    # the row of query 7 sees slots up to 387; later ones belong to other rows
    assert torch.isnan(out[0, 2, :388]).all() and torch.isfinite(out[0, 2, 388:]).all()


def test_score_strides(sv):
    # heads and tokens of q and k inside larger tensors, slots apart
    q, k, s = make(6, 2, 3, 2, 2, 64, 100, torch.bfloat16)
    qq = torch.zeros((2, 3, 6, 72), dtype=torch.bfloat16)
    qq[:, :, 1:5, 8:] = q
    kk = torch.zeros((2, 3, 2, 100, 72), dtype=torch.bfloat16)
    kk[:, 1, :, :, :64] = k
    begin, end = ints([97, 50]), ints([100, 52])
    a = sv.spec_cache_score(q.cuda(), k.cuda(), begin, end, s.cuda())
    b = sv.spec_cache_score(qq.cuda()[:, :, 1:5, 8:], kk.cuda()[:, 1, :, :, :64], begin, end, s.cuda())
    assert torch.equal(a, b)
    # a query shared by all requests and heads (stride 0)
    one = q[:1, :, :1].cuda()
    c = sv.spec_cache_score(one.expand(2, 3, 4, 64), k.cuda(), begin, end, s.cuda())
    d = sv.spec_cache_score(one.expand(2, 3, 4, 64).contiguous(), k.cuda(), begin, end, s.cuda())
    assert torch.equal(c, d)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_cache_score(q.cuda()[..., :60], k.cuda()[..., :60], begin, end, s.cuda())


def test_score_bad_windows(sv):
    q, k, s = make(7, 5, 2, 1, 1, 64, 40, torch.bfloat16)
    begin, end = [38, -1, 5, 39, 10], [40, 1, 4, 41, 13]
    status, sc = ints([0]), s.cuda()
    out = sv.spec_cache_score(q.cuda(), k.cuda(), ints(begin), ints(end), sc, status=status)
    assert status.item() == 16 and torch.equal(out[1:].cpu(), s[1:]) and not torch.equal(out[0].cpu(), s[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_score_nan_stays_in_its_head(sv, dtype):
    q, k, s = make(8, 1, 2, 2, 3, 64, 150, dtype)
    k[0, 1, 20, 3] = float("nan")
    q[0, 1, 5, 0] = float("nan")        # head 2's group, query 1
    out = sv.spec_cache_score(q.cuda(), k.cuda(), ints([148]), ints([150]), s.cuda()).cpu()
    assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 2]).all()


def test_score_does_not_depend_on_the_run(sv):
    q, k, s = make(9, 4, 8, 4, 2, 128, 3001, torch.bfloat16)
    q, k, s = q.cuda(), k.cuda(), s.cuda()
    begin, end = ints([2993, 1, 500, 2000]), ints([3001, 9, 508, 2003])
    a = sv.spec_cache_score(q, k, begin, end, s, out_scores=torch.zeros_like(s))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [sv.spec_cache_score(q, k, begin, end, s, out_scores=torch.zeros_like(s), stream=st) for st in streams]
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sv.spec_cache_score(q, k, begin, end, s, out_scores=out)
    graph.replay()
    torch.cuda.synchronize()
    for o in outs + [out]:
        assert torch.equal(o, a)


# ------------------------------------------------------------------ eviction
def check_evict(sv, scores, positions, lens, budget, sinks=0, recent=0, D=16, Dv=16, dtype=torch.bfloat16,
                inplace=False, transpose=False, status_want=0, seed=0):
    B, H, C = scores.shape
    g = torch.Generator().manual_seed(seed)
    k = torch.randint(-100, 100, (B, H, C, D), generator=g).to(dtype)
    v = torch.randint(-100, 100, (B, H, C, Dv), generator=g).to(dtype)
    kd, vd = k.cuda(), v.cuda()
    if transpose:
        kd, vd = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kd, vd))
    sc, po, ln = torch.from_numpy(scores).cuda(), ints(positions), ints(lens)
    osc = sc if inplace else torch.full_like(sc, -7.0)
    opo = po if inplace else torch.full_like(po, -7)
    oln = ln if inplace else torch.full_like(ln, -7)
    status = ints([0])
    got = sv.spec_cache_evict(kd, vd, sc, po, ln, budget, sinks, recent, osc, opo, oln, status)
    assert got[0] is osc and got[1] is opo and got[2] is oln
    rk, rv, rs, rp, rl = ref.evict(k.float().numpy(), v.float().numpy(), scores, np.asarray(positions),
                                   np.asarray(lens, np.int32), budget, sinks, recent)
    assert np.array_equal(kd.cpu().float().numpy(), rk) and np.array_equal(vd.cpu().float().numpy(), rv)
    assert np.array_equal(oln.cpu().numpy(), rl) and status.item() == status_want
    for b in range(B):
        n = rl[b]
        assert np.array_equal(osc.cpu().numpy()[b, :, :n].view(np.int32), rs[b, :, :n].view(np.int32))
        assert np.array_equal(opo.cpu().numpy()[b, :, :n], rp[b, :, :n])
        if not inplace:
            assert np.all(osc.cpu().numpy()[b, :, n:] == -7.0) and np.all(opo.cpu().numpy()[b, :, n:] == -7)


def cache(seed, B, H, C):
    r = np.random.RandomState(seed)
    scores = np.exp(2 * r.randn(B, H, C)).astype(np.float32)
    pos = np.stack([np.stack([r.permutation(2 * C)[:C] for _ in range(H)]) for _ in range(B)]).astype(np.int32)
    return scores, pos


@pytest.mark.parametrize("B, H, C, budget, sinks, recent", [
    (1, 1, 1, 1, 0, 0), (1, 1, 2, 1, 0, 1), (2, 3, 40, 32, 2, 8), (3, 2, 100, 99, 4, 50), (2, 2, 1000, 1, 0, 0),
    (1, 2, 4096, 4000, 0, 0), (2, 1, 4097, 2048, 16, 100), (1, 3, 9000, 300, 1, 1), (1, 2, 40000, 20000, 4, 64),
    (5, 8, 261, 256, 4, 64), (2, 2, 50, 60, 3, 3),
])
def test_evict(sv, B, H, C, budget, sinks, recent):
    scores, pos = cache(C + budget, B, H, C)
    r = np.random.RandomState(C)
    lens = r.randint(0, C + 1, B)
    lens[0] = C
    check_evict(sv, scores, pos, lens, budget, sinks, recent)
    check_evict(sv, scores, pos, lens, budget, sinks, recent, inplace=True, transpose=True)


@pytest.mark.parametrize("B, H, C, budget", [
    # moves and heads on either side of the choice between one kernel and two
    (2, 2, 400, 272), (2, 2, 400, 271), (16, 8, 900, 450), (127, 1, 900, 450), (16, 8, 4096, 2048), (130, 1, 300, 20),
])
def test_evict_between_one_kernel_and_two(sv, B, H, C, budget):
    scores, pos = cache(C + budget + B, B, H, C)
    lens = np.random.RandomState(B).randint(0, C + 1, B)
    lens[0] = C
    check_evict(sv, scores, pos, lens, budget, 2, 10)
    check_evict(sv, scores, pos, lens, budget, 2, 10, inplace=True)


@pytest.mark.parametrize("B, H, C, budget", [(16, 8, 1024, 512), (16, 8, 1026, 513), (51, 5, 1400, 700), (64, 4, 1400, 700)])
def test_evict_of_many_moves_in_one_kernel_or_two(sv, B, H, C, budget):
    scores, pos = cache(C + budget + B, B, H, C)
    lens = np.random.RandomState(B).randint(0, C + 1, B)
    lens[0] = C
    check_evict(sv, scores, pos, lens, budget, 2, 10)
    check_evict(sv, scores, pos, lens, budget, 2, 10, inplace=True)


@pytest.mark.parametrize("dtype, D, Dv", [(torch.float32, 1, 3), (torch.bfloat16, 5, 16), (torch.int8, 7, 1),
                                          (torch.float32, 128, 64), (torch.bfloat16, 576, 512), (torch.int8, 20, 4)])
def test_evict_rows(sv, dtype, D, Dv):
    scores, pos = cache(1, 2, 2, 90)
    check_evict(sv, scores, pos, [90, 70], 64, 2, 4, D, Dv, dtype)


def test_evict_ties_and_special_scores(sv):
    scores, pos = cache(2, 2, 3, 500)
    scores[0, 0] = 1.0                                   # all equal: the lowest slots stay
    scores[0, 1, ::2] = 0.0
    scores[0, 1, 1::2] = -0.0                            # both zeros tie
    scores[0, 2] = np.round(scores[0, 2])                # many ties at the border
    scores[1, 0, ::3] = -np.inf
    scores[1, 0, 1::3] = np.inf
    scores[1, 1] = -scores[1, 1]
    check_evict(sv, scores, pos, [500, 500], 200, 0, 0)
    check_evict(sv, scores, pos, [500, 500], 200, 10, 30)
    scores[1, 2, 100:400] = np.nan                       # NaN goes first
    check_evict(sv, scores, pos, [500, 500], 230, 0, 5, status_want=4)
    scores[1, 2] = np.nan
    check_evict(sv, scores, pos, [500, 500], 100, 0, 5, status_want=4)


def test_evict_same_position_twice(sv):
    # more protected slots than fit: the lowest slots of them
    scores, pos = cache(3, 1, 2, 300)
    pos[0, 0] = 0
    pos[0, 1, 100:] = 10 ** 6
    check_evict(sv, scores, pos, [300], 60, 2, 20)


def test_evict_leaves_bad_requests(sv):
    scores, pos = cache(4, 3, 2, 60)
    k = torch.rand((3, 2, 60, 8), device="cuda")
    old, sc, po, status = k.clone(), torch.from_numpy(scores).cuda(), ints(pos), ints([0])
    s, p, n = sv.spec_cache_evict(k, None, sc, po, ints([-1, 61, 60]), 20, status=status)
    assert status.item() == 16 and n.tolist() == [-1, 61, 20]
    assert torch.equal(k[:2], old[:2]) and np.array_equal(s.cpu().numpy()[:2], scores[:2])
    assert np.array_equal(p.cpu().numpy()[:2], pos[:2])
    want = ref.evict(old.cpu().numpy()[2:], old.cpu().numpy()[2:], scores[2:], pos[2:], np.array([60]), 20, 0, 0)
    assert np.array_equal(k.cpu().numpy()[2:], want[0]) and np.array_equal(s.cpu().numpy()[2:, :, :20], want[2][:, :, :20])


def test_evict_large(sv):
    # the largest slot count, eight blocks a head
    scores, pos = cache(5, 1, 1, 262144)
    check_evict(sv, scores, pos, [262144], 100000, 4, 1000, D=8, Dv=8)
    check_evict(sv, scores, pos, [262143], 262142, 4, 1000, D=8, Dv=8)


def test_evict_streams_and_a_graph(sv):
    scores, pos = cache(6, 2, 4, 5000)
    k = torch.rand((2, 4, 5000, 64), device="cuda")
    v = torch.rand_like(k)
    sc, po, ln = torch.from_numpy(scores).cuda(), ints(pos), ints([5000, 4100])

    def out():
        return torch.zeros_like(sc), torch.zeros_like(po), torch.zeros_like(ln)

    k0, v0, o0 = k.clone(), v.clone(), out()
    sv.spec_cache_evict(k0, v0, sc, po, ln, 4000, 4, 100, *o0)
    runs = []
    torch.cuda.synchronize()
    for st in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(st):
            runs.append((k.clone(), v.clone(), out()))
            sv.spec_cache_evict(runs[-1][0], runs[-1][1], sc, po, ln, 4000, 4, 100, *runs[-1][2])
    torch.cuda.synchronize()
    k1, v1, o1 = k.clone(), v.clone(), out()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_cache_evict(k1, v1, sc, po, ln, 4000, 4, 100, *o1)
    graph.replay()
    torch.cuda.synchronize()
    for a, c, o in runs + [(k1, v1, o1)]:
        assert torch.equal(a, k0) and torch.equal(c, v0) and all(torch.equal(x, y) for x, y in zip(o, o0))


# ------------------------------------------------------- offsets past 32 bits
def test_strides_past_32_bits(sv):
    # slots 2^27 elements apart: the last one starts 5 * 2^30 elements in
    step, n = 1 << 27, 40
    store = torch.empty(step * n, dtype=torch.bfloat16, device="cuda")
    k = store.as_strided((1, 1, n, 64), (0, 0, step, 1))
    q, small, s = make(3, 1, 2, 2, 1, 64, n, torch.bfloat16)
    k.copy_(small)
    got = sv.spec_cache_score(q.cuda(), k, ints([38]), ints([40]), s.cuda())
    want = sv.spec_cache_score(q.cuda(), small.cuda(), ints([38]), ints([40]), s.cuda())
    assert torch.equal(got, want)
    big = torch.randn((1, 40, 2, 64)).to(torch.bfloat16)      # 80 rows: the sweeps for many
    got = sv.spec_cache_score(big.cuda(), k, ints([0]), ints([40]), s.cuda())
    want = sv.spec_cache_score(big.cuda(), small.cuda(), ints([0]), ints([40]), s.cuda())
    assert torch.equal(got, want)
    scores, pos = cache(7, 1, 1, n)
    args = torch.from_numpy(scores).cuda(), ints(pos), ints([n]), 25, 2, 5
    dense = small.cuda()
    a = sv.spec_cache_evict(k, None, *[x.clone() if torch.is_tensor(x) else x for x in args])
    b = sv.spec_cache_evict(dense, None, *[x.clone() if torch.is_tensor(x) else x for x in args])
    assert torch.equal(k.contiguous(), dense) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    beams = store.as_strided((1, n, 64), (0, step, 1))        # the same rows as beams of one request
    par = torch.randperm(n, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None].cuda()
    want = beams[:, par[0].long()].clone()
    sv.spec_reorder_beams([beams], par)
    assert torch.equal(beams, want)


def test_workspaces_and_devices(sv):
    q, k, s = make(4, 1, 2, 2, 1, 64, 100, torch.bfloat16)
    q, k, s = q.cuda(), k.cuda(), s.cuda()
    need = sv.load_library().spec_score_workspace_size(1, 2, 2, 1, 100)
    begin, end = ints([98]), ints([100])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = sv.spec_cache_score(q, k, begin, end, s.clone(), workspace_buf=ws)
    assert torch.equal(a, sv.spec_cache_score(q, k, begin, end, s.clone()))
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_cache_score(q, k, begin, end, s, workspace_buf=ws[:need - 256])
    with pytest.raises(ValueError):
        sv.spec_cache_score(q, k.cpu(), begin, end, s)
    with pytest.raises(ValueError):
        sv.spec_cache_score(q, k, begin.cpu(), end, s)
    with pytest.raises(TypeError):
        sv.spec_cache_score(q.half(), k.half(), begin, end, s)
    with pytest.raises(ValueError):
        sv.spec_cache_evict(k, k[:, :, :50], s, ints(np.zeros((1, 1, 100))), end, 10)
