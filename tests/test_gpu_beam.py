"""spec_beam_select against the plain 64-bit implementation.

Parents and tokens have to be the documented ones exactly.  Scores: the sum
of the row's exponentials is off by at most 6e-6 (the kernel's own bound,
below which it recomputes what the order depends on), then one rounding to
fp32, half a step: 2^-24 of the value.
"""
import numpy as np
import pytest
import torch

import state_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from speculative_decoding_verification_87_b200 import binding, build
    build.build()
    binding.load_library()
    return binding


def check(sv, logits, scores, vocab, keep, temperature=1.0, finished=None, end_token=-1):
    """One call against the reference; logits and scores are CPU tensors."""
    fin = None if finished is None else finished.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s, p, t, f = sv.spec_beam_select(logits.cuda(), scores.cuda(), vocab, keep, temperature, fin, end_token,
                                     status=status)
    rs, rp, rt, rf, bad = ref.beam_select(logits.double().numpy(), scores.double().numpy(), vocab, keep,
                                          float(np.float32(temperature)),
                                          None if finished is None else finished.numpy(), end_token)
    s, p, t = s.cpu().numpy().astype(np.float64), p.cpu().numpy(), t.cpu().numpy()
    assert np.array_equal(p, rp) and np.array_equal(t, rt)
    real = rp >= 0
    assert np.all(s[~real] == -np.inf)
    assert np.all(np.abs(s[real] - rs[real]) <= 6e-6 + 2.0 ** -24 * np.abs(rs[real]))
    if f is not None:
        assert np.array_equal(f.cpu().numpy(), rf)
    assert int(status.item()) == (4 if bad.any() else 0)
    return s, p, t


def rows(seed, B, W, V, dtype, pad=0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    vec = 8 if dtype == torch.bfloat16 else 4
    stride = -(-V // vec) * vec + pad * vec
    x = torch.randn((B, W, stride), generator=g) * scale
    hot = torch.randint(0, V, (B, W, 4), generator=g)
    x.scatter_add_(2, hot, torch.full((B, W, 4), 8.0))
    x[:, :, V:] = float("nan")  # columns past the vocabulary are not read
    scores = torch.sort(torch.randn((B, W), generator=g) - 5, descending=True)[0]
    return x.to(dtype), scores


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, W, K, V, T, pad", [
    (1, 1, 1, 1, 1.0, 0), (2, 3, 4, 7, 1.0, 1), (3, 5, 9, 33, 0.7, 0), (1, 4, 4, 1024, 1.0, 0),
    (2, 4, 8, 1025, 1.0, 3), (2, 4, 8, 2048, 1.3, 0), (3, 2, 5, 2049, 1.0, 0), (5, 7, 14, 50257, 0.7, 2),
    (2, 16, 16, 32000, 1.0, 0), (1, 64, 64, 5003, 1.0, 0), (1, 3, 6, 128256, 1.0, 0), (37, 1, 2, 300, 0.01, 0),
    (2, 4, 8, 4001, 50.0, 0), (1, 2, 64, 20, 1.0, 0),
])
def test_select(sv, dtype, B, W, K, V, T, pad):
    x, s = rows(B * 1000 + V, B, W, V, dtype, pad)
    check(sv, x, s, V, K, T)


@pytest.mark.parametrize("seed", range(12))
def test_select_random(sv, seed):
    r = np.random.RandomState(seed)
    B, W, V = r.randint(1, 9), r.randint(1, 33), int(np.exp(r.uniform(np.log(3), np.log(40000))))
    K = r.randint(1, min(64, 2 * W) + 1)
    dtype = torch.bfloat16 if seed % 2 else torch.float32
    x, s = rows(seed, B, W, V, dtype, r.randint(0, 3), scale=r.choice([0.1, 3.0]))
    fin = torch.from_numpy((r.rand(B, W) < 0.3).astype(np.int32)) if seed % 3 == 0 else None
    check(sv, x, s, V, K, r.choice([0.5, 1.0, 2.0]), fin, V - 1 if fin is not None else -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, W, K, V", [(2, 4, 4, 300), (1, 3, 64, 5000), (1, 64, 64, 6000), (1, 2, 16, 70001)])
def test_equal_candidates_go_to_the_lowest_index(sv, dtype, B, W, K, V):
    # constant rows: every candidate of a beam ties
    x = torch.zeros((B, W, -(-V // 8) * 8), dtype=dtype)
    check(sv, x, torch.linspace(-1, -9, W).repeat(B, 1), V, K)
    # and equal beams on top: every candidate of the request ties
    check(sv, x, torch.full((B, W), -2.5), V, K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, W, K, V", [(2, 1, 16, 2000), (3, 1, 64, 5000), (2, 3, 64, 1500), (20, 20, 10, 4006), (1, 2, 33, 1024),
                                        (2, 1, 64, 70), (1, 1, 40, 32001)])
def test_fewer_items_than_beams_kept(sv, dtype, B, W, K, V):
    x, s = rows(V + K, B, W, V, dtype)
    check(sv, x, s, V, K)
    m = torch.rand(x.shape, generator=torch.Generator().manual_seed(2)) < 0.9
    x[m] = -float("inf")
    x[:, :, 0] = 0.0
    check(sv, x, s, V, K, 0.6)


def test_ties_inside_and_across_items(sv):
    # a few values only, so that the K-th best ties with many others
    g = torch.Generator().manual_seed(3)
    for V, K in ((9000, 5), (9000, 33), (2048, 16), (2047, 17)):
        x = torch.randint(-3, 3, (2, 4, -(-V // 8) * 8), generator=g).to(torch.bfloat16)
        x[:, :, 100:108] = 4.0
        check(sv, x, torch.tensor([[-1.0, -1.0, -2.0, -1.0]] * 2), V, K)


@pytest.mark.parametrize("gap", [0.0, 1e-7, 1e-6, 3e-6, 1e-5])
def test_beams_that_nearly_tie(sv, gap):
    # the same row under scores a few fp32 steps apart: the order has to be that
    # of the exact scores, far below what fp32 sums of exponentials resolve
    x, _ = rows(11, 2, 1, 9001, torch.float32)
    x = x.repeat(1, 4, 1)
    s = torch.tensor([[-3.0, -3.0 + gap, -3.0 + 2 * gap, -3.0 - gap]] * 2)
    check(sv, x, s, 9001, 16)
    # permuted columns: sums of the same numbers in another order.  Not for
    # gaps below half an fp32 step of 3 (2^-23 = 1.2e-7): -3 + gap rounds to -3,
    # the two sums are one real number and differ in fp64 rounding alone, which
    # the order documented does not reach
    y = x.clone()
    perm = torch.randperm(9001, generator=torch.Generator().manual_seed(1))
    y[:, 1, :9001] = x[:, 1, :9001][:, perm]
    if gap >= 2.0 ** -22:
        check(sv, y, s, 9001, 16)


def test_masked_rows_and_unused_beams(sv):
    inf = float("inf")
    x, s = rows(5, 3, 4, 777, torch.float32)
    x[0, 1, :777] = -inf                      # nothing to go on with
    x[1, :, :777] = -inf                      # a whole request with nothing
    x[2, :, 5:777] = -inf                     # 5 candidates a beam
    x[2, 1, :5] = -inf
    x[2, 2, :5] = torch.finfo(torch.float32).min   # the type's lowest value is a value
    s[0, 2] = -inf                            # a beam that is not in use
    s[2, 3] = -inf
    sc, p, t = check(sv, x, s, 777, 12)
    assert np.all(p[1] == -1) and not np.any(p[0] == 1) and not np.any(p[0] == 2)
    assert np.sum(p[2] >= 0) == 10            # beam 0: five, beam 2: five that tie
    # rows that are not read may hold anything
    x[0, 2], x[2, 3] = float("nan"), inf
    check(sv, x, s, 777, 12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_masked_by_the_lowest_value(sv, dtype):
    # whole items of it, a row of nothing else, and the type's largest beside it
    x, s = rows(6, 2, 4, 9000, dtype)
    low = torch.finfo(dtype).min
    x[:, 0, 50:9000] = low
    x[:, 1, :9000] = low
    x[:, 2, 4100:] = low
    x[1, 3, 17] = torch.finfo(dtype).max
    check(sv, x, s, 9000, 16)
    check(sv, x, s, 9000, 64, 0.25)


@pytest.mark.parametrize("T, scale", [(1e-6, 3.0), (1e-4, 3.0), (1.0, 3e4), (1e-3, 1e3), (1e-20, 1.0), (1e6, 3.0)])
def test_extreme_temperatures_and_logits(sv, T, scale):
    # products log2(e) l / T from 1e-6 to 1e21: the rounding of the largest must not reach the sums.
    # (Far larger T bring differences of scores, 1e-6 / T for fp32 logits near 10, below
    # fp64's step at the scores' size, 2e-15: there the documented order is none.)
    x, s = rows(7, 2, 3, 3001, torch.float32, scale=scale)
    check(sv, x, s, 3001, 5, T)
    check(sv, x.to(torch.bfloat16)[:, :, :3000].contiguous(), s, 3000, 5, T)


def test_finished_beams(sv):
    x, s = rows(8, 3, 5, 1500, torch.bfloat16)
    fin = torch.zeros((3, 5), dtype=torch.int32)
    fin[0] = 1                                # all ended: the beams themselves, in order
    fin[1, 1] = 7
    fin[2, 0] = 1
    s[2, 0] = -float("inf")
    x[0] = float("nan")
    check(sv, x, s, 1500, 5, 1.0, fin, 42)
    check(sv, x, s, 1500, 8, 1.0, fin, 0)
    # an end token without ended beams: out_finished on request
    out = torch.empty((3, 5), dtype=torch.int32, device="cuda")
    x[0] = 0.0
    _, _, t, f = sv.spec_beam_select(x.cuda(), s.cuda(), 1500, 5, end_token=3, out_finished=out)
    assert f is out and torch.equal(f, (t == 3).int())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("ended", [1, 2, 4])
def test_ended_beams_with_bad_scores(sv, value, ended):
    # candidates that no order ranks: more of them than one
    x, s = rows(19, 3, 4, 1200, torch.bfloat16)
    fin = torch.zeros((3, 4), dtype=torch.int32)
    fin[:, :ended] = 1
    s[1, :ended] = value
    s[1, 0] = 0.25 if ended == 4 else value
    _, p, _ = check(sv, x, s, 1200, 6, 1.0, fin, 11)
    assert np.all(p[1] == -1) and np.all(p[[0, 2], 0] >= 0)


@pytest.mark.parametrize("where", ["nan", "inf", "score nan", "score inf"])
def test_bad_inputs_are_reported(sv, where):
    x, s = rows(9, 3, 3, 2500, torch.float32)
    if where == "nan":
        x[1, 2, 2499] = float("nan")
    elif where == "inf":
        x[1, 0, 17] = float("inf")
    else:
        s[1, 1] = float(where.split()[1])
    _, p, _ = check(sv, x, s, 2500, 3)
    assert np.all(p[1] == -1) and np.all(p[[0, 2]] >= 0)


def test_outputs_over_inputs_and_determinism(sv):
    x, s = rows(21, 4, 6, 6001, torch.bfloat16)
    a = sv.spec_beam_select(x.cuda(), s.cuda(), 6001, 6)
    for _ in range(3):
        sc = s.cuda()
        b = sv.spec_beam_select(x.cuda(), sc, 6001, 6, out_scores=sc)
        assert b[0] is sc
        for u, v in zip(a[:3], b[:3]):
            assert torch.equal(u, v)


def test_two_streams_and_a_graph(sv):
    x, s = rows(31, 3, 4, 20001, torch.bfloat16)
    y, u = rows(32, 3, 4, 20001, torch.bfloat16)
    want = [sv.spec_beam_select(a.cuda(), c.cuda(), 20001, 4) for a, c in ((x, s), (y, u))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = [(a.cuda(), c.cuda()) for a, c in ((x, s), (y, u))]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [sv.spec_beam_select(a, c, 20001, 4, stream=st) for (a, c), st in zip(dev, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(i, j) for i, j in zip(w[:3], g[:3]))
    # captured: two steps that feed each other, replayed on new contents
    lx, sc = dev[0][0].clone(), dev[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s1, p1, t1, _ = sv.spec_beam_select(lx, sc, 20001, 4)
        s2, p2, t2, _ = sv.spec_beam_select(lx, s1, 20001, 4)
    for a, c in dev:
        lx.copy_(a)
        sc.copy_(c)
        graph.replay()
        e1 = sv.spec_beam_select(a, c, 20001, 4)
        e2 = sv.spec_beam_select(a, e1[0], 20001, 4)
        torch.cuda.synchronize()
        assert torch.equal(s1, e1[0]) and torch.equal(t1, e1[2])
        assert torch.equal(s2, e2[0]) and torch.equal(p2, e2[1]) and torch.equal(t2, e2[2])


def test_a_beam_search_over_several_steps(sv):
    # sums over steps, beams that fork and die, against the reference fed
    # with the library's own scores
    g = torch.Generator().manual_seed(77)
    B, W, V = 2, 5, 3001
    scores = torch.full((B, W), -float("inf"))
    scores[:, 0] = 0.0
    fin = torch.zeros((B, W), dtype=torch.int32)
    for step in range(6):
        x = (torch.randn((B, W, 3008), generator=g) * 3).to(torch.bfloat16)
        x[:, :, 9] += 6.0
        sc, p, t = check(sv, x, scores, V, W, 1.0, fin, 9)
        fin = torch.from_numpy((t == 9).astype(np.int32))
        scores = torch.from_numpy(sc.astype(np.float32))


def rounded(x):
    """Exact scores as fp32 holds them: past its range, the infinity of their sign."""
    with np.errstate(over="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("dtype, W, V, K, T, at, peak", [
    (torch.float32, 1, 5000, 6, 0.7, 2100, None), (torch.float32, 1, 1500, 64, 0.5, 1100, None),
    (torch.float32, 3, 5000, 20, 0.3, 4800, None), (torch.bfloat16, 1, 3048, 6, 0.7, 2100, None),
    (torch.bfloat16, 2, 3000, 12, 0.25, 2500, None), (torch.float32, 1, 128256, 8, 0.9, 127500, None),
    (torch.float32, 2, 2000, 9, 1.0, 1500, "max"), (torch.float32, 2, 5000, 9, 1.5, 1100, None),
])
def test_few_allowed_beside_the_lowest_value(sv, dtype, W, V, K, T, at, peak):
    # constrained decoding that masks with the type's lowest value: three tokens
    # a row may be taken, the rest of the K go to masked ones in index order,
    # although their scores lie past fp32's range (T < 1, or beside the largest)
    x = torch.full((2, W, -(-V // 8) * 8), torch.finfo(dtype).min, dtype=dtype)
    x[:, :, at:at + 3] = torch.tensor([1.0, 2.0, 3.0], dtype=dtype)
    if peak:
        x[:, :, at + 1] = torch.finfo(dtype).max
    x[1, :, 2] = -float("inf")      # not even a masked one
    s = torch.linspace(-1, -3, W).repeat(2, 1)
    got, p, t, _ = sv.spec_beam_select(x.cuda(), s.cuda(), V, K, T)
    rs, rp, rt, _, _ = ref.beam_select(x.double().numpy(), s.double().numpy(), V, K, float(np.float32(T)))
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)
    got, want = got.cpu().numpy().astype(np.float64), rounded(rs)
    real = np.isfinite(want)
    assert np.array_equal(got[~real], want[~real])
    assert np.all(np.abs(got[real] - rs[real]) <= 6e-6 + 2.0 ** -24 * np.abs(rs[real]))
    assert T > 1 or np.any(~real & (rp >= 0))    # some are past the range and are still candidates


@pytest.mark.parametrize("slope", [0.002 * 1.12 ** i for i in (1, 5, 7, 12, 14)])
@pytest.mark.parametrize("V", [1 << 20, (1 << 24) - 5])
def test_sums_of_long_rising_rows(sv, V, slope):
    # every item's maximum is above the one before: a sum that is rescaled at
    # each of them gathers their exponentials' errors
    x = (torch.arange(-(-V // 4) * 4) // 1024).double().mul_(slope / 32).float()
    s, p, t, _ = sv.spec_beam_select(x.view(1, 1, -1).cuda(), torch.zeros((1, 1), device="cuda"), V, 2)
    y = x[:V].double()
    best = y.max() - y.logsumexp(0)
    first = int((x[:V] == x[V - 1]).nonzero()[0])
    assert t.tolist() == [[first, first + 1]]
    assert np.all(np.abs(s.cpu().double().numpy() - float(best)) <= 6e-6 + 2.0 ** -24 * abs(float(best)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, W, K, V", [(149, 3, 5, 700), (300, 2, 4, 2100), (700, 1, 2, 90)])
def test_more_requests_than_start_together(sv, dtype, B, W, K, V):
    # requests whose blocks start after pass 1 has ended, ended and unused beams
    # and bad requests among them
    x, s = rows(B + V, B, W, V, dtype)
    fin = torch.zeros((B, W), dtype=torch.int32)
    fin[1::3, 0] = 1
    s[::7, W - 1] = -float("inf")
    x[147::10, 0, V - 1] = float("nan")
    s[B - 2, 0] = float("nan")
    _, p, _ = check(sv, x, s, V, K, 0.8, fin, 3)
    assert np.all(p[B - 2] == -1) and np.any(p[148:] >= 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_the_workspace_held_changes_nothing(sv, dtype):
    x, s = rows(23, 5, 4, 9001, dtype)
    x, s = x.cuda(), s.cuda()
    want = sv.spec_beam_select(x, s, 9001, 6)
    need = sv.load_library().spec_beam_workspace_size(5, 4, 9001)
    for fill in (0, 63, 127, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got = sv.spec_beam_select(x, s, 9001, 6, workspace_buf=ws)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
