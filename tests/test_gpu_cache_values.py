"""spec_cache_score at values that need care: large products, infinities,
values next to the type's limits, and its accuracy against emulations of what
it would be with less."""
import numpy as np
import pytest
import torch

from test_gpu_cache import UNIT, ints, make


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from speculative_decoding_verification_87_b200 import binding, build
    build.build()
    binding.load_library()
    return binding


# ------------------------------------------------------------- large products
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Q, G", [(1, 4), (6, 4), (23, 3)])
@pytest.mark.parametrize("a", [100.0, 113.5, 123.0, 131.0, 149.0, 167.0, -100.0, -131.0])
def test_equal_products_share_evenly(sv, dtype, Q, G, a):
    # All products of a query are the number a (exact in bf16), however large: a
    # query that sees n slots gives each 1/n.  The exponentials are 2^0 and
    # their sums whole numbers, so what rounds is the reciprocal (2^-23 where it
    # is approximate), its product with the exponential and the sum over the rows
    # (half a step each).
    n, D = 341, 64
    q, k = torch.zeros((1, Q, G, D), dtype=dtype), torch.zeros((1, 1, n, D), dtype=dtype)
    q[..., 3] = a
    k[..., 3] = 1.0
    out = sv.spec_cache_score(q.cuda(), k.cuda(), ints([n - Q]), ints([n]), torch.zeros((1, 1, n), device="cuda"), 1.0)
    want = np.zeros(n)
    for i in range(Q):
        want[:n - Q + i + 1] += G / (n - Q + i + 1)
    assert np.all(np.abs(out.cpu().numpy()[0, 0] - want) <= (Q * G + 4) * 2.0 ** -24 * want)


# ------------------------------------------------------------- infinities
def weights(q, k, begin, end, scores, scale):
    """state_ref.cache_score for products that may be -inf: such a slot weighs
    nothing, and a query with no other product adds nothing.  NaN and +inf: NaN."""
    B, H, C, D = k.shape
    G = q.shape[2] // H
    out, bound = scores.copy(), np.zeros_like(scores)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(B):
            b0, b1 = int(begin[b]), int(end[b])
            out[b, :, b0:b1] = 0.0
            for h in range(H):
                for i in range(b1 - b0):
                    n = b0 + i + 1
                    for g in range(G):
                        row, kk = q[b, i, h * G + g], k[b, h, :n]
                        s = scale * (kk @ row)
                        e = (D + 8) * UNIT * abs(scale) * (np.abs(kk) @ np.abs(row))
                        m = s.max()
                        if np.isnan(m) or m == np.inf:
                            out[b, h, :n] = np.nan
                            continue
                        w = np.exp(s - m) if m > -np.inf else np.zeros(n)
                        w /= max(w.sum(), 1e-300)
                        out[b, h, :n] += w
                        near = s > m - 200  # the others weigh less than 1e-80, whatever their products' rounding
                        bound[b, h, :n] += w * np.expm1(2 * e[near].max(initial=0.0) + 2.0 ** -18)
            bound[b, :, :b1] += ((b1 - b0) * G + 2) * 2.0 ** -24 * np.abs(np.nan_to_num(out[b, :, :b1])) + 1e-37
    return out, bound


def against_weights(sv, q, k, begin, end, scores, scale):
    got = sv.spec_cache_score(q.cuda(), k.cuda(), ints(begin), ints(end), scores.cuda(), scale).cpu().numpy()
    want, bound = weights(q.double().numpy(), k.double().numpy(), begin, end, scores.double().numpy(), scale)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    real = ~np.isnan(want)
    assert np.all(np.abs(got - want)[real] <= bound[real])
    return got


# rows of a key head: 4 and 16 (the stored form for bf16 and fp32), 18 and 72 (the sweeps, with rows left over in a tile of 16), 64
SHAPES = [(1, 4), (4, 4), (9, 2), (9, 8), (16, 4), (33, 5)]
INF = float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Q, G", SHAPES)
def test_products_of_minus_infinity_weigh_nothing(sv, dtype, Q, G):
    q, k, s = make(Q + G, 3, Q, G, 2, 64, 150, dtype)
    q[..., 7] = q[..., 7].abs() + 0.25
    k[0, :, 20:90:3, 7] = -INF          # some slots
    k[1, 0, :, 7] = -INF                # every slot of a head: its queries add nothing
    k[1, 1, 64:, 7] = -INF              # the last tiles of a head
    k[2, 0, :60, 7] = -INF              # the first ones, and the step's own slots
    k[2, 1, 150 - Q:, 7] = -INF
    begin, end = [150 - Q, 149 - Q, 150 - Q], [150, 149, 150]
    got = against_weights(sv, q, k, begin, end, s, 0.125)
    assert np.all(got[0, :, 20:90:3] == s.numpy()[0, :, 20:90:3])
    assert np.array_equal(got[1, 0, :149 - Q], s.numpy()[1, 0, :149 - Q]) and np.all(got[1, 0, 149 - Q:149] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Q, G", SHAPES)
def test_values_next_to_the_limits(sv, dtype, Q, G):
    # the type's largest and lowest values as keys or queries, where their
    # products are ordinary numbers, nothing, or past the range
    low = torch.finfo(dtype).min
    q, k, s = make(Q * G, 4, Q, G, 2, 64, 130, dtype)
    q[:, :, :, 5] = 0.0
    k[0, :, ::2, 5] = low               # times zero
    k[0, :, 1::2, 5] = -low
    q[1, :, :, 5] = 2.0 ** -125         # products of 8
    k[1, 0, ::3, 5] = low
    k[1, 1, 40:, 5] = -low
    q[2, :, :, 5] = 1.0                 # a cache masked through its keys
    k[2, 0, ::3, 5] = low
    k[2, 0, 77, 5] = low
    k[2, 1, :100, 5] = low
    q[3, :, 0, 9] = -low                # and large queries
    k[3, :, :, 9] = 2.0 ** -126
    begin, end = [130 - Q] * 4, [130] * 4
    against_weights(sv, q, k, begin, end, s, 0.125)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Q, G", SHAPES)
def test_infinite_products(sv, dtype, Q, G):
    # +inf and 0 * inf give NaN to the slots that the query sees, -inf none
    q, k, s = make(Q * G, 3, Q, G, 2, 64, 130, dtype)
    q[..., 4] = q[..., 4].abs() + 0.25
    q[1, Q - 1, 0, 4] *= -1             # head 0: the last query's products are +inf
    k[:2, :, 50, 4] = -INF
    q[2, 0, 2 * G - 1, 4] = 0.0         # head 1: 0 * inf in the first query
    k[2, 1, 129 - Q, 4] = INF
    q[2, :, :G, 4] = -INF               # head 0: the queries' own infinities
    k[2, 0, :, 4] = k[2, 0, :, 4].abs() + 0.25
    begin, end = [130 - Q] * 3, [130] * 3
    got = against_weights(sv, q, k, begin, end, s, 0.125)
    assert np.isfinite(got[0]).all() and np.isnan(got[1, 0]).all() and np.isfinite(got[1, 1]).all()


# ------------------------------------------------------------- accuracy
def parts(x, count):
    """x as a sum of bf16 numbers, the remainder of each rounded in turn."""
    out, rest = [], x.clone()
    for _ in range(count):
        p = rest.to(torch.bfloat16).float()
        out.append(p.double())
        rest = rest - p
    return out


SIX = ((2, 0), (1, 1), (0, 2), (1, 0), (0, 1), (0, 0))


def products(q, k, pairs, step=None):
    """Products of fp32 rows by parts, in 64 bits; with `step`, summed up `step`
    elements of a pair at a time in a 24-bit accumulator that truncates."""
    p, r = parts(q, 3), parts(k, 3)
    if step is None:
        return sum(p[a] @ r[b].T for a, b in pairs)
    acc = torch.zeros((q.shape[0], k.shape[0]), dtype=torch.float64)
    for d in range(0, q.shape[1], step):
        for a, b in pairs:
            acc += p[a][:, d:d + step] @ r[b][:, d:d + step].T
            m, e = torch.frexp(acc)
            acc = torch.ldexp(torch.trunc(m * 2.0 ** 24) * 2.0 ** -24, e)
    return acc


def summed(s):
    return s.softmax(1).sum(0)


def error(x, exact):
    return float((x - exact).norm() / exact.norm())


# (D, rows, slots, scale): one query of all rows, so that every row sees every slot
F32_CASES = [(64, 8, 3000, 0.125), (64, 32, 700, 1.0), (64, 40, 700, 1.0), (32, 12, 2000, 0.25)]


def f32_case(D, R, n, scale):
    g = torch.Generator().manual_seed(D + R)
    q, k = torch.randn((R, D), generator=g), torch.randn((n, D), generator=g)
    exact = summed(q.double() @ k.double().T * scale)
    # half of what two parts a number (four products) are off
    limit = 0.5 * error(summed(products(q, k, SIX[1:2] + SIX[3:]) * scale), exact)
    return q, k, exact, limit


@pytest.mark.parametrize("D, R, n, scale", F32_CASES)
def test_the_f32_limit_tells_the_forms_apart(D, R, n, scale):
    # six products stay within it even in an accumulator that truncates; the three
    # largest alone do not
    q, k, exact, limit = f32_case(D, R, n, scale)
    assert error(summed(products(q, k, SIX, 16) * scale), exact) < limit
    assert error(summed(products(q, k, SIX[3:]) * scale), exact) > 2 * limit


@pytest.mark.gpu
@pytest.mark.parametrize("D, R, n, scale", F32_CASES)
def test_f32_accuracy(sv, D, R, n, scale):
    q, k, exact, limit = f32_case(D, R, n, scale)
    out = sv.spec_cache_score(q.view(1, 1, R, D).cuda(), k.view(1, 1, n, D).cuda(), ints([n - 1]), ints([n]),
                              torch.zeros((1, 1, n), device="cuda"), scale)
    assert error(out.cpu().double()[0, 0], exact) <= limit


def peaked(R, n):
    """bf16 keys that lean on the first query, as real ones do: a few slots carry the weight."""
    g = torch.Generator().manual_seed(R)
    q = torch.randn((R, 128), generator=g).to(torch.bfloat16)
    k = torch.randn((n, 128), generator=g) + 0.5 * torch.randn((n, 1), generator=g) * q[:1].float()
    k = k.to(torch.bfloat16)
    return q, k, summed(q.double() @ k.double().T * 128 ** -0.5)


# Products of 128 bf16 terms that are summed 16 at a time with truncation come
# out 4e-7 off (below), the exponentials (2^-22 each, of changing sign) 1e-7;
# accumulators that keep fewer bits of each step were 6e-6 off.
PEAKED_LIMIT = 1e-6


@pytest.mark.parametrize("R, n", [(8, 4000), (128, 4000)])
def test_the_peaked_limit(R, n):
    q, k, exact = peaked(R, n)
    s = products(q.float(), k.float(), SIX[5:], 16) * 128 ** -0.5
    assert error(summed(s), exact) < 0.5 * PEAKED_LIMIT


@pytest.mark.gpu
@pytest.mark.parametrize("R, n", [(8, 4000), (128, 4000)])
def test_peaked_accuracy(sv, R, n):
    q, k, exact = peaked(R, n)
    out = sv.spec_cache_score(q.view(1, 1, R, 128).cuda(), k.view(1, 1, n, 128).cuda(), ints([n - 1]), ints([n]),
                              torch.zeros((1, 1, n), device="cuda"))
    assert error(out.cpu().double()[0, 0], exact) <= PEAKED_LIMIT


# ------------------------------------------------------------- workspaces
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Q, G", SHAPES + [(8, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_workspace_of_the_form_is_enough(sv, dtype, Q, G, D):
    q, k, s = make(3 * Q + G, 2, Q, G, 2, D, 300, dtype)
    begin, end = ints([300 - Q, 250 - Q]), ints([300, 250])
    need = sv.load_library().spec_score_workspace_size_for(int(dtype == torch.bfloat16), D, 2, Q, 2 * G, 2, 300)
    want = sv.spec_cache_score(q.cuda(), k.cuda(), begin, end, s.cuda())
    store = torch.full((need + 1024,), 171, dtype=torch.uint8, device="cuda")
    got = sv.spec_cache_score(q.cuda(), k.cuda(), begin, end, s.cuda(), workspace_buf=store[:need])
    assert torch.equal(got, want) and torch.all(store[need:] == 171)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_cache_score(q.cuda(), k.cuda(), begin, end, s.cuda(), workspace_buf=store[:need - 1])


@pytest.mark.gpu
def test_heads_in_groups(sv):
    # 32 rows of 65536 slots are 8 MiB of products a head: 40 heads go 32 and 8 at
    # a time, a request's heads on both sides
    B, H, C, R, D = 8, 5, 65536, 32, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((B, 1, H * R, D), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((B, H, C, D), generator=g, device="cuda").to(torch.bfloat16)
    s = torch.rand((B, H, C), generator=g, device="cuda")
    end = torch.tensor([C - 4099 * b for b in range(B)], dtype=torch.int32)
    end[4] = C + 1                      # a request that is left as it was
    status = ints([0])
    out = sv.spec_cache_score(q, k, end.cuda() - 1, end.cuda(), s, out_scores=torch.full_like(s, -7.0), status=status)
    assert status.item() == 16 and torch.all(out[4] == -7.0)
    scale = D ** -0.5
    for b in range(B):
        n = int(end[b])
        if n > C:
            continue
        assert torch.all(out[b, :, n:] == -7.0)
        for h in range(H):
            x, y = q[b, 0, h * R:(h + 1) * R].double(), k[b, h, :n].double()
            w = (x @ y.T * scale).softmax(1)
            # as state_ref.cache_score bounds it
            e = (D + 8) * UNIT * scale * (x.abs() @ y.abs().T).amax(1, keepdim=True)
            want = s[b, h, :n].double()
            want[n - 1] = 0
            want = want + w.sum(0)
            bound = (w * torch.expm1(2 * e + 2.0 ** -18)).sum(0) + (R + 2) * 2.0 ** -24 * want
            assert torch.all((out[b, h, :n].double() - want).abs() <= bound)
