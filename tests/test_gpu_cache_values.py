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
