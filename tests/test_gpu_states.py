"""spec_reorder_beams and spec_commit_path: bytes, so every comparison is exact."""
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


def state(seed, shape, dtype=torch.int16, offset=0):
    """A CUDA tensor of `shape` that starts `offset` elements into its storage, and its values."""
    n = int(np.prod(shape))
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-100, 100, (n,), generator=g).to(dtype)
    store = torch.zeros(n + offset, dtype=dtype, device="cuda")
    store[offset:] = x.cuda()
    return store[offset:].reshape(shape), x.reshape(shape).numpy()


def ints(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype, offset", [(torch.int64, 0), (torch.float32, 0), (torch.int16, 0), (torch.int16, 1),
                                           (torch.int16, 2), (torch.int16, 4), (torch.int8, 3)])
@pytest.mark.parametrize("shape, axis", [((2, 4, 3, 50, 16), 3), ((2, 4, 50, 3, 16), 2), ((1, 7, 2, 9, 5), 3),
                                         ((3, 2, 33), 2), ((3, 2, 33), None), ((2, 5), None), ((2, 64, 3, 8), None),
                                         ((1, 33, 2, 300, 8), 3)])
def test_reorder(sv, dtype, offset, shape, axis):
    B, W = shape[:2]
    r = np.random.RandomState(B * 10 + W)
    par = r.randint(-1, W, (B, W)).astype(np.int32)
    xs, vs = zip(*(state(i, shape, dtype, offset) for i in range(3)))
    begin = end = None
    if axis is not None:
        begin = r.randint(0, shape[axis] + 1, B).astype(np.int32)
        end = np.array([r.randint(b, shape[axis] + 1) for b in begin], np.int32)
    status = ints([0])
    got = sv.spec_reorder_beams(list(xs), ints(par), axis, None if axis is None else ints(begin),
                                None if axis is None else ints(end), status)
    for x, v in zip(got, vs):
        assert np.array_equal(x.cpu().numpy(), ref.reorder_beams(v, par, axis, begin, end))
    assert status.item() == 0


@pytest.mark.parametrize("par", [[0, 1, 2, 3], [3, 0, 1, 2], [1, 0, 3, 2], [2, 2, 2, 2], [-1, -1, -1, -1], [0, 0, 0, 0],
                                 [1, 2, 3, 3], [3, 3, 0, -1]])
def test_reorder_shapes_of_parents(sv, par):
    x, v = state(1, (1, 4, 2, 77, 24))
    sv.spec_reorder_beams([x], ints([par]), 3)
    assert np.array_equal(x.cpu().numpy(), ref.reorder_beams(v, np.array([par])))


def test_reorder_fewer_children_than_beams_and_no_window(sv):
    x, v = state(1, (2, 6, 40, 8))
    par = np.array([[5, 4, 3], [1, 1, 1]])
    sv.spec_reorder_beams([x], ints(par), 2)
    assert np.array_equal(x.cpu().numpy(), ref.reorder_beams(v, par))
    # only one of begin and end; an empty window
    x, v = state(2, (2, 6, 40, 8))
    sv.spec_reorder_beams([x], ints(par), 2, begin=ints([3, 40]))
    v = ref.reorder_beams(v, par, 2, np.array([3, 40]), None)
    sv.spec_reorder_beams([x], ints(par), 2, end=ints([0, 7]))
    assert np.array_equal(x.cpu().numpy(), ref.reorder_beams(v, par, 2, None, np.array([0, 7])))


def test_reorder_leaves_bad_requests(sv):
    x, v = state(4, (5, 3, 20, 8))
    par = np.array([[1, 2, 0], [3, 0, 0], [0, -2, 1], [1, 1, 1], [2, 2, 2]])
    begin, end = np.array([2, 0, 0, 5, -1]), np.array([21, 20, 20, 4, 9])
    status = ints([0])
    sv.spec_reorder_beams([x], ints(par), 2, ints(begin), ints(end), status)
    assert np.array_equal(x.cpu().numpy(), v) and status.item() == 2 | 16
    status.zero_()
    begin, end = np.array([2, 0, 0, 4, 0]), np.array([20, 20, 20, 4, 9])
    sv.spec_reorder_beams([x], ints(par), 2, ints(begin), ints(end), status)
    par[1:3] = -1
    assert np.array_equal(x.cpu().numpy(), ref.reorder_beams(v, par, 2, begin, end)) and status.item() == 2


def test_reorder_strided_views(sv):
    # one layer of a [layers][B][W][H][T][D] cache, and every second request
    full, v = state(6, (2, 4, 3, 2, 15, 8))
    par = np.array([[2, 0, 1], [1, 1, 2]])
    sv.spec_reorder_beams([full[1, ::2], full[0, 1::2]], ints(par), 3)
    w = v.copy()
    w[1, ::2] = ref.reorder_beams(v[1, ::2], par)
    w[0, 1::2] = ref.reorder_beams(v[0, 1::2], par)
    assert np.array_equal(full.cpu().numpy(), w)
    with pytest.raises(ValueError):
        sv.spec_reorder_beams([full[0].transpose(3, 4)], ints(np.zeros((4, 3))), 3)
    with pytest.raises(ValueError):
        sv.spec_reorder_beams([full[0], full[1, :, :, :, :14]], ints(np.zeros((4, 3))), 3)
    with pytest.raises(ValueError):
        sv.spec_reorder_beams([full[0]], ints(np.zeros((3, 3))), 3)


@pytest.mark.parametrize("dtype, offset", [(torch.int64, 0), (torch.float32, 0), (torch.int16, 0), (torch.int16, 1), (torch.int8, 3)])
@pytest.mark.parametrize("shape, axis, nodes, depth", [((3, 2, 60, 16), 2, 21, 4), ((3, 60, 2, 16), 1, 21, 4),
                                                       ((2, 300, 9), 1, 200, 60), ((4, 70), 1, 60, 6),
                                                       ((1, 5, 33, 40), 2, 1, 1)])
def test_commit(sv, dtype, offset, shape, axis, nodes, depth):
    B = shape[0]
    r = np.random.RandomState(nodes + depth)
    path = np.full((B, depth + 1), -1, np.int32)
    for b in range(B):
        n = r.randint(0, min(depth + 1, nodes) + 1) if b else min(depth + 1, nodes)
        path[b, :n] = np.sort(r.permutation(nodes)[:n])
    base = r.randint(0, shape[axis] - nodes + 1, B).astype(np.int32)
    xs, vs = zip(*(state(i, shape, dtype, offset) for i in range(2)))
    status = ints([0])
    lens = sv.spec_commit_path(list(xs), ints(base), ints(path), nodes, axis, status=status)
    for x, v in zip(xs, vs):
        w, n = ref.commit_path(v, base, path, axis)
        assert np.array_equal(x.cpu().numpy(), w)
        assert np.array_equal(lens.cpu().numpy(), n)
    assert status.item() == 0


def test_commit_leaves_bad_requests(sv):
    x, v = state(3, (7, 2, 30, 8))
    path = np.array([[0, 2, 5, -1], [0, 2, 2, -1], [0, 3, 10, -1], [2, 1, -1, -1], [0, 2, 4, 6], [0, 2, 4, 6], [0, -1, -2, -1]])
    base = np.array([20, 0, 0, 0, 21, -1, 0])
    status = ints([0])
    lens = sv.spec_commit_path([x], ints(base), ints(path), 10, 2, status=status)
    w = v.copy()
    w[:1] = ref.commit_path(v[:1], base[:1], path[:1], 2)[0]
    assert np.array_equal(x.cpu().numpy(), w) and status.item() == 2 | 16
    assert lens.cpu().tolist() == [23, 0, 0, 0, 21, -1, 0]


def test_commit_of_lengths_alone_and_without_base(sv):
    lens = sv.spec_commit_path([], ints([4, 9]), ints([[0, 3, -1], [-1, -1, -1]]), 5, 1)
    assert lens.cpu().tolist() == [6, 9]
    x, v = state(3, (2, 12, 4, 8))           # the queries' rows of a tree
    path = np.array([[0, 1, 11], [0, 4, -1]])
    lens = sv.spec_commit_path([x], None, ints(path), 12, 1)
    assert np.array_equal(x.cpu().numpy(), ref.commit_path(v, np.zeros(2, int), path, 1)[0])
    assert lens.cpu().tolist() == [3, 2]
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_commit_path([x], lens, ints(path), 12, 1, out_lens=lens)


def test_many_states_and_a_graph(sv):
    xs, vs = zip(*(state(i, (2, 3, 11, 8)) for i in range(128)))
    par = ints([[1, 2, 0], [2, 2, -1]])
    begin, end = ints([0, 3]), ints([11, 9])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_reorder_beams(list(xs), par, 2, begin, end)
    for x, v in zip(xs, vs):
        x.copy_(torch.from_numpy(v))
    graph.replay()
    graph.replay()
    for x, v in zip(xs, vs):
        for _ in range(2):
            v = ref.reorder_beams(v, par.cpu().numpy(), 2, begin.cpu().numpy(), end.cpu().numpy())
        assert np.array_equal(x.cpu().numpy(), v)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_reorder_beams(list(xs) + [xs[0]], par, 2)
