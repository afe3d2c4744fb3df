"""Host checks of the beam, path and cache calls, made before anything
touches the device, and the plain implementations on hand-worked cases."""
import ctypes

import numpy as np
import pytest

import state_ref as ref

OK, EINVAL, EALIGN, EUNSUPPORTED, EWORKSPACE = 0, -1, -2, -3, -5
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_87_b200 import binding, build
    build.build()
    return binding.load_library()


def _select(lib, **kw):
    a = dict(logits=0x1000, dtype=1, stride=128, scores=0x2000, finished=0, end=-1, batch=2, beams=4,
             vocab=100, t=1.0, keep=4, out=0x3000, ws=0x10000, ws_bytes=1 << 30)
    a.update(kw)
    return lib.spec_beam_select(P(a["logits"]), a["dtype"], a["stride"], P(a["scores"]), P(a["finished"]),
                                a["end"], a["batch"], a["beams"], a["vocab"], a["t"], a["keep"], P(a["out"]),
                                P(0x4000), P(0x5000), None, None, P(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("want, change", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(beams=0)), (EINVAL, dict(keep=0)),
    (EUNSUPPORTED, dict(beams=65)), (EUNSUPPORTED, dict(keep=65)),
    (EINVAL, dict(t=0.0)), (EINVAL, dict(t=float("inf"))), (EINVAL, dict(t=float("nan"))), (EINVAL, dict(t=1e-40)),
    (EINVAL, dict(dtype=2)), (EINVAL, dict(vocab=0)), (EINVAL, dict(vocab=129)),
    (EINVAL, dict(end=100)), (EINVAL, dict(end=-2)), (EINVAL, dict(finished=0x6000)),
    (EALIGN, dict(stride=100)), (EALIGN, dict(logits=0x1008)),
    (EINVAL, dict(logits=0)), (EINVAL, dict(scores=0)), (EINVAL, dict(out=0)),
    (EWORKSPACE, dict(ws=0)), (EWORKSPACE, dict(ws=0x10010)), (EWORKSPACE, dict(ws_bytes=256)),
    (EUNSUPPORTED, dict(batch=1 << 30, beams=64, ws_bytes=1 << 62)),
    (OK, dict(batch=0)), (OK, dict(batch=0, logits=0, scores=0, out=0, ws=0)),
])
def test_select_refusals(lib, want, change):
    assert _select(lib, **change) == want


def _beams(lib, **kw):
    a = dict(states=(0x1000, 0x2000), n=2, request=4096, beam=1024, segments=2, segment=512, unit=16, cap=32,
             parents=0x9000, batch=2, beams=4, width=4)
    a.update(kw)
    st = None if a["states"] is None else (P * len(a["states"]))(*a["states"])
    return lib.spec_reorder_beams(st, a["n"], a["request"], a["beam"], a["segments"], a["segment"], a["unit"],
                                  a["cap"], None, None, P(a["parents"]), a["batch"], a["beams"], a["width"],
                                  None, None)


@pytest.mark.parametrize("want, change", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(beams=0)), (EINVAL, dict(width=0)), (EINVAL, dict(width=5)),
    (EUNSUPPORTED, dict(beams=65, request=1 << 20)), (EINVAL, dict(n=-1)), (EUNSUPPORTED, dict(n=129)),
    (EINVAL, dict(segments=0)), (EINVAL, dict(unit=0)), (EINVAL, dict(cap=0)),
    (EINVAL, dict(segment=511)), (EINVAL, dict(beam=1023)), (EINVAL, dict(request=4095)),
    (EINVAL, dict(request=-4096)), (EINVAL, dict(beam=-1024)), (EUNSUPPORTED, dict(request=1 << 60)),
    (EUNSUPPORTED, dict(beam=1 << 60)), (EUNSUPPORTED, dict(unit=1 << 40)),
    (EUNSUPPORTED, dict(unit=(1 << 31) - 1, cap=(1 << 31) - 1, segment=1 << 46, beam=1 << 46)),
    (EINVAL, dict(parents=0)), (EINVAL, dict(states=None)), (EINVAL, dict(states=(0x1000, 0))),
    (OK, dict(batch=0)), (OK, dict(n=0, states=None)),
])
def test_reorder_refusals(lib, want, change):
    assert _beams(lib, **change) == want


def test_a_state_that_comes_twice_is_refused(lib):
    assert _beams(lib, states=(0x1000, 0x2000, 0x1000), n=3) == EINVAL
    assert _path(lib, states=(0x1000, 0x1000), n=2) == EINVAL


def test_select_in_place_needs_as_many_kept_as_held(lib):
    assert _select(lib, keep=3, out=0x2000) == EINVAL
    assert _select(lib, keep=5, out=0x2000) == EINVAL
    # keep == beams gets past that check, to the workspace's
    assert _select(lib, keep=4, out=0x2000, ws=0) == EWORKSPACE


def _path(lib, **kw):
    a = dict(states=(0x1000, 0x2000), n=2, request=4096, segments=2, segment=512, unit=16, cap=32,
             base=0x8000, path=0x9000, batch=2, nodes=10, width=5, lens=0xa000)
    a.update(kw)
    st = None if a["states"] is None else (P * len(a["states"]))(*a["states"])
    return lib.spec_commit_path(st, a["n"], a["request"], a["segments"], a["segment"], a["unit"], a["cap"],
                                P(a["base"]), P(a["path"]), a["batch"], a["nodes"], a["width"], P(a["lens"]),
                                None, None)


@pytest.mark.parametrize("want, change", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(nodes=0)), (EINVAL, dict(width=0)),
    (EUNSUPPORTED, dict(nodes=1025)), (EUNSUPPORTED, dict(width=1025)),
    (EINVAL, dict(segment=511)), (EINVAL, dict(request=1023)), (EINVAL, dict(path=0)),
    (EINVAL, dict(lens=0x8000)), (EINVAL, dict(states=None)), (EINVAL, dict(states=(0, 0x1000))),
    (EUNSUPPORTED, dict(n=129)), (EUNSUPPORTED, dict(segments=1 << 20, request=1 << 40)),
    (OK, dict(batch=0)), (OK, dict(n=0, lens=0)),
])
def test_commit_refusals(lib, want, change):
    assert _path(lib, **change) == want


def _score(lib, **kw):
    a = dict(q=0x1000, k=0x2000, dtype=1, qr=1024, qt=512, qh=64, kr=4096, kh=1024, ks=64, begin=0x3000,
             end=0x4000, batch=2, queries=2, q_heads=8, kv_heads=4, dim=64, cap=16, scale=0.1, scores=0x5000,
             out=0x6000, ws=0x10000, ws_bytes=1 << 30)
    a.update(kw)
    return lib.spec_cache_score(P(a["q"]), P(a["k"]), a["dtype"], a["qr"], a["qt"], a["qh"], a["kr"], a["kh"],
                                a["ks"], P(a["begin"]), P(a["end"]), a["batch"], a["queries"], a["q_heads"],
                                a["kv_heads"], a["dim"], a["cap"], a["scale"], P(a["scores"]), P(a["out"]),
                                None, P(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("want, change", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(queries=0)), (EINVAL, dict(kv_heads=0)), (EINVAL, dict(q_heads=6)),
    (EINVAL, dict(q_heads=2)), (EINVAL, dict(dim=0)), (EINVAL, dict(cap=0)), (EINVAL, dict(dtype=3)),
    (EINVAL, dict(scale=float("nan"))), (EINVAL, dict(scale=float("inf"))),
    (EALIGN, dict(dim=60)), (EALIGN, dict(qt=511)), (EALIGN, dict(ks=63)), (EALIGN, dict(k=0x2002)),
    (EUNSUPPORTED, dict(dim=264)), (EUNSUPPORTED, dict(dtype=0, dim=4)), (EUNSUPPORTED, dict(queries=40000)),
    (EUNSUPPORTED, dict(batch=70000)), (EUNSUPPORTED, dict(kr=1 << 50)), (EINVAL, dict(kr=-64)),
    (EINVAL, dict(q=0)), (EINVAL, dict(k=0)), (EINVAL, dict(begin=0)), (EINVAL, dict(end=0)),
    (EINVAL, dict(scores=0)), (EINVAL, dict(out=0)),
    (EWORKSPACE, dict(ws=0)), (EWORKSPACE, dict(ws=0x10008)), (EWORKSPACE, dict(ws_bytes=16)),
    (OK, dict(batch=0)),
])
def test_score_refusals(lib, want, change):
    assert _score(lib, **change) == want


@pytest.mark.parametrize("want, scale", [
    (EINVAL, 3e38), (EINVAL, -3e38),   # finite, but not in units of log2
    (OK, 2e38),
])
def test_score_scales_within_fp32(lib, want, scale):
    assert _score(lib, scale=scale, batch=0) == want


@pytest.mark.parametrize("want, cap", [(EUNSUPPORTED, (1 << 30) + 1), (OK, 1 << 30)])
def test_score_capacity_limit(lib, want, cap):
    assert _score(lib, cap=cap, batch=0) == want


def _evict(lib, **kw):
    a = dict(k=0x1000, v=0x2000, kr=8192, kh=2048, ks=128, kb=128, vr=8192, vh=2048, vs=128, vb=128,
             scores=0x3000, positions=0x4000, lens=0x5000, batch=2, heads=4, cap=16, budget=8, sinks=2, recent=4,
             out=0x6000, ws=0x10000, ws_bytes=1 << 30)
    a.update(kw)
    return lib.spec_cache_evict(P(a["k"]), P(a["v"]), a["kr"], a["kh"], a["ks"], a["kb"], a["vr"], a["vh"],
                                a["vs"], a["vb"], P(a["scores"]), P(a["positions"]), P(a["lens"]), a["batch"],
                                a["heads"], a["cap"], a["budget"], a["sinks"], a["recent"], P(a["out"]),
                                P(0x7000), P(0x8000), None, P(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("want, change", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(heads=0)), (EINVAL, dict(cap=0)), (EINVAL, dict(budget=0)),
    (EINVAL, dict(sinks=-1)), (EINVAL, dict(recent=-1)), (EINVAL, dict(sinks=5)),
    (EINVAL, dict(kb=0)), (EINVAL, dict(ks=127)), (EINVAL, dict(vs=127)), (EINVAL, dict(vb=0)),
    (EINVAL, dict(kr=-1)), (EUNSUPPORTED, dict(vr=1 << 50)), (EUNSUPPORTED, dict(cap=262145)),
    (EUNSUPPORTED, dict(batch=1 << 30)),
    (EINVAL, dict(k=0)), (EINVAL, dict(scores=0)), (EINVAL, dict(positions=0)), (EINVAL, dict(lens=0)),
    (EINVAL, dict(out=0)), (EWORKSPACE, dict(ws=0)), (EWORKSPACE, dict(ws=0x10080)),
    (EWORKSPACE, dict(ws_bytes=16)), (OK, dict(batch=0)),
])
def test_evict_refusals(lib, want, change):
    assert _evict(lib, **change) == want


def test_workspace_sizes(lib):
    assert lib.spec_beam_workspace_size(4, 8, 128256) >= 4 * 8 * 126 * 8
    assert lib.spec_beam_workspace_size(4, 65, 100) == 0 and lib.spec_beam_workspace_size(4, 0, 100) == 0
    assert lib.spec_beam_workspace_size(0, 8, 100) > 0 and lib.spec_beam_workspace_size(-1, 8, 100) == 0
    assert lib.spec_score_workspace_size(2, 3, 8, 4, 1000) > 0
    assert lib.spec_score_workspace_size(2, 3, 6, 4, 1000) == 0
    assert lib.spec_evict_workspace_size(2, 4, 1000, 900) >= 2 * 4 * 100 * 8
    assert lib.spec_evict_workspace_size(2, 4, 1000, 1000) > 0 and lib.spec_evict_workspace_size(2, 4, 0, 1) == 0


def test_binding_refuses_host_tensors():
    import torch
    from speculative_decoding_verification_87_b200 import binding as sv
    x = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError):
        sv.spec_beam_select(x, torch.zeros(1, 2), 8, 2)
    with pytest.raises(ValueError):
        sv.spec_reorder_beams([x], torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.spec_commit_path([x], None, torch.zeros(1, 2, dtype=torch.int32), 2, 1)
    k = torch.zeros(1, 1, 4, 8)
    with pytest.raises(ValueError):
        sv.spec_cache_score(k, k, x, x, x)
    with pytest.raises(ValueError):
        sv.spec_cache_evict(k, k, x, x, x, 2)


# ------------------------------------------------------- the plain implementations, by hand
def test_reference_select_by_hand():
    # two beams over three tokens: probabilities 1/2, 1/4, 1/4 and 1/4, 1/2, 1/4
    x = np.log(np.array([[[2.0, 1.0, 1.0], [1.0, 2.0, 1.0]]]))
    s, p, t, f, bad = ref.beam_select(x, np.array([[0.0, np.log(0.5)]]), 3, 5, end_token=1,
                                      finished=np.zeros((1, 2), int))
    # sums: 1/2 1/4 1/4 | 1/8 1/4 1/8 -> ties to the lower beam, then token
    assert p.tolist() == [[0, 0, 0, 1, 1]] and t.tolist() == [[0, 1, 2, 1, 0]]
    assert np.allclose(np.exp(s), [[0.5, 0.25, 0.25, 0.25, 0.125]]) and f.tolist() == [[0, 1, 0, 1, 0]]
    # an ended beam has one candidate, a beam at -inf none; what is left over is empty
    s, p, t, f, bad = ref.beam_select(x, np.array([[-np.inf, -1.0]]), 3, 2, end_token=2,
                                      finished=np.array([[0, 1]]))
    assert p.tolist() == [[1, -1]] and t.tolist() == [[2, -1]] and s.tolist() == [[-1.0, -np.inf]]


def test_reference_moves_by_hand():
    x = np.arange(8).reshape(1, 4, 2)
    assert ref.reorder_beams(x, np.array([[1, 0, 0, -1]])).tolist() == [[[2, 3], [0, 1], [0, 1], [6, 7]]]
    y = ref.reorder_beams(x, np.array([[3, 3]]), axis=2, begin=np.array([1]), end=np.array([2]))
    assert y.tolist() == [[[0, 7], [2, 7], [4, 5], [6, 7]]]
    z, n = ref.commit_path(np.arange(6).reshape(1, 6), np.array([1]), np.array([[0, 2, 4, -1]]), 1)
    assert z.tolist() == [[0, 1, 3, 5, 4, 5]] and n.tolist() == [4]


def test_reference_weights_by_hand():
    # equal keys: a query spreads its weight evenly over the slots it sees
    q, k = np.ones((1, 2, 2, 8)), np.ones((1, 1, 5, 8))
    out, _ = ref.cache_score(q, k, np.array([2]), np.array([4]), np.full((1, 1, 5), 0.5), 1.0, 2.0 ** -24)
    third, fourth = 2 / 3, 2 / 4
    assert np.allclose(out, [[[0.5 + third + fourth, 0.5 + third + fourth, third + fourth, fourth, 0.5]]])


def test_reference_evict_by_hand():
    k = np.arange(6.0).reshape(1, 1, 6, 1)
    s = np.array([[[0.1, 5.0, 0.2, 3.0, 0.3, 0.0]]])
    p = np.arange(6)[None, None]
    # position 0 (sink) and 5 (newest) stay, then scores 5 and 3: slot 2 is given up for slot 5
    k2, _, s2, p2, n = ref.evict(k, k, s, p, np.array([6]), 4, 1, 1)
    assert k2[0, 0, :, 0].tolist() == [0, 1, 5, 3, 4, 5] and p2[0, 0, :4].tolist() == [0, 1, 5, 3] and n.tolist() == [4]


@pytest.mark.parametrize("want, change", [
    (EINVAL, dict(kh=0)), (EINVAL, dict(kr=0)), (EINVAL, dict(vh=0)), (EINVAL, dict(vr=0)),       # expanded heads, requests
    (EINVAL, dict(kh=2047)), (EINVAL, dict(kr=8191)), (EINVAL, dict(kh=1 << 42, kr=1 << 42)),
    (OK, dict(kh=128, ks=512)), (OK, dict(kr=128, kh=256, ks=1024)), (OK, dict(vh=0, heads=1)), (OK, dict(v=0, vh=0)),
])
def test_evict_rows_that_overlap_are_refused(lib, want, change):
    # what gets past the check stops at the workspace's
    assert _evict(lib, ws=0, **change) == (EWORKSPACE if want == OK else want)


def test_score_workspace_of_a_type_and_head_dimension(lib):
    size, f32, bf16 = lib.spec_score_workspace_size_for, 0, 1
    # 32 rows of 64 elements are swept twice: their products are not stored
    assert 0 < size(bf16, 64, 32, 8, 32, 8, 32768) < 1 << 20
    # where they are, in groups of heads that fit 256 MiB (and the chunks' statistics)
    most = (256 << 20) + (8 << 20)
    assert 256 * 4 * 32768 * 4 <= size(bf16, 128, 32, 1, 32, 8, 32768) <= most
    assert size(bf16, 128, 32, 8, 32, 8, 32768) <= most and size(bf16, 128, 64, 4, 32, 8, 1 << 20) <= most
    # a head that does not fit by itself is swept
    assert size(bf16, 128, 1, 32, 1, 1, 1 << 30) < 1 << 20
    # what is enough for any of them
    for args in ((1, 2, 2, 1, 100), (32, 8, 32, 8, 32768), (4, 1, 32, 8, 9000), (2, 40, 8, 2, 500), (1, 3, 1, 1, 64)):
        each = [size(t, d, *args) for t in (f32, bf16) for d in range(8, 257, 8)]
        assert lib.spec_score_workspace_size(*args) == max(each) and min(each) > 0
    assert size(2, 64, 1, 1, 1, 1, 10) == 0 and size(bf16, 0, 1, 1, 1, 1, 10) == 0 and size(bf16, 64, 1, 1, 3, 2, 10) == 0
    assert size(bf16, 64, 0, 1, 1, 1, 10) > 0
