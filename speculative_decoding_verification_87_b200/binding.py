"""ctypes binding of libspecverify.so: argument marshalling only.

Each function takes torch CUDA tensors, checks their shapes and dtypes,
passes raw device pointers and the current CUDA stream to the C ABI of the
same name (declared in include/specverify.h) and returns the output
tensors.  Every step of the computation runs in the library's kernels; there
is no fallback.  If the library has not been built, the first call raises.

Build it with ``python -m speculative_decoding_verification_87_b200.build``.
"""
import array
import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SPEC_F32, SPEC_BF16 = 0, 1
SPEC_OK = 0
STATUS_TOKEN, STATUS_TREE, STATUS_LOGIT, STATUS_TIMEOUT, STATUS_CAPACITY = 1, 2, 4, 8, 16
MAX_K, MAX_NODES = 32, 1024
MAX_BEAMS, MAX_STATES, MAX_HEAD_DIM, MAX_SLOTS = 64, 128, 256, 262144
SYMBOLS = ("spec_verify_workspace_size", "spec_verify_strerror", "spec_verify_linear",
           "spec_verify_greedy", "spec_verify_tree", "spec_verify_debug_uniforms",
           "spec_verify_linear_noalloc", "spec_verify_debug_exp2", "spec_verify_greedy_walk",
           "spec_verify_tree_greedy_walk", "spec_verify_debug_wait_expiry", "spec_plug_tokens",
           "spec_shard_row_stats", "spec_shard_decide", "spec_shard_decide_greedy",
           "spec_shard_draw_sums", "spec_shard_draw_pick", "spec_shard_emit",
           "spec_beam_workspace_size", "spec_beam_select", "spec_reorder_beams",
           "spec_commit_path", "spec_score_workspace_size", "spec_score_workspace_size_for",
           "spec_cache_score", "spec_evict_workspace_size", "spec_cache_evict")
NOALLOC_SCRATCH_BYTES = 8 << 20

_lib = None
_lock = threading.Lock()
_ws_cache = {}

_P, _I, _I64, _U32, _U64, _F, _SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                     ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float,
                                     ctypes.c_size_t)


class SpecVerifyError(RuntimeError):
    pass


def load_library(path: str = LIB_PATH):
    """Load libspecverify.so and declare its C signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise SpecVerifyError(
                f"{path} is missing: build it with "
                "`python -m speculative_decoding_verification_87_b200.build`")
        L = ctypes.CDLL(path)
        L.spec_verify_workspace_size.argtypes = [_I, _I, _I]
        L.spec_verify_workspace_size.restype = _SZ
        L.spec_verify_strerror.argtypes = [_I]
        L.spec_verify_strerror.restype = ctypes.c_char_p
        L.spec_verify_linear.argtypes = [_P, _P, _I, _I64, _P, _I, _I, _I, _F, _U64, _U32, _P, _P,
                                         _P, _P, _P, _P, _SZ, _P]
        L.spec_verify_linear.restype = _I
        L.spec_verify_greedy.argtypes = [_P, _I, _I64, _P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]
        L.spec_verify_greedy.restype = _I
        L.spec_verify_tree.argtypes = [_P, _P, _I, _I64, _P, _P, _I, _I, _I, _I, _I, _F, _U64,
                                       _U32, _P, _P, _P, _P, _P, _SZ, _P]
        L.spec_verify_tree.restype = _I
        L.spec_verify_debug_uniforms.argtypes = [_U64, _U32, _U32, _I, _I, _I, _P, _P]
        L.spec_verify_debug_uniforms.restype = _I
        L.spec_verify_linear_noalloc.argtypes = [_P, _P, _I, _I64, _P, _I, _I, _I, _F, _U64, _U32,
                                                 _P, _P, _P, _P, _P, _P]
        L.spec_verify_linear_noalloc.restype = _I
        L.spec_verify_greedy_walk.argtypes = [_P, _I, _I64, _P, _I, _I, _I, _P, _P, _P, _P]
        L.spec_verify_greedy_walk.restype = _I
        L.spec_verify_tree_greedy_walk.argtypes = [_P, _I, _I64, _P, _P, _I, _I, _I, _I, _P, _P,
                                                   _P, _P, _P]
        L.spec_verify_tree_greedy_walk.restype = _I
        L.spec_verify_debug_exp2.argtypes = [_P, _P, _I, _I, _P]
        L.spec_verify_debug_exp2.restype = _I
        L.spec_verify_debug_wait_expiry.argtypes = [_P, _P, _I, _I64, _P, _I, _I, _I, _F, _U32,
                                                    _P, _P, _P, _P, _SZ, _P]
        L.spec_verify_debug_wait_expiry.restype = _I
        L.spec_plug_tokens.argtypes = [_P, _P, _P, _I, _I, _P, _P, _P, _I, _P, _P]
        L.spec_plug_tokens.restype = _I
        L.spec_shard_row_stats.argtypes = [_P, _P, _I, _I64, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P,
                                           _P]
        L.spec_shard_row_stats.restype = _I
        L.spec_shard_decide.argtypes = [_P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _U64, _U32, _P, _P,
                                        _P, _P, _P]
        L.spec_shard_decide.restype = _I
        L.spec_shard_decide_greedy.argtypes = [_P, _P, _I, _P, _I, _I, _I, _P, _P, _P, _P]
        L.spec_shard_decide_greedy.restype = _I
        L.spec_shard_draw_sums.argtypes = [_P, _P, _I, _I64, _I, _I, _I, _I, _F, _P, _P, _I, _P, _P]
        L.spec_shard_draw_sums.restype = _I
        L.spec_shard_draw_pick.argtypes = [_P, _P, _I, _I64, _I, _I, _I, _I, _F, _P, _P, _P, _I, _I,
                                           _P, _P]
        L.spec_shard_draw_pick.restype = _I
        L.spec_shard_emit.argtypes = [_P, _P, _I, _I, _P, _P]
        L.spec_shard_emit.restype = _I
        L.spec_beam_workspace_size.argtypes = [_I, _I, _I]
        L.spec_beam_workspace_size.restype = _SZ
        L.spec_beam_select.argtypes = [_P, _I, _I64, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P,
                                       _P, _P, _SZ, _P]
        L.spec_beam_select.restype = _I
        L.spec_reorder_beams.argtypes = [_P, _I, _I64, _I64, _I, _I64, _I64, _I, _P, _P, _P, _I, _I,
                                         _I, _P, _P]
        L.spec_reorder_beams.restype = _I
        L.spec_commit_path.argtypes = [_P, _I, _I64, _I, _I64, _I64, _I, _P, _P, _I, _I, _I, _P, _P,
                                       _P]
        L.spec_commit_path.restype = _I
        L.spec_score_workspace_size.argtypes = [_I, _I, _I, _I, _I]
        L.spec_score_workspace_size.restype = _SZ
        L.spec_score_workspace_size_for.argtypes = [_I, _I, _I, _I, _I, _I, _I]
        L.spec_score_workspace_size_for.restype = _SZ
        L.spec_cache_score.argtypes = [_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _I,
                                       _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _SZ, _P]
        L.spec_cache_score.restype = _I
        L.spec_evict_workspace_size.argtypes = [_I, _I, _I, _I]
        L.spec_evict_workspace_size.restype = _SZ
        L.spec_cache_evict.argtypes = [_P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P,
                                       _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]
        L.spec_cache_evict.restype = _I
        _lib = L
        return L


def _check(rc: int, what: str):
    if rc != SPEC_OK:
        msg = load_library().spec_verify_strerror(rc).decode()
        raise SpecVerifyError(f"{what} failed ({rc}): {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _need_cuda(name, t, dtype=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def workspace_size(batch: int, rows_per_req: int, vocab: int) -> int:
    return int(load_library().spec_verify_workspace_size(batch, rows_per_req, vocab))


def workspace(batch: int, rows_per_req: int, vocab: int, device=None) -> torch.Tensor:
    """A cached uint8 device buffer large enough for the call (256-byte aligned)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    need = workspace_size(batch, rows_per_req, vocab)
    if need == 0:
        raise ValueError("invalid workspace request")
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.empty(need + 256, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    off = (-buf.data_ptr()) % 256
    return buf[off:off + need]


def spec_verify_linear(target_logits, draft_logits, draft_tokens, vocab, temperature, seed=0,
                       offset=0, out_tokens=None, accepted_len=None, dbg_logp=None,
                       dbg_logq=None, status=None, workspace_buf=None, stream=None):
    """target_logits [B][k+1][stride], draft_logits [B][k][stride] (bf16/fp32),
    draft_tokens [B][k] int32.  Returns (out_tokens [B][k+1], accepted_len [B])."""
    _need_cuda("target_logits", target_logits)
    B, R, stride = target_logits.shape
    k = R - 1
    _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, stride))
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if accepted_len is None:
        accepted_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _need_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    for name, t in (("dbg_logp", dbg_logp), ("dbg_logq", dbg_logq)):
        if t is not None:
            _need_cuda(name, t, torch.float32, (B, k))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    if workspace_buf is None:
        workspace_buf = workspace(B, 2 * k + 1, vocab, dev) if B > 0 else None
    ws_bytes = 0 if workspace_buf is None else workspace_buf.numel()
    rc = load_library().spec_verify_linear(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), stride,
        _ptr(draft_tokens), B, k, vocab, float(temperature), int(seed), int(offset),
        _ptr(out_tokens), _ptr(accepted_len), _ptr(dbg_logp), _ptr(dbg_logq), _ptr(status),
        _ptr(workspace_buf), ws_bytes, _stream(stream))
    _check(rc, "spec_verify_linear")
    return out_tokens, accepted_len


def spec_verify_greedy(target_logits, draft_tokens, vocab, out_tokens=None, accepted_len=None,
                       status=None, workspace_buf=None, stream=None, workspace_free=False):
    """target_logits [B][k+1][stride], draft_tokens [B][k] int32.  By default
    the streamed form runs in a cached workspace (or workspace_buf);
    workspace_free=True runs the cluster form, which needs none."""
    _need_cuda("target_logits", target_logits)
    B, R, stride = target_logits.shape
    k = R - 1
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if accepted_len is None:
        accepted_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _need_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    if workspace_free:
        workspace_buf = None
    elif workspace_buf is None and B > 0:
        workspace_buf = workspace(B, k + 1, vocab, dev)
    ws_bytes = 0 if workspace_buf is None else workspace_buf.numel()
    rc = load_library().spec_verify_greedy(
        _ptr(target_logits), _dtype_code(target_logits), stride, _ptr(draft_tokens), B, k, vocab,
        _ptr(out_tokens), _ptr(accepted_len), _ptr(status), _ptr(workspace_buf), ws_bytes,
        _stream(stream))
    _check(rc, "spec_verify_greedy")
    return out_tokens, accepted_len


def spec_verify_greedy_walk(target_logits, draft_tokens, vocab, out_tokens=None,
                            accepted_len=None, status=None, stream=None):
    """As spec_verify_greedy, reading only target rows 0..n of each request."""
    _need_cuda("target_logits", target_logits)
    B, R, stride = target_logits.shape
    k = R - 1
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if accepted_len is None:
        accepted_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _need_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    rc = load_library().spec_verify_greedy_walk(
        _ptr(target_logits), _dtype_code(target_logits), stride, _ptr(draft_tokens), B, k, vocab,
        _ptr(out_tokens), _ptr(accepted_len), _ptr(status), _stream(stream))
    _check(rc, "spec_verify_greedy_walk")
    return out_tokens, accepted_len


def spec_verify_tree_greedy_walk(target_logits, node_tokens, parents, max_depth, vocab,
                                 out_tokens=None, accepted_len=None, out_path_nodes=None,
                                 status=None, stream=None):
    """As spec_verify_tree with stochastic=False, reading only the rows of
    kept nodes.  Returns (out_tokens [B][D+1], accepted_len [B],
    out_path_nodes [B][D+1] or None)."""
    _need_cuda("target_logits", target_logits)
    B, N, stride = target_logits.shape
    _need_cuda("node_tokens", node_tokens, torch.int32, (B, N))
    _need_cuda("parents", parents, torch.int32, (B, N))
    dev = target_logits.device
    W = max_depth + 1
    if out_tokens is None:
        out_tokens = torch.empty((B, W), dtype=torch.int32, device=dev)
    if accepted_len is None:
        accepted_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _need_cuda("out_tokens", out_tokens, torch.int32, (B, W))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    if out_path_nodes is not None:
        _need_cuda("out_path_nodes", out_path_nodes, torch.int32, (B, W))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    rc = load_library().spec_verify_tree_greedy_walk(
        _ptr(target_logits), _dtype_code(target_logits), stride, _ptr(node_tokens),
        _ptr(parents), B, N, max_depth, vocab, _ptr(out_tokens), _ptr(accepted_len),
        _ptr(out_path_nodes), _ptr(status), _stream(stream))
    _check(rc, "spec_verify_tree_greedy_walk")
    return out_tokens, accepted_len, out_path_nodes


def spec_verify_tree(target_logits, draft_logits, node_tokens, parents, max_depth, vocab,
                     stochastic, temperature=1.0, seed=0, offset=0, out_tokens=None,
                     accepted_len=None, out_path_nodes=None, status=None, workspace_buf=None,
                     stream=None):
    """target_logits [B][N][stride]; draft_logits [B][N][stride] or None (greedy);
    node_tokens, parents [B][N] int32.  stochastic: 0 (or False) greedy, 1 (or
    True) an independent test per node, 2 distribution-exact (siblings tested
    in turn against the residual).  Returns (out_tokens [B][D+1],
    accepted_len [B], out_path_nodes [B][D+1] or None)."""
    stochastic = int(stochastic)
    if stochastic not in (0, 1, 2):
        raise ValueError("stochastic must be 0, 1 or 2")
    _need_cuda("target_logits", target_logits)
    B, N, stride = target_logits.shape
    if stochastic:
        _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, N, stride))
    _need_cuda("node_tokens", node_tokens, torch.int32, (B, N))
    _need_cuda("parents", parents, torch.int32, (B, N))
    dev = target_logits.device
    W = max_depth + 1
    if out_tokens is None:
        out_tokens = torch.empty((B, W), dtype=torch.int32, device=dev)
    if accepted_len is None:
        accepted_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _need_cuda("out_tokens", out_tokens, torch.int32, (B, W))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    if out_path_nodes is not None:
        _need_cuda("out_path_nodes", out_path_nodes, torch.int32, (B, W))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    if workspace_buf is None:
        workspace_buf = workspace(B, 2 * N, vocab, dev) if B > 0 else None
    ws_bytes = 0 if workspace_buf is None else workspace_buf.numel()
    rc = load_library().spec_verify_tree(
        _ptr(target_logits), _ptr(draft_logits if stochastic else None),
        _dtype_code(target_logits), stride, _ptr(node_tokens), _ptr(parents), B, N, max_depth,
        vocab, int(stochastic), float(temperature), int(seed), int(offset), _ptr(out_tokens),
        _ptr(accepted_len), _ptr(out_path_nodes), _ptr(status), _ptr(workspace_buf), ws_bytes,
        _stream(stream))
    _check(rc, "spec_verify_tree")
    return out_tokens, accepted_len, out_path_nodes


def spec_verify_debug_uniforms(seed, offset, purpose, batch, count, first_position=0,
                               device=None, stream=None):
    """[batch][count] float64 device tensor of the kernels' uniforms."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    out = torch.empty((batch, count), dtype=torch.float64, device=device)
    rc = load_library().spec_verify_debug_uniforms(int(seed), int(offset), int(purpose), batch,
                                                   count, first_position, _ptr(out),
                                                   _stream(stream))
    _check(rc, "spec_verify_debug_uniforms")
    return out


def spec_verify_debug_exp2(z, kind=0, stream=None):
    """2^z (z <= 0) from one of the kernels' exponentials (kind 0: fp64
    table driven; 1: fp32 FMA-pipe polynomial; 2: fp32 special-function
    unit); z a float64 CUDA tensor."""
    _need_cuda("z", z, torch.float64)
    out = torch.empty_like(z)
    rc = load_library().spec_verify_debug_exp2(_ptr(z), _ptr(out), z.numel(), int(kind),
                                               _stream(stream))
    _check(rc, "spec_verify_debug_exp2")
    return out


def spec_verify_debug_wait_expiry(target_logits, draft_logits, draft_tokens, vocab, temperature,
                                  poll_limit, status, out_tokens=None, accepted_len=None,
                                  workspace_buf=None, stream=None):
    """spec_verify_linear with its waits made to expire after poll_limit polls
    (diagnostic: pass 1 stores nothing, so every decide step gives up and
    reports SPEC_STATUS_TIMEOUT into status; the outputs stay -1)."""
    _need_cuda("target_logits", target_logits)
    B, R, stride = target_logits.shape
    k = R - 1
    _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, stride))
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    _need_cuda("status", status, torch.int32)
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if accepted_len is None:
        accepted_len = torch.empty((B,), dtype=torch.int32, device=dev)
    if workspace_buf is None:
        workspace_buf = workspace(B, 2 * k + 1, vocab, dev) if B > 0 else None
    ws_bytes = 0 if workspace_buf is None else workspace_buf.numel()
    rc = load_library().spec_verify_debug_wait_expiry(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), stride,
        _ptr(draft_tokens), B, k, vocab, float(temperature), int(poll_limit), _ptr(out_tokens),
        _ptr(accepted_len), _ptr(status), _ptr(workspace_buf), ws_bytes, _stream(stream))
    _check(rc, "spec_verify_debug_wait_expiry")
    return out_tokens, accepted_len


def spec_verify_linear_noalloc(target_logits, draft_logits, draft_tokens, vocab, temperature,
                               seed, offset, out_tokens, accepted_len, dbg_logp=None,
                               dbg_logq=None, status=None, stream=None):
    """Linear verification through the entry point that allocates nothing.

    For callers that cannot allocate device memory (a plugin whose host
    framework owns the device pool, a serving loop that forbids cudaMalloc
    while running): the outputs must be passed in, no workspace is taken,
    and the library uses its own static 8 MiB device scratch.  Calls that
    overlap on the GPU share that scratch and must not be issued
    concurrently."""
    _need_cuda("target_logits", target_logits)
    B, R, stride = target_logits.shape
    k = R - 1
    _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, stride))
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    _need_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    for name, t in (("dbg_logp", dbg_logp), ("dbg_logq", dbg_logq)):
        if t is not None:
            _need_cuda(name, t, torch.float32, (B, k))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    rc = load_library().spec_verify_linear_noalloc(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), stride,
        _ptr(draft_tokens), B, k, vocab, float(temperature), int(seed), int(offset),
        _ptr(out_tokens), _ptr(accepted_len), _ptr(dbg_logp), _ptr(dbg_logq), _ptr(status),
        _stream(stream))
    _check(rc, "spec_verify_linear_noalloc")
    return out_tokens, accepted_len


def spec_plug_tokens(in_tokens, out_tokens, accepted_len, next_tokens=None, seq_tokens=None,
                     seq_len=None, status=None, stream=None):
    """Write the next step's input tokens from a verification's outputs on
    the device (no host synchronisation).  in_tokens, out_tokens [B][k+1],
    accepted_len [B] int32; next_tokens [B][k+1] (output, allocated when
    None and want); seq_tokens [B][cap] and seq_len [B] updated in place.
    Returns next_tokens."""
    _need_cuda("out_tokens", out_tokens, torch.int32)
    B, W = out_tokens.shape
    k = W - 1
    _need_cuda("in_tokens", in_tokens, torch.int32, (B, W))
    _need_cuda("accepted_len", accepted_len, torch.int32, (B,))
    if next_tokens is None:
        next_tokens = torch.empty((B, W), dtype=torch.int32, device=out_tokens.device)
    _need_cuda("next_tokens", next_tokens, torch.int32, (B, W))
    cap = 0
    if seq_tokens is not None or seq_len is not None:
        _need_cuda("seq_tokens", seq_tokens, torch.int32)
        if seq_tokens.dim() != 2 or seq_tokens.shape[0] != B:
            raise ValueError("seq_tokens must be [B][capacity]")
        cap = seq_tokens.shape[1]
        _need_cuda("seq_len", seq_len, torch.int32, (B,))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    rc = load_library().spec_plug_tokens(_ptr(in_tokens), _ptr(out_tokens), _ptr(accepted_len), B,
                                         k, _ptr(next_tokens), _ptr(seq_tokens), _ptr(seq_len), cap,
                                         _ptr(status), _stream(stream))
    _check(rc, "spec_plug_tokens")
    return next_tokens


# ------------------------------------------------------------ beams, paths and caches
# These calls run on the device of their tensors, whichever is current, and
# on `stream` (a stream of that device; default: the device's current one).
# What they allocate belongs to that stream.

class _On:
    """The context in which a call on `dev` runs; `handle` is its stream.
    Leaves the current device and stream alone where they are the call's."""
    __slots__ = ("handle", "outer")

    def __init__(self, dev, stream):
        self.outer = None
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
            self.outer, self.handle = torch.cuda.stream(stream), stream.cuda_stream
        else:
            if dev.index != torch._C._cuda_getDevice():
                self.outer = torch.cuda.device(dev)
            # the handle alone: torch.cuda.current_stream() makes a Stream
            # object for it, 2 us of a 10 us call (and as the tensors exist,
            # CUDA is up, which torch.cuda.current_device() would look at)
            self.handle = torch._C._cuda_getCurrentRawStream(dev.index)

    def __enter__(self):
        if self.outer is not None:
            self.outer.__enter__()
        return self.handle

    def __exit__(self, *error):
        if self.outer is not None:
            return self.outer.__exit__(*error)


def _at(t):
    """A tensor's address as ctypes takes it for a pointer argument."""
    return None if t is None else t.data_ptr()


def _need(i, name, t, dtype, shape=None):
    """_need_cuda on device i; one comparison of each kind where all is well."""
    if (t is None or t.get_device() != i or t.dtype is not dtype or (shape is not None and t.shape != shape)
            or not t.is_contiguous()):
        _need_cuda(name, t, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{i}")


@functools.lru_cache(maxsize=256)
def _bytes(call, *sizes):
    """A workspace size of the library by its function's name."""
    return getattr(load_library(), call)(*sizes)


def _scratch(need, buf, dev):
    """A workspace of `need` bytes: the caller's, or a new one (the caching
    allocator's blocks are 512-byte aligned; a captured graph gets its own)."""
    if buf is not None:
        _need(dev.index, "workspace_buf", buf, torch.uint8)
        return buf
    if need == 0:
        raise ValueError("invalid workspace request")
    return torch.empty(need, dtype=torch.uint8, device=dev)


def spec_beam_select(logits, scores, vocab, keep, temperature=1.0, finished=None, end_token=-1,
                     out_scores=None, out_parents=None, out_tokens=None, out_finished=None,
                     status=None, workspace_buf=None, stream=None):
    """The `keep` best continuations (beam, token) of each request by summed
    log probability.  logits [B][W][stride] (bf16/fp32), scores [B][W] fp32,
    finished [B][W] int32 or None (an ended beam goes on as end_token with
    its score unchanged).  Returns (scores [B][keep], parents [B][keep],
    tokens [B][keep], finished [B][keep] or None)."""
    _need_cuda("logits", logits)
    B, W, stride = logits.shape
    keep = int(keep)
    dev = logits.device
    i = dev.index
    _need(i, "scores", scores, torch.float32, (B, W))
    if finished is not None:
        _need(i, "finished", finished, torch.int32, (B, W))
    with _On(dev, stream) as handle:
        if out_scores is None:
            out_scores = torch.empty((B, keep), dtype=torch.float32, device=dev)
        if out_parents is None:
            out_parents = torch.empty((B, keep), dtype=torch.int32, device=dev)
        if out_tokens is None:
            out_tokens = torch.empty((B, keep), dtype=torch.int32, device=dev)
        if out_finished is None and finished is not None:
            out_finished = torch.empty((B, keep), dtype=torch.int32, device=dev)
        _need(i, "out_scores", out_scores, torch.float32, (B, keep))
        _need(i, "out_parents", out_parents, torch.int32, (B, keep))
        _need(i, "out_tokens", out_tokens, torch.int32, (B, keep))
        if out_finished is not None:
            _need(i, "out_finished", out_finished, torch.int32, (B, keep))
        if status is not None:
            _need(i, "status", status, torch.int32)
        lib = load_library()
        code = _dtype_code(logits)
        ws = None
        if B > 0:
            need = _bytes("spec_beam_workspace_size", B, W, vocab)
            ws = _scratch(need, workspace_buf, dev) if need else workspace_buf
        rc = lib.spec_beam_select(
            _at(logits), code, stride, _at(scores), _at(finished), int(end_token), B, W, vocab,
            float(temperature), keep, _at(out_scores), _at(out_parents), _at(out_tokens),
            _at(out_finished), _at(status), _at(ws), 0 if ws is None else ws.numel(),
            handle)
    _check(rc, "spec_beam_select")
    return out_scores, out_parents, out_tokens, out_finished


def _one_stride(sizes, strides):
    """(count, stride) of the flattened dimensions, or None if no single stride steps over them."""
    count, step = 1, 0
    for n, s in zip(reversed(sizes), reversed(strides)):
        if n == 1:
            continue
        if count == 1:
            step = s
        elif s != count * step:
            return None
        count *= n
    return count, step


@functools.lru_cache(maxsize=256)
def _layout(shape, stride, e, lead, axis):
    """Of a state of these sizes and strides and e bytes an element:
    (segments, segment stride, unit bytes, capacity).  Kept per layout: a
    serving loop has a few and asks for them at every step."""
    if len(shape) < lead or (axis is not None and not lead <= axis < len(shape)):
        raise ValueError("axis must be a dimension after the request's and the beam's")
    inner = lead if axis is None else axis + 1
    whole = _one_stride(shape[inner:], stride[inner:])
    if whole is None or (whole[0] > 1 and whole[1] != 1):
        raise ValueError("the dimensions of a unit must be contiguous")
    unit = whole[0] * e
    if axis is None:
        return 1, 0, unit, 1
    if shape[axis] > 1 and stride[axis] * e != unit:
        raise ValueError("the units must follow one another")
    seg = _one_stride(shape[lead:axis], stride[lead:axis])
    if seg is None:
        raise ValueError("the dimensions before the units must have one stride")
    return seg[0], seg[1] * e, unit, shape[axis]


def _state_layout(states, lead, axis):
    """The common layout of `states`, whose first `lead` dimensions are the
    request (and the beam): (segments, segment stride, unit bytes, capacity)
    and the device.  axis: the dimension of the units (positions), or None
    where a whole state is one unit."""
    t = states[0]
    if not t.is_cuda:
        raise ValueError("the states must be CUDA tensors")
    shape, stride, dtype, dev = t.shape, t.stride(), t.dtype, t.get_device()
    for x in states:
        if x.shape != shape or x.stride() != stride or x.dtype is not dtype or x.get_device() != dev:
            raise ValueError("the states must share device, dtype, shape and strides")
    return *_layout(shape, stride, t.element_size(), lead, axis), t.device


def _pointers(states):
    """The states' addresses as an array of 64-bit integers."""
    return array.array("Q", [t.data_ptr() for t in states])


def spec_reorder_beams(states, parents, axis=None, begin=None, end=None, status=None, stream=None):
    """states[s][b][j] <- states[s][b][parents[b][j]], in place.  states: a
    list of tensors [B][W][...] of one layout (at most MAX_STATES); parents
    [B][width] int32, width <= W (-1: left as it was).  axis: the dimension
    of positions, of which only [begin[b], end[b]) move ([B] int32, None: the
    first and one past the last); axis None moves whole states.  Returns
    states."""
    states = list(states)
    _need_cuda("parents", parents, torch.int32)
    if parents.dim() != 2:
        raise ValueError("parents must be [B][width]")
    B, width = parents.shape
    if not states:
        return states
    segments, seg_stride, unit, cap, dev = _state_layout(states, 2, axis)
    W = states[0].shape[1]
    if states[0].shape[0] != B:
        raise ValueError(f"parents must have {states[0].shape[0]} rows, got {B}")
    if axis is None and (begin is not None or end is not None):
        raise ValueError("begin and end need axis")
    _need(dev.index, "parents", parents, torch.int32)
    for name, t in (("begin", begin), ("end", end), ("status", status)):
        if t is not None:
            _need(dev.index, name, t, torch.int32, None if t is status else (B,))
    e = states[0].element_size()
    addresses = _pointers(states)
    with _On(dev, stream) as handle:
        rc = load_library().spec_reorder_beams(
            addresses.buffer_info()[0], len(states), states[0].stride(0) * e, states[0].stride(1) * e,
            segments, seg_stride, unit, cap, _at(begin), _at(end), _at(parents), B, W, width,
            _at(status), handle)
    _check(rc, "spec_reorder_beams")
    return states


def spec_commit_path(states, base, path, num_nodes, axis, out_lens=None, status=None, stream=None):
    """Move the rows of an accepted tree path together, in place: position
    base[b] + i <- base[b] + path[b][i].  states: a list of tensors [B][...]
    of one layout whose dimension `axis` holds the positions; base [B] int32
    or None (0); path [B][width] int32 (spec_verify_tree's out_path_nodes).
    Returns the new lengths [B] int32 (base + nodes of the path)."""
    states = list(states)
    _need_cuda("path", path, torch.int32)
    if path.dim() != 2:
        raise ValueError("path must be [B][width]")
    B, width = path.shape
    segments, seg_stride, unit, cap, dev = 1, 0, 1, 1 << 30, path.device
    if states:
        segments, seg_stride, unit, cap, dev = _state_layout(states, 1, axis)
        if states[0].shape[0] != B:
            raise ValueError(f"path must have {states[0].shape[0]} rows, got {B}")
    _need(dev.index, "path", path, torch.int32)
    if base is not None:
        _need(dev.index, "base", base, torch.int32, (B,))
    with _On(dev, stream) as handle:
        if out_lens is None:
            out_lens = torch.empty((B,), dtype=torch.int32, device=dev)
        _need(dev.index, "out_lens", out_lens, torch.int32, (B,))
        if status is not None:
            _need(dev.index, "status", status, torch.int32)
        step = states[0].stride(0) * states[0].element_size() if states else cap
        addresses = _pointers(states)
        rc = load_library().spec_commit_path(
            addresses.buffer_info()[0], len(states), step, segments, seg_stride, unit, cap, _at(base),
            _at(path), B, int(num_nodes), width, _at(out_lens), _at(status), handle)
    _check(rc, "spec_commit_path")
    return out_lens


def _inner_contiguous(name, t, dims):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")


def spec_cache_score(q, k, begin, end, scores, scale=None, out_scores=None, status=None,
                     workspace_buf=None, stream=None):
    """Add the attention weight that a step's queries give a cache's slots.
    q [B][Q][heads][D], k [B][kv_heads][capacity][D] (bf16/fp32, any strides
    with D contiguous: a cache [B][capacity][kv_heads][D] is passed as
    k.transpose(1, 2)); begin, end [B] int32: filled slots before and after
    the step (query i sits at slot begin + i; end - begin <= Q);
    scores [B][kv_heads][capacity] fp32.  scale: default D ** -0.5.  Writes
    out_scores (default: scores, in place) below `end` and returns it."""
    _inner_contiguous("q", q, 4)
    _inner_contiguous("k", k, 4)
    B, Q, Hq, D = q.shape
    H, cap = k.shape[1], k.shape[2]
    if k.dtype != q.dtype or tuple(k.shape) != (B, H, cap, D):
        raise ValueError(f"k must be [{B}][kv_heads][capacity][{D}] of {q.dtype}, got {tuple(k.shape)} {k.dtype}")
    dev = q.device
    i = dev.index
    if k.get_device() != i:
        raise ValueError(f"k is on {k.device}, not on {dev}")
    _need(i, "begin", begin, torch.int32, (B,))
    _need(i, "end", end, torch.int32, (B,))
    _need(i, "scores", scores, torch.float32, (B, H, cap))
    out_scores = scores if out_scores is None else out_scores
    _need(i, "out_scores", out_scores, torch.float32, (B, H, cap))
    if status is not None:
        _need(i, "status", status, torch.int32)
    scale = D ** -0.5 if scale is None else float(scale)
    lib = load_library()
    code = _dtype_code(q)
    with _On(dev, stream) as handle:
        ws = None
        if B > 0:
            need = _bytes("spec_score_workspace_size_for", code, D, B, Q, Hq, H, cap)
            ws = _scratch(need, workspace_buf, dev) if need else workspace_buf
        rc = lib.spec_cache_score(
            _at(q), _at(k), code, *q.stride()[:3], *k.stride()[:3], _at(begin), _at(end), B, Q, Hq, H, D, cap, scale,
            _at(scores), _at(out_scores), _at(status), _at(ws),
            0 if ws is None else ws.numel(), handle)
    _check(rc, "spec_cache_score")
    return out_scores


def spec_cache_evict(k, v, scores, positions, lens, budget, sinks=0, recent=0, out_scores=None,
                     out_positions=None, out_lens=None, status=None, workspace_buf=None, stream=None):
    """Cut a cache down to `budget` slots a head by accumulated attention
    weight, k and v in place.  k, v [B][H][capacity][D] (any dtype, any
    strides with D contiguous; v may be None), scores [B][H][capacity] fp32,
    positions the same shape int32, lens [B] int32.  Positions < sinks and the
    `recent` newest stay in any case.  Returns (out_scores, out_positions,
    out_lens); the first two default to in place, out_lens to a new tensor."""
    _inner_contiguous("k", k, 4)
    B, H, cap, _ = k.shape
    dev = k.device
    i = dev.index
    if v is not None:
        _inner_contiguous("v", v, 4)
        if tuple(v.shape[:3]) != (B, H, cap):
            raise ValueError(f"v must be [{B}][{H}][{cap}][D], got {tuple(v.shape)}")
        if v.get_device() != i:
            raise ValueError(f"v is on {v.device}, not on {dev}")
    _need(i, "scores", scores, torch.float32, (B, H, cap))
    _need(i, "positions", positions, torch.int32, (B, H, cap))
    _need(i, "lens", lens, torch.int32, (B,))
    out_scores = scores if out_scores is None else out_scores
    out_positions = positions if out_positions is None else out_positions
    _need(i, "out_scores", out_scores, torch.float32, (B, H, cap))
    _need(i, "out_positions", out_positions, torch.int32, (B, H, cap))

    def layout(t):
        e, s = t.element_size(), t.stride()
        return s[0] * e, s[1] * e, s[2] * e, t.shape[3] * e

    lib = load_library()
    with _On(dev, stream) as handle:
        if out_lens is None:
            out_lens = torch.empty((B,), dtype=torch.int32, device=dev)
        _need(i, "out_lens", out_lens, torch.int32, (B,))
        if status is not None:
            _need(i, "status", status, torch.int32)
        ws = None
        if B > 0:
            need = _bytes("spec_evict_workspace_size", B, H, cap, int(budget))
            ws = _scratch(need, workspace_buf, dev) if need else workspace_buf
        rc = lib.spec_cache_evict(
            _at(k), _at(v), *layout(k), *(layout(v) if v is not None else (0, 0, 0, 0)),
            _at(scores), _at(positions), _at(lens), B, H, cap, int(budget), int(sinks),
            int(recent), _at(out_scores), _at(out_positions), _at(out_lens), _at(status),
            _at(ws), 0 if ws is None else ws.numel(), handle)
    _check(rc, "spec_cache_evict")
    return out_scores, out_positions, out_lens


# ------------------------------------------------------------ vocabulary-sharded steps
SHARD_DRAW_WORDS = 6


def spec_shard_row_stats(target_logits, draft_logits, draft_tokens, vocab_lo, vocab_hi,
                         temperature=1.0, stream=None):
    """Per-row statistics of this rank's columns [vocab_lo, vocab_hi).
    Stochastic (draft_logits given): dict(max [B][2k+1] f32, sum [B][2k+1]
    f64, probe [B][k][2] f32); greedy (draft_logits None): dict(max
    [B][k+1] f32, arg [B][k+1] int32)."""
    _need_cuda("target_logits", target_logits)
    B, R1, stride = target_logits.shape
    k = R1 - 1
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    dev = target_logits.device
    stoch = draft_logits is not None
    if stoch:
        _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, stride))
    R = 2 * k + 1 if stoch else k + 1
    mx = torch.empty((B, R), dtype=torch.float32, device=dev)
    sm = torch.empty((B, R), dtype=torch.float64, device=dev) if stoch else None
    arg = None if stoch else torch.empty((B, R), dtype=torch.int32, device=dev)
    probe = torch.empty((B, k, 2), dtype=torch.float32, device=dev) if stoch else None
    rc = load_library().spec_shard_row_stats(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), stride,
        _ptr(draft_tokens), B, k, int(vocab_lo), int(vocab_hi), float(temperature), _ptr(mx),
        _ptr(sm), _ptr(arg), _ptr(probe), _stream(stream))
    _check(rc, "spec_shard_row_stats")
    return dict(max=mx, sum=sm, arg=arg, probe=probe)


def spec_shard_decide(max_all, sum_all, probe_all, bounds, draft_tokens, vocab, temperature,
                      seed=0, offset=0, status=None, stream=None):
    """Merge the ranks' statistics (rank order) and run the accept tests.
    Returns (out_tokens [B][k+1] with the drawn slot still -1,
    accepted_len [B], draw [B][6] f64)."""
    _need_cuda("max_all", max_all, torch.float32)
    W, B, R = max_all.shape
    k = (R - 1) // 2
    _need_cuda("sum_all", sum_all, torch.float64, (W, B, R))
    _need_cuda("probe_all", probe_all, torch.float32, (W, B, k, 2))
    _need_cuda("bounds", bounds, torch.int32, (W + 1,))
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    dev = max_all.device
    out = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    acc = torch.empty((B,), dtype=torch.int32, device=dev)
    draw = torch.empty((B, SHARD_DRAW_WORDS), dtype=torch.float64, device=dev)
    rc = load_library().spec_shard_decide(
        _ptr(max_all), _ptr(sum_all), _ptr(probe_all), _ptr(bounds), W, _ptr(draft_tokens), B, k,
        int(vocab), float(temperature), int(seed), int(offset), _ptr(out), _ptr(acc), _ptr(draw),
        _ptr(status), _stream(stream))
    _check(rc, "spec_shard_decide")
    return out, acc, draw


def spec_shard_decide_greedy(max_all, arg_all, draft_tokens, vocab, status=None, stream=None):
    """Greedy verification from the ranks' (max, lowest argmax) per target row."""
    _need_cuda("max_all", max_all, torch.float32)
    W, B, R = max_all.shape
    k = R - 1
    _need_cuda("arg_all", arg_all, torch.int32, (W, B, R))
    _need_cuda("draft_tokens", draft_tokens, torch.int32, (B, k))
    if status is not None:
        _need_cuda("status", status, torch.int32)
    dev = max_all.device
    out = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    acc = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = load_library().spec_shard_decide_greedy(_ptr(max_all), _ptr(arg_all), W, _ptr(draft_tokens),
                                                 B, k, int(vocab), _ptr(out), _ptr(acc),
                                                 _ptr(status), _stream(stream))
    _check(rc, "spec_shard_decide_greedy")
    return out, acc


def spec_shard_draw_sums(target_logits, draft_logits, vocab_lo, vocab_hi, temperature, draw,
                         norm_parts=None, stream=None):
    """fp64 sums over this rank's columns of each request's draw rows:
    without norm_parts (sum e, sum f); with the ranks' gathered first sums
    [W][B][2] (the draw mass, sum e).  Returns [B][2] f64."""
    _need_cuda("target_logits", target_logits)
    B, R1, stride = target_logits.shape
    k = R1 - 1
    _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, stride))
    _need_cuda("draw", draw, torch.float64, (B, SHARD_DRAW_WORDS))
    W = 1
    if norm_parts is not None:
        _need_cuda("norm_parts", norm_parts, torch.float64)
        W = norm_parts.shape[0]
    sums = torch.empty((B, 2), dtype=torch.float64, device=target_logits.device)
    rc = load_library().spec_shard_draw_sums(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), stride, B, k,
        int(vocab_lo), int(vocab_hi), float(temperature), _ptr(draw), _ptr(norm_parts), W,
        _ptr(sums), _stream(stream))
    _check(rc, "spec_shard_draw_sums")
    return sums


def spec_shard_draw_pick(target_logits, draft_logits, vocab_lo, vocab_hi, temperature, draw,
                         norm_parts, mass_parts, shard_index, stream=None):
    """The token of each request if this rank owns the part of the running
    mass that holds u * Z (drawn inside its columns), else -1.  [B] int32."""
    _need_cuda("target_logits", target_logits)
    B, R1, stride = target_logits.shape
    k = R1 - 1
    _need_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, stride))
    _need_cuda("draw", draw, torch.float64, (B, SHARD_DRAW_WORDS))
    _need_cuda("norm_parts", norm_parts, torch.float64)
    W = norm_parts.shape[0]
    _need_cuda("mass_parts", mass_parts, torch.float64, (W, B, 2))
    token = torch.empty((B,), dtype=torch.int32, device=target_logits.device)
    rc = load_library().spec_shard_draw_pick(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), stride, B, k,
        int(vocab_lo), int(vocab_hi), float(temperature), _ptr(draw), _ptr(norm_parts),
        _ptr(mass_parts), W, int(shard_index), _ptr(token), _stream(stream))
    _check(rc, "spec_shard_draw_pick")
    return token


def spec_shard_emit(token, draw, out_tokens, stream=None):
    """out_tokens[b][n] = token[b] for every request that draws one."""
    _need_cuda("out_tokens", out_tokens, torch.int32)
    B, W1 = out_tokens.shape
    _need_cuda("token", token, torch.int32, (B,))
    _need_cuda("draw", draw, torch.float64, (B, SHARD_DRAW_WORDS))
    rc = load_library().spec_shard_emit(_ptr(token), _ptr(draw), B, W1 - 1, _ptr(out_tokens),
                                        _stream(stream))
    _check(rc, "spec_shard_emit")
    return out_tokens
