"""Python binding of libgdn.so: the Gated DeltaNet recurrence on MI355X (gfx950).

Thin ctypes wrappers with the same names as the C ABI in include/gdn.h. They check that
tensors are contiguous CUDA (HIP) tensors of the right dtype, allocate outputs and the
workspace with torch when the caller does not pass them, and hand raw device pointers and
the current stream to the library. Every step of the computation runs in the library's
HIP kernels; there is no Python or CPU fallback, and a missing libgdn.so is an error.

For a hybrid stack's softmax-attention layers there are a paged key-value cache
(gdn_kv_write, gdn_kv_read), attention over packed prompts (gdn_attn_prefill) and of one new
token over the cache (gdn_attn_decode); around them the norms and rotary positions of queries and
keys (gdn_qk_norm_rope), the cache written with them on the way (gdn_kv_append), and attention of
several new tokens over the cache, with a sliding window (gdn_attn_extend). Their tensors are
described at each function.

Layouts of the recurrence (see include/gdn.h): q, k [n, t, h_qk, d]; v [n, t, h_v, d]; g, beta [n, t, h_v]
fp32; state [n, h_v, d, d] fp32 with element [i][j] = S[j][i]; out [n, t, h_v, d] fp32.
"""
import ctypes
import os

import torch

__all__ = [
    "GdnError", "gdn_abi_version", "gdn_status_str", "gdn_workspace_bytes",
    "gdn_prefill_chunked", "gdn_prefill_scan", "gdn_decode_step", "gdn_prefill_choose",
    "gdn_prefill", "gdn_prefill_workspace_bytes", "library_path", "Dims", "BoundCall",
    "bind_prefill_chunked", "bind_prefill_scan", "bind_decode_step", "DecodeGraph",
    "gdn_prefill_segmented", "gdn_prefill_segmented_workspace_bytes", "gdn_prefill_scan_blockwise",
    "calib_mfma_bf16", "calib_stream_copy", "gdn_prefill_segmented_noalloc", "gdn_noalloc_scratch_bytes",
    "debug_fill_lds", "gdn_kv_write", "gdn_kv_read", "gdn_attn_prefill", "gdn_attn_decode",
    "gdn_attn_prefill_workspace_bytes", "gdn_attn_decode_workspace_bytes", "KvCache", "AttnDims",
    "gdn_qk_norm_rope", "gdn_kv_append", "gdn_attn_extend", "gdn_attn_extend_workspace_bytes", "NormRope",
    "ExtendDims",
]

GDN_F32, GDN_BF16, GDN_FP8 = 0, 1, 2
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdn.so")
_lib = None


class Dims(ctypes.Structure):
    """gdn_dims from include/gdn.h."""
    _fields_ = [("n", ctypes.c_int64), ("t", ctypes.c_int64), ("h_qk", ctypes.c_int32),
                ("h_v", ctypes.c_int32), ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("qkv_dtype", ctypes.c_int32), ("l2_eps", ctypes.c_float)]


class KvCache(ctypes.Structure):
    """gdn_kv_cache from include/gdn.h."""
    _fields_ = [("n", ctypes.c_int64), ("num_pages", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("store", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


class AttnDims(ctypes.Structure):
    """gdn_attn_dims from include/gdn.h."""
    _fields_ = [("n", ctypes.c_int64), ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
                ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64)]


class NormRope(ctypes.Structure):
    """gdn_norm_rope from include/gdn.h."""
    _fields_ = [("eps", ctypes.c_float), ("weight_bias", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("rope_scale", ctypes.c_float), ("freq", ctypes.c_void_p),
                ("axis", ctypes.c_void_p), ("pos", ctypes.c_void_p)]


class ExtendDims(ctypes.Structure):
    """gdn_extend_dims from include/gdn.h."""
    _fields_ = [("total_q", ctypes.c_int64), ("max_q", ctypes.c_int64), ("max_len", ctypes.c_int64),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("h_q", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64)]


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdn_status_str(status)}")


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                           "(the HIP library is required, there is no fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, D = ctypes.c_void_p, ctypes.POINTER(Dims)
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    K = ctypes.POINTER(KvCache)
    sig = {
        "gdn_abi_version": (i32, []),
        "gdn_status_str": (ctypes.c_char_p, [ctypes.c_int32]),
        "gdn_workspace_bytes": (sz, [D, i32]),
        "gdn_prefill_chunked": (ctypes.c_int, [D, i32] + [P] * 9 + [sz, P]),
        "gdn_prefill_scan": (ctypes.c_int, [D] + [P] * 9 + [sz, P]),
        "gdn_decode_step": (ctypes.c_int, [D] + [P] * 9),
        "gdn_prefill_choose": (ctypes.c_int, [D, ctypes.POINTER(i32)]),
        "gdn_prefill_workspace_bytes": (sz, [D]),
        "gdn_prefill": (ctypes.c_int, [D] + [P] * 9 + [sz, P]),
        "gdn_decode_graph_create": (ctypes.c_int, [D, i32] + [ctypes.POINTER(P)] * 7 + [P, ctypes.POINTER(P)]),
        "gdn_graph_launch": (ctypes.c_int, [P, P]),
        "gdn_graph_destroy": (ctypes.c_int, [P]),
        "gdn_calib_mfma_bf16_flops": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int32]),
        "gdn_calib_mfma_bf16": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int32, P, P]),
        "gdn_prefill_scan_blockwise": (ctypes.c_int, [D, ctypes.c_int64] + [P] * 9 + [sz, P]),
        "gdn_prefill_segmented_workspace_bytes": (sz, [D, ctypes.c_int64, ctypes.c_int32]),
        "gdn_prefill_segmented": (ctypes.c_int, [D, ctypes.c_int64, ctypes.c_int32] + [P] * 9
                                  + [sz, P]),
        "gdn_noalloc_scratch_bytes": (sz, []),
        "gdn_calib_stream_copy": (ctypes.c_int, [P, P, ctypes.c_int64, ctypes.c_int32, P]),
        "gdn_prefill_segmented_noalloc": (ctypes.c_int, [D, ctypes.c_int64] + [P] * 9),
        "gdn_kv_write": (ctypes.c_int, [K, i64, i32, P, i64, i64, P, i64, i64, P, P, P]),
        "gdn_kv_read": (ctypes.c_int, [K, i64, i32, P, P, P, P, P]),
        "gdn_attn_prefill_workspace_bytes": (sz, [ctypes.POINTER(AttnDims)]),
        "gdn_attn_prefill": (ctypes.c_int, [ctypes.POINTER(AttnDims)] + [P] * 8 + [sz, P]),
        "gdn_attn_decode_workspace_bytes": (sz, [K, i32, i64]),
        "gdn_attn_decode": (ctypes.c_int, [K, i32, i32, ctypes.c_float, i64, P, i64, i64, P, P, P,
                                           P, sz, P]),
        "gdn_qk_norm_rope": (ctypes.c_int, [ctypes.POINTER(NormRope), i64, i32, i32, i32, i32, P, i64, i64, P, i64,
                                            i64, P, P, P]),
        "gdn_kv_append": (ctypes.c_int, [K, ctypes.POINTER(NormRope), i64, i32, P, i64, i64, P, i64, i64, P, P, i32,
                                         P, i64, i64, P, P]),
        "gdn_attn_extend_workspace_bytes": (sz, [K, ctypes.POINTER(ExtendDims)]),
        "gdn_attn_extend": (ctypes.c_int, [K, ctypes.POINTER(ExtendDims)] + [P] * 6 + [sz, P]),
        "gdn_debug_fill_lds": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_int32, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


def gdn_abi_version() -> int:
    return _load().gdn_abi_version()


def gdn_status_str(status: int) -> str:
    return _load().gdn_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise GdnError(status, where)


def make_dims(n, t, h_qk, h_v, d, dtype=torch.bfloat16, l2_eps=1e-6) -> Dims:
    return Dims(int(n), int(t), int(h_qk), int(h_v), int(d), int(d),
                _DTYPES.get(dtype, -1), float(l2_eps))


def _dims_of(q, v, l2_eps) -> Dims:
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [n, t, h_qk, d] and v [n, t, h_v, d]")
    n, t, h_qk, d_k = q.shape
    d = Dims(n, t, h_qk, v.shape[2], d_k, v.shape[3], _DTYPES.get(q.dtype, -1), float(l2_eps))
    return d


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check_tensor(name, x, shape, dtype, dev):
    """x must be a contiguous CUDA (HIP) tensor on dev with exactly this shape and dtype."""
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not x.is_cuda or x.device != dev:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor on {dev}")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps):
    """Check every tensor of a call against the sizes q and v define (all before any
    launch: a wrong shape, dtype, device or layout would otherwise reach the kernels as a
    raw pointer) and allocate out / state_out when they are not given."""
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise ValueError("q and v must be torch tensors")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [n, t, h_qk, d] and v [n, t, h_v, d]")
    if q.dtype not in _DTYPES:
        raise ValueError("q, k, v must share one dtype, bfloat16 or float32")
    dev = q.device
    n, t, h_qk, d = q.shape
    h_v = v.shape[2]
    f32 = torch.float32
    _check_tensor("q", q, (n, t, h_qk, d), q.dtype, dev)
    _check_tensor("k", k, (n, t, h_qk, d), q.dtype, dev)
    _check_tensor("v", v, (n, t, h_v, v.shape[3]), q.dtype, dev)
    if v.shape[3] != d:
        raise ValueError(f"v must have shape {(n, t, h_v, d)}, got {tuple(v.shape)}")
    _check_tensor("g", g, (n, t, h_v), f32, dev)
    _check_tensor("beta", beta, (n, t, h_v), f32, dev)
    if state_in is not None:
        _check_tensor("state_in", state_in, (n, h_v, d, d), f32, dev)
    dims = _dims_of(q, v, l2_eps)
    if out is None:
        out = torch.empty((n, t, h_v, d), device=dev, dtype=f32)
    else:
        _check_tensor("out", out, (n, t, h_v, d), f32, dev)
    if state_out is None:
        state_out = torch.empty((n, h_v, d, d), device=dev, dtype=f32)
    else:
        _check_tensor("state_out", state_out, (n, h_v, d, d), f32, dev)
    return dims, out, state_out


def _check_workspace(workspace, dev):
    """A caller-supplied workspace: a contiguous uint8 tensor on the call's device."""
    if workspace is None:
        return 0
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 torch tensor")
    if not workspace.is_cuda or workspace.device != dev:
        raise ValueError(f"workspace must be a CUDA (HIP) tensor on {dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.numel()


def _workspace(dims, chunk, workspace, dev):
    need = _load().gdn_workspace_bytes(ctypes.byref(dims), int(chunk))
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    return workspace, _check_workspace(workspace, dev)


def gdn_workspace_bytes(n, t, h_qk, h_v, d, dtype=torch.bfloat16, chunk=64) -> int:
    """Workspace bytes for gdn_prefill_chunked (chunk > 0) or gdn_prefill_scan (chunk 0)."""
    return _load().gdn_workspace_bytes(ctypes.byref(make_dims(n, t, h_qk, h_v, d, dtype)),
                                       int(chunk))


def gdn_prefill_chunked(q, k, v, g, beta, state_in=None, *, chunk=64, l2_eps=1e-6, out=None,
                        state_out=None, workspace=None, stream=None):
    """Chunked prefill. Returns (out, state_out)."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    workspace, wbytes = _workspace(dims, chunk, workspace, q.device)
    _check(_load().gdn_prefill_chunked(
        ctypes.byref(dims), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state_in), _ptr(out), _ptr(state_out), _ptr(workspace), wbytes,
        _stream(q.device, stream)), "gdn_prefill_chunked")
    return out, state_out


def gdn_prefill_scan(q, k, v, g, beta, state_in=None, *, l2_eps=1e-6, out=None,
                     state_out=None, workspace=None, stream=None):
    """Direct-scan prefill. Returns (out, state_out)."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    workspace, wbytes = _workspace(dims, 0, workspace, q.device)
    _check(_load().gdn_prefill_scan(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_in),
        _ptr(out), _ptr(state_out), _ptr(workspace), wbytes, _stream(q.device, stream)),
        "gdn_prefill_scan")
    return out, state_out


def gdn_prefill_scan_blockwise(q, k, v, g, beta, state_in=None, *, block_t, l2_eps=1e-6,
                               out=None, state_out=None, workspace=None, stream=None):
    """The residency ablation of gdn_prefill_scan: one scan launch per block of block_t
    tokens, the state written to and read back from state_out between blocks. Returns
    (out, state_out)."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    workspace, wbytes = _workspace(dims, 0, workspace, q.device)
    _check(_load().gdn_prefill_scan_blockwise(
        ctypes.byref(dims), int(block_t), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state_in), _ptr(out), _ptr(state_out), _ptr(workspace), wbytes,
        _stream(q.device, stream)), "gdn_prefill_scan_blockwise")
    return out, state_out


def calib_mfma_bf16(iters, blocks, sink, stream=None) -> int:
    """Launch the bf16 MFMA loop (measurement only) into `sink` (a float32 device tensor of
    at least blocks * 256 elements); returns the flops the launch performs."""
    assert sink.dtype == torch.float32 and sink.is_cuda and sink.numel() >= blocks * 256
    _check(_load().gdn_calib_mfma_bf16(int(iters), int(blocks), _ptr(sink),
                                       _stream(sink.device, stream)), "gdn_calib_mfma_bf16")
    return int(_load().gdn_calib_mfma_bf16_flops(int(iters), int(blocks)))


def calib_stream_copy(src, dst, blocks=1024, stream=None):
    """Launch the streaming-copy calibration kernel (measurement only): dst <- src, two
    contiguous device tensors of the same byte size (a multiple of 16)."""
    nbytes = src.numel() * src.element_size()
    if not (src.is_cuda and dst.is_cuda and src.is_contiguous() and dst.is_contiguous()
            and dst.numel() * dst.element_size() == nbytes):
        raise ValueError("src and dst must be contiguous device tensors of the same byte size")
    _check(_load().gdn_calib_stream_copy(_ptr(src), _ptr(dst), nbytes, int(blocks),
                                         _stream(src.device, stream)), "gdn_calib_stream_copy")


def debug_fill_lds(sink, pattern=0x7FC00000, blocks=1024, stream=None):
    """Fill the LDS of every CU with a 32-bit pattern (testing only; default a quiet NaN),
    so that a kernel launched next on the same stream that reads LDS it never wrote sees
    that pattern. `sink`: an int32 device tensor of at least one element, written only if
    the fill failed."""
    _check_tensor("sink", sink, (sink.numel(),), torch.int32, sink.device)
    if sink.numel() < 1:
        raise ValueError("sink: need at least one element")
    _check(_load().gdn_debug_fill_lds(int(pattern) & 0xFFFFFFFF, int(blocks), _ptr(sink),
                                      _stream(sink.device, stream)), "gdn_debug_fill_lds")


def gdn_decode_step(q, k, v, g, beta, state_in=None, *, l2_eps=1e-6, out=None,
                    state_out=None, stream=None):
    """One decode token per sequence (t == 1). Returns (out, state_out); pass
    state_out=state_in to update the state in place."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    _check(_load().gdn_decode_step(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_in),
        _ptr(out), _ptr(state_out), _stream(q.device, stream)), "gdn_decode_step")
    return out, state_out


def gdn_prefill_choose(t, h_qk=16, h_v=32, d=128, n=1, dtype=torch.bfloat16) -> int:
    """The measured scan/chunk choice: 0 for the direct scan, else a chunk size."""
    res = ctypes.c_int32(-1)
    _check(_load().gdn_prefill_choose(ctypes.byref(make_dims(n, t, h_qk, h_v, d, dtype)),
                                      ctypes.byref(res)), "gdn_prefill_choose")
    return res.value


def gdn_prefill_workspace_bytes(n, t, h_qk, h_v, d, dtype=torch.bfloat16) -> int:
    return _load().gdn_prefill_workspace_bytes(ctypes.byref(make_dims(n, t, h_qk, h_v, d, dtype)))


def gdn_prefill(q, k, v, g, beta, state_in=None, *, l2_eps=1e-6, out=None, state_out=None,
                workspace=None, stream=None):
    """Prefill with the method gdn_prefill_choose picks. Returns (out, state_out)."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    if workspace is None:
        need = _load().gdn_prefill_workspace_bytes(ctypes.byref(dims))
        if need > 0:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    wbytes = _check_workspace(workspace, q.device)
    _check(_load().gdn_prefill(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_in),
        _ptr(out), _ptr(state_out), _ptr(workspace), wbytes, _stream(q.device, stream)),
        "gdn_prefill")
    return out, state_out


class BoundCall:
    """One library call with its arguments marshalled once (for loops that replay the same
    call, such as benchmarks or a layer stack). Calling it enqueues the kernels on the
    stream that was current at bind time and raises GdnError on a non-OK status."""

    def __init__(self, fn, args, where, keep):
        self._fn, self._args, self._where, self._keep = fn, args, where, keep

    def __call__(self):
        st = self._fn(*self._args)
        if st != 0:
            raise GdnError(st, self._where)


def bind_prefill_chunked(q, k, v, g, beta, state_in, out, state_out, workspace, *, chunk=64,
                         l2_eps=1e-6, stream=None) -> BoundCall:
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    nbytes = _check_workspace(workspace, q.device)
    args = (ctypes.byref(dims), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
            _ptr(state_in), _ptr(out), _ptr(state_out), _ptr(workspace), nbytes,
            _stream(q.device, stream))
    return BoundCall(_load().gdn_prefill_chunked, args, "gdn_prefill_chunked",
                     (dims, q, k, v, g, beta, state_in, out, state_out, workspace))


def bind_prefill_scan(q, k, v, g, beta, state_in, out, state_out, workspace, *, l2_eps=1e-6,
                      stream=None) -> BoundCall:
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    nbytes = _check_workspace(workspace, q.device)
    args = (ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_in),
            _ptr(out), _ptr(state_out), _ptr(workspace), nbytes, _stream(q.device, stream))
    return BoundCall(_load().gdn_prefill_scan, args, "gdn_prefill_scan",
                     (dims, q, k, v, g, beta, state_in, out, state_out, workspace))


def bind_decode_step(q, k, v, g, beta, state_in, out, state_out, *, l2_eps=1e-6,
                     stream=None) -> BoundCall:
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    args = (ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_in),
            _ptr(out), _ptr(state_out), _stream(q.device, stream))
    return BoundCall(_load().gdn_decode_step, args, "gdn_decode_step",
                     (dims, q, k, v, g, beta, state_in, out, state_out))


def gdn_prefill_segmented_workspace_bytes(n, t, h_qk, h_v, d, seg_t, overlapped=False,
                                          dtype=torch.bfloat16) -> int:
    return _load().gdn_prefill_segmented_workspace_bytes(
        ctypes.byref(make_dims(n, t, h_qk, h_v, d, dtype)), int(seg_t), int(bool(overlapped)))


def gdn_prefill_segmented(q, k, v, g, beta, state_in=None, *, seg_t, overlapped=False,
                          l2_eps=1e-6, out=None, state_out=None, workspace=None, stream=None):
    """Prefill as consecutive segments of seg_t tokens per sequence with one reused
    workspace (sized by seg_t; two segment slots when overlapped, so that a segment's
    per-chunk preparation runs on a side stream during the previous segment's sequential
    pass). Returns (out, state_out)."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    ov = int(bool(overlapped))
    if workspace is None:
        need = _load().gdn_prefill_segmented_workspace_bytes(ctypes.byref(dims), int(seg_t), ov)
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    wbytes = _check_workspace(workspace, q.device)
    _check(_load().gdn_prefill_segmented(
        ctypes.byref(dims), int(seg_t), ov, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state_in), _ptr(out), _ptr(state_out), _ptr(workspace), wbytes,
        _stream(q.device, stream)), "gdn_prefill_segmented")
    return out, state_out


def gdn_noalloc_scratch_bytes() -> int:
    """Size of the library's static per-GPU workspace used by gdn_prefill_segmented_noalloc."""
    return int(_load().gdn_noalloc_scratch_bytes())


def gdn_prefill_segmented_noalloc(q, k, v, g, beta, state_in=None, *, seg_t, l2_eps=1e-6,
                                  out, state_out, stream=None):
    """gdn_prefill_segmented (in order) with the library's static workspace instead of a
    caller's: the library allocates nothing. The caller passes the outputs. Returns
    (out, state_out)."""
    dims, out, state_out = _prepare(q, k, v, g, beta, state_in, out, state_out, l2_eps)
    _check(_load().gdn_prefill_segmented_noalloc(
        ctypes.byref(dims), int(seg_t), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state_in), _ptr(out), _ptr(state_out), _stream(q.device, stream)),
        "gdn_prefill_segmented_noalloc")
    return out, state_out


class DecodeGraph:
    """gdn_decode_graph_create / gdn_graph_launch / gdn_graph_destroy: one decode token
    through len(q) stacked layers as dependent per-layer steps, recorded once as a HIP
    graph. Each layer's inputs are [n, 1, ...] tensors as for gdn_decode_step; its state
    (state[i]) is updated in place and its output written to out[i] (allocated when not
    given). The tensors are referenced by address: write each token's inputs into them in
    place and call launch(). `stream` (a non-default torch stream) is used only to record.
    """

    def __init__(self, q, k, v, g, beta, state, out=None, *, l2_eps=1e-6, stream):
        layers = len(q)
        if not all(len(x) == layers for x in (k, v, g, beta, state)):
            raise ValueError("one tensor per layer in every list")
        if out is None:
            out = [torch.empty(v[i].shape, device=v[i].device, dtype=torch.float32)
                   for i in range(layers)]
        for i in range(layers):
            _prepare(q[i], k[i], v[i], g[i], beta[i], state[i], out[i], state[i], l2_eps)
            # one gdn_dims describes every layer: each layer must match layer 0 exactly
            if (q[i].shape != q[0].shape or v[i].shape != v[0].shape
                    or q[i].dtype != q[0].dtype or q[i].device != q[0].device):
                raise ValueError(f"layer {i}: q/v shapes, dtype and device must equal layer 0's")
        self.tensors = (list(q), list(k), list(v), list(g), list(beta), list(state), list(out))
        self.out = self.tensors[6]
        dims = _dims_of(q[0], v[0], l2_eps) if layers else make_dims(0, 1, 1, 1, 16)
        arr = lambda xs: (ctypes.c_void_p * max(1, layers))(*[x.data_ptr() for x in xs])
        self._arrays = [arr(xs) for xs in self.tensors]
        handle = ctypes.c_void_p()
        _check(_load().gdn_decode_graph_create(
            ctypes.byref(dims), layers, *[ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p)) for a in self._arrays],
            ctypes.c_void_p(stream.cuda_stream), ctypes.byref(handle)), "gdn_decode_graph_create")
        self._handle = handle

    def launch(self, stream=None):
        dev = self.tensors[0][0].device if self.tensors[0] else None
        _check(_load().gdn_graph_launch(self._handle, _stream(dev, stream)), "gdn_graph_launch")

    def close(self):
        if getattr(self, "_handle", None) is not None and self._handle.value:
            _check(_load().gdn_graph_destroy(self._handle), "gdn_graph_destroy")
        self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- attention layers

# These calls are short (a few microseconds of GPU work at a decode step), so their checks are
# written to cost little: a tensor's pointer comes out of the same function that checks it.

_POOLS = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float8_e4m3fn: GDN_FP8}
_Tensor, _i32, _u8 = torch.Tensor, torch.int32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


def _bad(name, x, what):
    """Why x is not `what`."""
    if not isinstance(x, _Tensor):
        raise ValueError(f"{name} must be a torch tensor: {what}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor: {what}")
    raise ValueError(f"{name} must be {what}; got {x.dtype} {tuple(x.shape)}, strides {x.stride()}, on {x.device}")


def _rows(name, x, dtype, index):
    """(pointer, token stride, head stride) of a [tokens, heads, d] tensor with contiguous d on the
    GPU of this index. The stride of a dimension of one entry means nothing to torch: one that every
    layout of the other dimension allows stands for it."""
    if not isinstance(x, _Tensor) or x.dtype != dtype or x.dim() != 3 or x.get_device() != index:
        _bad(name, x, f"{dtype} [tokens, heads, d] on GPU {index}")
    st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    t, h, d = x.shape
    if h == 1:
        sh = d
    if t <= 1:
        st = d
    return x.data_ptr(), st, sh


def _dense(name, x, shape, dtype, index):
    """Pointer of a contiguous tensor of this shape and dtype on the GPU of this index."""
    if not isinstance(x, _Tensor) or x.dtype != dtype or x.shape != shape or x.get_device() != index \
            or not x.is_contiguous():
        _bad(name, x, f"contiguous {dtype} {tuple(shape)} on GPU {index}")
    return x.data_ptr()


def _index(name, x, shape, index):
    """Pointer of an int32 tensor, or None."""
    return None if x is None else _dense(name, x, shape, _i32, index)


def _cache_of(k_cache, v_cache, page_table, k_scale, v_scale):
    """(gdn_kv_cache, GPU index, [h_kv, d]) of the pools and the page table."""
    store = _POOLS.get(k_cache.dtype) if isinstance(k_cache, _Tensor) else None
    if store is None or k_cache.dim() != 4 or not k_cache.is_contiguous() or not k_cache.is_cuda:
        _bad("k_cache", k_cache, "contiguous bfloat16, float32 or float8_e4m3fn [num_pages, h_kv, page_size, d]")
    index, shape = k_cache.get_device(), k_cache.shape
    pages, h, size, d = shape
    v = _dense("v_cache", v_cache, shape, k_cache.dtype, index)
    ks = vs = None
    if store == GDN_FP8:
        ks = _dense("k_scale", k_scale, shape[:3], _u8, index)
        vs = _dense("v_scale", v_scale, shape[:3], _u8, index)
    if not isinstance(page_table, _Tensor) or page_table.dtype != _i32 or page_table.dim() != 2 \
            or page_table.get_device() != index or not page_table.is_contiguous():
        _bad("page_table", page_table, f"contiguous int32 [n, max_pages] on GPU {index}")
    n, width = page_table.shape
    return KvCache(n, pages, width, size, h, d, store, k_cache.data_ptr(), v, ks, vs, page_table.data_ptr()), index


def _queue(index, stream):
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, index, stream):
    """A new tensor that the call's stream may write and the current one read: the allocator gives
    memory out again in the order of the stream it was allocated on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    with torch.cuda.stream(stream):
        x = torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    x.record_stream(torch.cuda.current_stream(index))
    return x


def _gpu(x):
    """Index of x's GPU; a tensor elsewhere gives -1, which no other tensor's matches."""
    return x.get_device() if isinstance(x, _Tensor) and x.is_cuda else -2


def _dtype_id(x):
    t = _DTYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if t is None:
        raise ValueError("tensors of rows must be bfloat16 or float32")
    return t


def gdn_kv_write(k, v, k_cache, v_cache, page_table, start, cu_seqlens=None, *, k_scale=None,
                 v_scale=None, stream=None):
    """Write new tokens into a paged cache, quantised as they are written.

    k, v [total, h_kv, d] (bfloat16 or float32; tokens and heads may be strided): the new tokens
    of n sequences, packed; sequence s has rows cu_seqlens[s] to cu_seqlens[s + 1] - 1
    (cu_seqlens int32 [n + 1]; None: one token per sequence) and its row i goes to position
    start[s] + i (start int32 [n]). k_cache, v_cache [num_pages, h_kv, page_size, d]: of k's
    dtype, or float8_e4m3fn with k_scale, v_scale uint8 [num_pages, h_kv, page_size].
    page_table int32 [n, max_pages]; a page id of -1 is a page that is not there, and what
    would go there is dropped. Updates the cache in place; returns nothing."""
    t = _dtype_id(k)
    c, gpu = _cache_of(k_cache, v_cache, page_table, k_scale, v_scale)
    kp, kt, kh = _rows("k", k, k.dtype, gpu)
    vp, vt, vh = _rows("v", v, k.dtype, gpu)
    total = k.shape[0]
    if k.shape[1:] != (c.h_kv, c.d) or v.shape != k.shape:
        raise ValueError(f"k and v must have shape {(total, c.h_kv, c.d)}")
    sp = _index("start", start, (c.n,), gpu)
    cp = _index("cu_seqlens", cu_seqlens, (c.n + 1,), gpu)
    st = _load().gdn_kv_write(ctypes.byref(c), total, t, kp, kt, kh, vp, vt, vh, sp, cp,
                              _queue(gpu, stream))
    if st:
        raise GdnError(st, "gdn_kv_write")


def gdn_kv_read(k_cache, v_cache, page_table, start, cu_seqlens, total, *, dtype=torch.bfloat16,
                k_scale=None, v_scale=None, k_out=None, v_out=None, stream=None):
    """Read tokens back from a paged cache, packed: position start[s] + i of sequence s becomes
    row cu_seqlens[s] + i of the returned k, v [total, h_kv, d] (of dtype; zeros from pages that
    are not there). total is the packed length, cu_seqlens[n], which the host has to know
    (cu_seqlens None: one token per sequence). Arguments as for gdn_kv_write."""
    t = _DTYPES.get(dtype)
    if t is None:
        raise ValueError("dtype must be bfloat16 or float32")
    c, gpu = _cache_of(k_cache, v_cache, page_table, k_scale, v_scale)
    shape = (int(total), c.h_kv, c.d)
    if k_out is None:
        k_out = _empty(shape, dtype, gpu, stream)
    if v_out is None:
        v_out = torch.empty_like(k_out) if stream is None else _empty(shape, dtype, gpu, stream)
    st = _load().gdn_kv_read(
        ctypes.byref(c), shape[0], t, _dense("k_out", k_out, shape, dtype, gpu),
        _dense("v_out", v_out, shape, dtype, gpu), _index("start", start, (c.n,), gpu),
        _index("cu_seqlens", cu_seqlens, (c.n + 1,), gpu), _queue(gpu, stream))
    if st:
        raise GdnError(st, "gdn_kv_read")
    return k_out, v_out


def gdn_attn_prefill_workspace_bytes(n, total_q, total_k, h_q, h_kv, d, dtype=torch.bfloat16) -> int:
    """Workspace bytes of gdn_attn_prefill for these sizes."""
    t = _DTYPES.get(dtype, -1)
    dims = AttnDims(n, total_q, total_k, h_q, h_kv, d, t, 1, 1.0, h_q * d, d, h_kv * d, d, h_kv * d, d)
    return int(_load().gdn_attn_prefill_workspace_bytes(ctypes.byref(dims)))


def gdn_attn_prefill(q, k, v, cu_q, cu_k=None, *, causal=True, scale=None, out=None, lse=None,
                     workspace=None, stream=None):
    """Attention over packed prompts, with grouped heads.

    q [total_q, h_q, d], k and v [total_k, h_kv, d] (bfloat16 or float32; tokens and heads may be
    strided); cu_q, cu_k int32 [n + 1]: sequence s has query rows cu_q[s] to cu_q[s + 1] - 1 and
    key rows cu_k[s] to cu_k[s + 1] - 1 (cu_k None: the same). With causal, a sequence's last
    query sees its last key, so a segment of new tokens may follow a context. scale defaults to
    1 / sqrt(d). Rows that see no key give 0. Pass lse (float32 [total_q, h_q]) to have the
    logarithm of each row's sum written to it; workspace: uint8, used where few rows meet many
    keys (allocated if not given). Returns out [total_q, h_q, d] of q's dtype."""
    t = _dtype_id(q)
    gpu = _gpu(q)
    qp, qt, qh = _rows("q", q, q.dtype, gpu)
    kp, kt, kh = _rows("k", k, q.dtype, gpu)
    vp, vt, vh = _rows("v", v, q.dtype, gpu)
    tq, hq, d = q.shape
    tk, hk, _ = k.shape
    if k.shape[2] != d or v.shape != k.shape:
        raise ValueError(f"k and v must have the same shape [tokens, heads, {d}]")
    n = cu_q.shape[0] - 1 if isinstance(cu_q, torch.Tensor) and cu_q.dim() == 1 else -1
    if n < 0:
        raise ValueError("cu_q must be an int32 tensor [n + 1]")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None \
            else _empty(q.shape, q.dtype, gpu, stream)
        op = out.data_ptr()
    else:
        op = _dense("out", out, (tq, hq, d), q.dtype, gpu)
    lp = None if lse is None else _dense("lse", lse, (tq, hq), torch.float32, gpu)
    dims = AttnDims(n, tq, tk, hq, hk, d, t, 1 if causal else 0, d ** -0.5 if scale is None else scale,
                    qt, qh, kt, kh, vt, vh)
    lib = _load()
    if workspace is None:
        need = lib.gdn_attn_prefill_workspace_bytes(ctypes.byref(dims))
        if need:
            workspace = _empty(need, _u8, gpu, stream)
    wbytes = 0 if workspace is None else _check_workspace(workspace, q.device)
    st = lib.gdn_attn_prefill(ctypes.byref(dims), qp, kp, vp, _index("cu_q", cu_q, (n + 1,), gpu),
                              _index("cu_k", cu_k, (n + 1,), gpu), op, lp,
                              None if workspace is None else workspace.data_ptr(), wbytes, _queue(gpu, stream))
    if st:
        raise GdnError(st, "gdn_attn_prefill")
    return out


def gdn_attn_decode_workspace_bytes(n, max_pages, page_size, h_q, h_kv, d, max_len,
                                    store=torch.bfloat16) -> int:
    """Workspace bytes of gdn_attn_decode for these sizes."""
    c = KvCache(n, 0, max_pages, page_size, h_kv, d, _POOLS.get(store, -1))
    return int(_load().gdn_attn_decode_workspace_bytes(ctypes.byref(c), h_q, max_len))


def gdn_attn_decode(q, k_cache, v_cache, page_table, lens, *, max_len=None, k_scale=None,
                    v_scale=None, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence over a paged cache (a long one is split, which takes a
    workspace: uint8, allocated if not given).

    q [n, h_q, d] (bfloat16 or float32; tokens and heads may be strided): row s attends to
    positions 0 to lens[s] - 1 of sequence s (lens int32 [n]; the new token's own position,
    written before by gdn_kv_write, is one of them). max_len is a bound on lens that the host
    knows (default: what the page table can hold); positions from it on are not read. The cache
    as for gdn_kv_write. scale defaults to 1 / sqrt(d); lse as for gdn_attn_prefill, [n, h_q].
    Returns out [n, h_q, d] of q's dtype."""
    t = _dtype_id(q)
    c, gpu = _cache_of(k_cache, v_cache, page_table, k_scale, v_scale)
    qp, qt, qh = _rows("q", q, q.dtype, gpu)
    n, hq, d = q.shape
    if n != c.n or d != c.d:
        raise ValueError(f"q must have shape [{c.n}, h_q, {c.d}]")
    if max_len is None:
        max_len = c.max_pages * c.page_size
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None \
            else _empty(q.shape, q.dtype, gpu, stream)
        op = out.data_ptr()
    else:
        op = _dense("out", out, (n, hq, d), q.dtype, gpu)
    lp = None if lse is None else _dense("lse", lse, (n, hq), torch.float32, gpu)
    lib = _load()
    if workspace is None:
        need = lib.gdn_attn_decode_workspace_bytes(ctypes.byref(c), hq, max_len)
        if need:
            workspace = _empty(need, _u8, gpu, stream)
    wbytes = 0 if workspace is None else _check_workspace(workspace, q.device)
    st = lib.gdn_attn_decode(
        ctypes.byref(c), hq, t, d ** -0.5 if scale is None else scale, max_len, qp, qt, qh,
        _index("lens", lens, (n,), gpu), op, lp, None if workspace is None else workspace.data_ptr(),
        wbytes, _queue(gpu, stream))
    if st:
        raise GdnError(st, "gdn_attn_decode")
    return out


# ---------------------------------------------------------------- around the attention layers

def _new(x, index, stream):
    """An output of x's shape and type, dense, for a call on `stream`."""
    return torch.empty_like(x, memory_format=_dense_format) if stream is None else _empty(x.shape, x.dtype, index, stream)


_dense_format, _f32 = torch.contiguous_format, torch.float32
_this_gpu = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _launch(name, call, index, stream):
    """Enqueue call(stream handle) with the tensors' GPU as the current one, as the library expects it."""
    if stream is None:
        queue = _raw_stream(index)
    elif stream.device_index == index:
        queue = stream.cuda_stream
    else:
        raise ValueError(f"stream must be one of GPU {index}")
    if _this_gpu() == index:
        st = call(queue)
    else:
        with torch.cuda.device(index):
            st = call(queue)
    if st:
        raise GdnError(st, name)


def _norm_rope(total, d, dtype, index, positions, freq, axis, interleaved, rope_scale, q_weight, k_weight,
               weight_bias, eps, placed):
    """gdn_norm_rope of these tensors; placed: without positions a token turns by its place."""
    rot, axes, fp, ap, pp = 0, 1, None, None, None
    if freq is not None:
        if not isinstance(freq, _Tensor) or freq.dim() != 1:
            raise ValueError("freq must be a float32 tensor [rot / 2]")
        half = freq.shape
        rot = 2 * half[0]
        fp = _dense("freq", freq, half, _f32, index)
        if axis is not None:
            ap = _dense("axis", axis, half, _u8, index)
        if positions is not None:
            shape = positions.shape if isinstance(positions, _Tensor) else ()
            if len(shape) == 2:
                axes = shape[0]
            if len(shape) not in (1, 2) or shape[-1] != total:
                _bad("positions", positions, f"int32 [{total}] or [axes, {total}] on GPU {index}")
            pp = _dense("positions", positions, shape, _i32, index)
        elif not placed:
            raise ValueError("positions are needed with freq")
    elif positions is not None or axis is not None:
        raise ValueError("positions and axis need freq")
    qw = None if q_weight is None else _dense("q_weight", q_weight, (d,), dtype, index)
    kw = None if k_weight is None else _dense("k_weight", k_weight, (d,), dtype, index)
    return NormRope(eps, weight_bias, qw, kw, rot, 1 if interleaved else 0, axes, rope_scale, fp, ap, pp)


def gdn_qk_norm_rope(q, k=None, positions=None, *, freq=None, axis=None, interleaved=False, rope_scale=1.0,
                     q_weight=None, k_weight=None, weight_bias=0.0, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head, and their rotary positions, in one pass.

    q [total, h_q, d] and k [total, h_kv, d] (bfloat16 or float32; tokens and heads may be strided; k
    may be None). With q_weight (k_weight) [d], of q's dtype, each row is divided by the root of its
    mean square plus eps and multiplied by weight_bias + weight. With freq (float32 [rot / 2], rot a
    multiple of 16) the first rot elements are then turned, pair p by the angle freq[p] * position and
    times rope_scale: elements p and p + rot / 2, or with interleaved 2 p and 2 p + 1. positions: int32
    [total], or [axes, total] with axis (uint8 [rot / 2]) the axis of each pair. Computed in fp32,
    angles in 64 bits, rounded once. Returns (q_out, k_out), dense, of q's dtype (k_out None
    without k)."""
    t = _dtype_id(q)
    gpu = _gpu(q)
    qp, qt, qh = _rows("q", q, q.dtype, gpu)
    total, hq, d = q.shape
    kp, kt, kh, hk, kop = None, 0, 0, 0, None
    if k is not None:
        kp, kt, kh = _rows("k", k, q.dtype, gpu)
        hk = k.shape[1]
        if k.shape[0] != total or k.shape[2] != d:
            raise ValueError(f"k must have shape [{total}, h_kv, {d}]")
    elif k_out is not None:
        raise ValueError("k_out needs k")
    f = _norm_rope(total, d, q.dtype, gpu, positions, freq, axis, interleaved, rope_scale, q_weight, k_weight,
                   weight_bias, eps, False)
    if q_out is None:
        q_out = _new(q, gpu, stream)
        qop = q_out.data_ptr()
    else:
        qop = _dense("q_out", q_out, q.shape, q.dtype, gpu)
    if k is not None:
        if k_out is None:
            k_out = _new(k, gpu, stream)
            kop = k_out.data_ptr()
        else:
            kop = _dense("k_out", k_out, k.shape, q.dtype, gpu)
    lib = _load()
    _launch("gdn_qk_norm_rope", lambda queue: lib.gdn_qk_norm_rope(
        ctypes.byref(f), total, hq, hk, d, t, qp, qt, qh, kp, kt, kh, qop, kop, queue), gpu, stream)
    return q_out, k_out


def gdn_kv_append(k, v, k_cache, v_cache, page_table, start, cu_seqlens=None, *, positions=None, freq=None, axis=None,
                  interleaved=False, rope_scale=1.0, k_weight=None, q=None, q_weight=None, weight_bias=0.0, eps=1e-6,
                  q_out=None, k_scale=None, v_scale=None, stream=None):
    """Write new tokens into a paged cache, their keys normed and rotated on the way, and their queries
    too: what an attention layer does between its projections and its attention, in one launch.

    k, v, the cache, start and cu_seqlens as for gdn_kv_write; weights, freq, positions and the rest as
    for gdn_qk_norm_rope, but that without positions a token turns by its place in its sequence,
    start[s] + i. q [total, h_q, d] (may be strided, and None) is normed and rotated into q_out
    (dense), which is returned (None without q); rows of no sequence are left as they are there."""
    t = _dtype_id(k)
    c, gpu = _cache_of(k_cache, v_cache, page_table, k_scale, v_scale)
    kp, kt, kh = _rows("k", k, k.dtype, gpu)
    vp, vt, vh = _rows("v", v, k.dtype, gpu)
    total = k.shape[0]
    if k.shape[1:] != (c.h_kv, c.d) or v.shape != k.shape:
        raise ValueError(f"k and v must have shape {(total, c.h_kv, c.d)}")
    sp = _index("start", start, (c.n,), gpu)
    cp = _index("cu_seqlens", cu_seqlens, (c.n + 1,), gpu)
    f = _norm_rope(total, c.d, k.dtype, gpu, positions, freq, axis, interleaved, rope_scale, q_weight, k_weight,
                   weight_bias, eps, True)
    qp, qt, qh, hq, qop = None, 0, 0, 0, None
    if q is not None:
        qp, qt, qh = _rows("q", q, k.dtype, gpu)
        hq = q.shape[1]
        if q.shape[0] != total or q.shape[2] != c.d:
            raise ValueError(f"q must have shape [{total}, h_q, {c.d}]")
        if q_out is None:
            q_out = _new(q, gpu, stream)
            qop = q_out.data_ptr()
        else:
            qop = _dense("q_out", q_out, q.shape, k.dtype, gpu)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    lib = _load()
    _launch("gdn_kv_append", lambda queue: lib.gdn_kv_append(
        ctypes.byref(c), ctypes.byref(f), total, t, kp, kt, kh, vp, vt, vh, sp, cp, hq, qp, qt, qh, qop, queue),
        gpu, stream)
    return q_out


def gdn_attn_extend_workspace_bytes(n, max_pages, page_size, total_q, h_q, h_kv, d, *, max_q=None, max_len=None, window=0,
                                    sinks=0, dtype=torch.bfloat16, store=None) -> int:
    """Workspace bytes of gdn_attn_extend for these sizes (max_q, max_len as there; store: the cache's
    dtype if not dtype)."""
    store = dtype if store is None else store
    c = KvCache(n, 1, max_pages, page_size, h_kv, d, _POOLS.get(store, -1))
    dims = ExtendDims(total_q, total_q if max_q is None else max_q, max_pages * page_size if max_len is None else max_len,
                      window, sinks, h_q, _DTYPES.get(dtype, -1), 1.0, h_q * d, d)
    return int(_load().gdn_attn_extend_workspace_bytes(ctypes.byref(c), ctypes.byref(dims)))


def gdn_attn_extend(q, k_cache, v_cache, page_table, lens, cu_q=None, *, window=0, sinks=0, max_q=None, max_len=None,
                    k_scale=None, v_scale=None, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache that holds them already: the next piece of a prompt,
    a few drafted tokens, or one token per sequence (cu_q None).

    q [total, h_q, d] (bfloat16 or float32; tokens and heads may be strided): sequence s has rows
    cu_q[s] to cu_q[s + 1] - 1 (int32 [n + 1]), the last of which is the token at position
    lens[s] - 1 (int32 [n]; the new tokens, written before, are counted). A row sees the positions up
    to its own; with window > 0 only the last `window` of them, and the first `sinks` of the sequence.
    max_q and max_len are bounds on a sequence's rows and length that the host knows (default: total
    and what the page table can hold; tight ones divide the work better): rows from max_q on are not
    computed, positions from max_len on not read. The cache as for gdn_kv_write, lse and workspace
    as for gdn_attn_prefill, scale defaults to 1 / sqrt(d). Returns out [total, h_q, d] of q's dtype."""
    t = _dtype_id(q)
    c, gpu = _cache_of(k_cache, v_cache, page_table, k_scale, v_scale)
    qp, qt, qh = _rows("q", q, q.dtype, gpu)
    total, hq, d = q.shape
    if d != c.d:
        raise ValueError(f"q must have shape [total, h_q, {c.d}]")
    if cu_q is None and total != c.n:
        raise ValueError(f"without cu_q, q must have one row per sequence, {c.n}")
    if max_q is None:
        max_q = total if cu_q is not None else 1
    if max_len is None:
        max_len = c.max_pages * c.page_size
    if out is None:
        out = _new(q, gpu, stream)
        op = out.data_ptr()
    else:
        op = _dense("out", out, q.shape, q.dtype, gpu)
    lp = None if lse is None else _dense("lse", lse, (total, hq), _f32, gpu)
    dims = ExtendDims(total, max_q if cu_q is not None else min(max_q, 1), max_len, window, sinks, hq, t,
                      d ** -0.5 if scale is None else scale, qt, qh)
    lib = _load()
    if workspace is None:
        need = lib.gdn_attn_extend_workspace_bytes(ctypes.byref(c), ctypes.byref(dims))
        if need:
            workspace = _empty(need, _u8, gpu, stream)
    wbytes = 0 if workspace is None else _check_workspace(workspace, q.device)
    cp, np = _index("cu_q", cu_q, (c.n + 1,), gpu), _index("lens", lens, (c.n,), gpu)
    wp = None if workspace is None else workspace.data_ptr()
    _launch("gdn_attn_extend", lambda queue: lib.gdn_attn_extend(
        ctypes.byref(c), ctypes.byref(dims), qp, cp, np, op, lp, wp, wbytes, queue), gpu, stream)
    return out
