"""norm_rope_cache_amd: the DSpark draft's context K/V chain on MI355X (gfx950).

A thin ctypes binding over libnrc.so (include/nrc.h). Each function checks
torch tensor dtypes/shapes, passes raw device pointers and the current HIP
stream, and raises NrcError on a non-zero status. Every step of the chain
runs in the library's HIP kernels; there is no CPU or PyTorch fallback: if
libnrc.so is missing, every call raises.

    context_norms(x, hidden_w, pre_w, L, ...)      -> [L, T, 8192] bf16
    context_norms_ex(...)                          the same with FP32 / input-scaled weights
    context_kv_project(normed, w_kv)               -> [L, T, N] bf16 ([L, D, N] or [L, N, D] weights)
    context_kv_store(kv, positions, slots, cos_sin, caches, H, ...)   (in place)
    context_kv_store_ex(...)                       per-layer slot lists, strided cache views
    context_hidden_norm(x, ...) -> (h, r)          pre-pass of the fused path
    context_kv_project_fused(h, r, pre_w, w_kv)    projection with the layer norms fused in
    context_kv_chain(...)                          the whole chain (unfused by default)
    draft_boundary(branch, stream_in, alpha, beta, ...)   the residual boundary

and the operators that use the cache the chain fills:

    rope_table(count, rotary_dim, ...)             the cos/sin table, also for stretched contexts
    rope_rotate(x, positions, cos_sin, ...)        query heads, or their gradients, rotated by it
    context_tree_attention(q, cache, tables, ...)  drafted tokens attending to the cache -> (out, lse)
    context_attention_mass(q, cache, tables, ..., lse, ...)   the weight each cached cell receives
    context_kv_evict(cache, tables, lens, weights, ...)       the cells of most weight kept (in place)

Of these rope_rotate records a gradient; the others' outputs carry no graph.
"""

import ctypes
import os

__all__ = [
    "NrcError",
    "context_norms",
    "context_norms_ex",
    "context_kv_project",
    "context_kv_store",
    "context_kv_store_ex",
    "draft_boundary",
    "context_kv_chain",
    "context_hidden_norm",
    "context_kv_project_fused",
    "context_kv_project_noalloc",
    "rope_table",
    "rope_rotate",
    "context_tree_attention",
    "context_attention_mass",
    "context_kv_evict",
    "kv_views",
    "check_scalars",
    "check_bf16_pair",
    "library_path",
    "abi_version",
]

HIDDEN = 8192
HEAD_DIM = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libnrc.so")
_lib = None

_torch = None  # the module, once a call has needed it (importing the package does not)


def _get_torch():
    global _torch
    import torch

    _torch = torch
    return torch


_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float


class NrcError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"libnrc status {code}: {message}")
        self.code = code


def library_path():
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"libnrc.so not built at {_LIB_PATH}: run `python -m norm_rope_cache_amd.build` "
            "(there is no fallback path)")
    L = ctypes.CDLL(_LIB_PATH)
    L.nrc_last_error.restype = ctypes.c_char_p
    L.nrc_last_error.argtypes = []
    L.nrc_abi_version.restype = _i32
    L.nrc_abi_version.argtypes = []
    L.nrc_context_norms.restype = _i32
    L.nrc_context_norms.argtypes = [_vp, _i64, _i64, _vp, _vp, _i32, _f32, _f32, _f32, _f32, _vp, _vp]
    L.nrc_context_norms_ex.restype = _i32
    L.nrc_context_norms_ex.argtypes = [_vp, _i64, _i64, _vp, _i32, _vp, _i32, _i32, _f32, _f32, _f32, _f32,
                                       ctypes.c_uint32, _vp, _vp]
    L.nrc_context_kv_store_ex.restype = _i32
    L.nrc_context_kv_store_ex.argtypes = [_vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp,
                                          _i64, _i64, _i64, _i64, _i64, _i32, _i32, _f32, _vp]
    L.nrc_context_kv_project_ex.restype = _i32
    L.nrc_context_kv_project_ex.argtypes = [_vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp]
    L.nrc_draft_boundary.restype = _i32
    L.nrc_draft_boundary.argtypes = [_vp, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _f32, _f32, _f32,
                                     _f32, ctypes.c_uint32, _vp, _vp, _vp]
    L.nrc_context_kv_project.restype = _i32
    L.nrc_context_kv_project.argtypes = [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp]
    L.nrc_context_kv_project_workspace_bytes.restype = _i64
    L.nrc_context_kv_project_workspace_bytes.argtypes = [_i32, _i64, _i64, _i64]
    L.nrc_context_kv_project_split.restype = _i32
    L.nrc_context_kv_project_split.argtypes = [_vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp]
    L.nrc_context_kv_project_noalloc.restype = _i32
    L.nrc_context_kv_project_noalloc.argtypes = [_vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp]
    L.nrc_context_kv_project_timed.restype = _i32
    L.nrc_context_kv_project_timed.argtypes = [_vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _vp,
                                               _vp]
    L.nrc_context_kv_store.restype = _i32
    L.nrc_context_kv_store.argtypes = [
        _vp, _vp, _i64, _i64, _i64, _i64, _vp, ctypes.POINTER(_vp), _i64, _i64, _vp, _i64,
        ctypes.POINTER(_vp), _i64, _i64, _i32, _i32, _f32, _vp]
    L.nrc_context_kv_project_store.restype = _i32
    L.nrc_context_kv_project_store.argtypes = [
        _vp, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, ctypes.POINTER(_vp), _i64, _vp, _i64,
        ctypes.POINTER(_vp), _i64, _i64, _f32, _vp]
    L.nrc_context_hidden_norm.restype = _i32
    L.nrc_context_hidden_norm.argtypes = [_vp, _i64, _i64, _vp, _vp, _i32, _f32, _f32, _f32, _f32, _vp, _vp, _vp]
    L.nrc_context_kv_project_fused.restype = _i32
    L.nrc_context_kv_project_fused.argtypes = [_vp, _vp, _vp, _f32, _vp, _vp, _i32, _i64, _i64, _i64, _vp]
    L.nrc_context_kv_project_fused_split.restype = _i32
    L.nrc_context_kv_project_fused_split.argtypes = [_vp, _vp, _vp, _f32, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i64,
                                                     _vp]
    L.nrc_check_scalars.restype = _i32
    L.nrc_check_scalars.argtypes = [_vp, _vp, _vp, _i64, _vp]
    L.nrc_traffic_twin.restype = _i32
    L.nrc_traffic_twin.argtypes = [_vp, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _vp]
    L.nrc_check_bf16_pair.restype = _i32
    L.nrc_check_bf16_pair.argtypes = [_vp, _vp, _i64, _vp]
    f64 = ctypes.c_double
    L.nrc_rope_table.restype = _i32
    L.nrc_rope_table.argtypes = [_i64, _i64, _i32, _i32, f64, _i32, f64, f64, f64, f64, f64, _vp, _i32, _vp]
    L.nrc_rope_rotate.restype = _i32
    L.nrc_rope_rotate.argtypes = [_vp, _i32, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _vp,
                                  _i64, _i64, _vp]
    L.nrc_rope_rotate_ex.restype = _i32
    L.nrc_rope_rotate_ex.argtypes = L.nrc_rope_rotate.argtypes[:-1] + [ctypes.c_uint32, _vp]
    paged = [_vp, _i64, _i64, _i64, _i64, _i64, _i32, _vp, _i64, _i64, _i32]
    queries = [_vp, _i64, _i64, _i64, _i32] + paged + [_vp, _vp, _i32, _i64, _vp, _i32, _f32, _f32]
    L.nrc_context_tree_attention.restype = _i32
    L.nrc_context_tree_attention.argtypes = queries + [_vp, _vp, _vp, _i64, _vp]
    L.nrc_context_tree_attention_ex.restype = _i32
    L.nrc_context_tree_attention_ex.argtypes = L.nrc_context_tree_attention.argtypes[:-1] + [ctypes.c_uint32, _vp]
    L.nrc_context_tree_attention_workspace_bytes.restype = _i64
    L.nrc_context_tree_attention_workspace_bytes.argtypes = [_i32, _i64, _i32, _i32, _i32, _i64]
    L.nrc_context_attention_mass.restype = _i32
    L.nrc_context_attention_mass.argtypes = queries + [_vp, _vp, _i64, _i64, _f32, _vp, _i64, _i64, _i64, _vp]
    L.nrc_context_kv_evict.restype = _i32
    L.nrc_context_kv_evict.argtypes = paged + [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i32, _i32, _i32, _vp,
                                               _vp, _vp, _vp, _i64, _vp]
    L.nrc_context_kv_evict_workspace_bytes.restype = _i64
    L.nrc_context_kv_evict_workspace_bytes.argtypes = [_i32, _i32, _i64, _i32]
    _lib = L
    return L


def abi_version():
    return int(_load().nrc_abi_version())


def _check(code):
    if code != 0:
        msg = _load().nrc_last_error().decode(errors="replace")
        raise NrcError(code, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, ref):
    """The HIP stream for a call on ref's GPU: the given torch stream, which
    must belong to that GPU, or that GPU's current stream."""
    torch = _torch or _get_torch()
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(ref.get_device())  # the handle alone, without a stream object
    if stream.device != ref.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {ref.device}")
    return stream.cuda_stream


def _call(ref, fn, *args):
    """One C-ABI call with ref's GPU as the current device (the library sizes
    its launches and finds its scratch on the current device), raising
    NrcError on a non-zero status."""
    torch = _torch or _get_torch()
    dev = ref.get_device()
    if dev >= 0 and dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            code = fn(*args)
    else:
        code = fn(*args)
    if code != 0:
        _check(code)


def _all_on(ref, **tensors):
    """_same_device for every operand given (None: absent)."""
    for name, t in tensors.items():
        if t is not None:
            _same_device(t, ref, name)


def _bf16(t, name, contiguous=True):
    import torch

    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _same_device(t, ref, name):
    """Raise unless t is a tensor on ref's GPU: a host pointer handed to a
    kernel would fault the device instead of failing."""
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != ref.device:
        where = "not a tensor" if not isinstance(t, torch.Tensor) else str(t.device)
        raise ValueError(f"{name} must be a tensor on {ref.device} ({where})")
    return t


def context_norms(x, hidden_w, pre_w, L, hidden_eps=1e-6, pre_eps=1e-6, hidden_center=0.0, pre_center=0.0,
                  out=None, stream=None):
    """stack([pre_norm_l(hidden_norm(x)) for l]): x [T, 8192] bf16 ->
    [L, T, 8192] bf16 (written into `out` when given)."""
    import torch

    _bf16(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, 8192]")
    T, D = x.shape
    if hidden_w is not None:
        _bf16(hidden_w, "hidden_w")
        if tuple(hidden_w.shape) != (D,):
            raise ValueError("hidden_w must be [D]")
    if pre_w is not None:
        _bf16(pre_w, "pre_w")
        if tuple(pre_w.shape) != (L, D):
            raise ValueError("pre_w must be [L, D]")
    if out is None:
        out = torch.empty((L, T, D), dtype=torch.bfloat16, device=x.device)
    else:
        _bf16(out, "out")
        if tuple(out.shape) != (L, T, D):
            raise ValueError("out must be [L, T, D]")
    _all_on(x, hidden_w=hidden_w, pre_w=pre_w, out=out)
    _call(x, _load().nrc_context_norms, _ptr(x), T, D, _ptr(hidden_w), _ptr(pre_w), L, hidden_eps, pre_eps,
          hidden_center, pre_center, _ptr(out), _stream(stream, x))
    return out


WEIGHT_NONE, WEIGHT_BF16, WEIGHT_F32 = 0, 1, 2
HIDDEN_INPUT_SCALE, PRE_INPUT_SCALE = 1, 2


def _weight_kind(w, name, shape):
    import torch

    if w is None:
        return WEIGHT_NONE
    if not w.is_cuda or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")
    if tuple(w.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if w.dtype == torch.bfloat16:
        return WEIGHT_BF16
    if w.dtype == torch.float32:
        return WEIGHT_F32
    raise ValueError(f"{name} must be bf16 or float32, not {w.dtype}")


def context_norms_ex(x, hidden_w, pre_w, L, hidden_eps=1e-6, pre_eps=1e-6, hidden_center=0.0, pre_center=0.0,
                     hidden_input_scale=False, pre_input_scale=False, out=None, stream=None):
    """context_norms with bf16 or float32 weights and, per norm, the weight
    scaling the norm's input instead of its output."""
    import torch

    _bf16(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, 8192]")
    T, D = x.shape
    hk = _weight_kind(hidden_w, "hidden_w", (D,))
    pk = _weight_kind(pre_w, "pre_w", (L, D))
    if out is None:
        out = torch.empty((L, T, D), dtype=torch.bfloat16, device=x.device)
    else:
        _bf16(out, "out")
        if tuple(out.shape) != (L, T, D):
            raise ValueError("out must be [L, T, D]")
    _all_on(x, hidden_w=hidden_w, pre_w=pre_w, out=out)
    flags = (HIDDEN_INPUT_SCALE if hidden_input_scale else 0) | (PRE_INPUT_SCALE if pre_input_scale else 0)
    _call(x, _load().nrc_context_norms_ex, _ptr(x), T, D, _ptr(hidden_w), hk, _ptr(pre_w), pk, L, hidden_eps, pre_eps,
          hidden_center, pre_center, flags, _ptr(out), _stream(stream, x))
    return out


def _boundary_kind(w, name):
    import torch

    if w is None:
        return WEIGHT_NONE
    if not w.is_cuda or not w.is_contiguous() or tuple(w.shape) != (8192,):
        raise ValueError(f"{name} must be a contiguous device tensor of shape [8192]")
    kinds = {torch.bfloat16: WEIGHT_BF16, torch.float32: WEIGHT_F32, torch.float16: 3}
    if w.dtype not in kinds:
        raise ValueError(f"{name} must be bf16, float32 or float16, not {w.dtype}")
    return kinds[w.dtype]


def draft_boundary(branch, stream_in, alpha, beta, post_w=None, pre_w=None, post_eps=1e-6, pre_eps=1e-6,
                   post_center=0.0, pre_center=0.0, post_input_scale=False, pre_input_scale=False,
                   store_stream=True, out=None, stream_out=None, stream=None):
    """One residual boundary: (new FP32 stream or None, bf16 out [m, 8192]).

    branch [m, 8192] bf16; stream_in [m, 8192] float32 or bf16; alpha, beta
    float32 [8192]; post_w / pre_w [8192] bf16, float32 or float16 (None:
    weightless); *_input_scale: that weight scales the norm's input."""
    import torch

    _bf16(branch, "branch")
    if branch.dim() != 2:
        raise ValueError("branch must be [m, 8192]")
    m, D = branch.shape
    if tuple(stream_in.shape) != (m, D) or not stream_in.is_contiguous() or not stream_in.is_cuda:
        raise ValueError("stream_in must be a contiguous device tensor shaped like the branch")
    if stream_in.dtype == torch.float32:
        sk = 0
    elif stream_in.dtype == torch.bfloat16:
        sk = 1
    else:
        raise ValueError("stream_in must be float32 or bf16")
    for g, name in ((alpha, "alpha"), (beta, "beta")):
        if g.dtype != torch.float32 or tuple(g.shape) != (D,) or not g.is_contiguous() or not g.is_cuda:
            raise ValueError(f"{name} must be a contiguous float32 device tensor [8192]")
    pk = _boundary_kind(post_w, "post_w")
    qk = _boundary_kind(pre_w, "pre_w")
    if out is None:
        out = torch.empty((m, D), dtype=torch.bfloat16, device=branch.device)
    else:
        _bf16(out, "out")
        if tuple(out.shape) != (m, D):
            raise ValueError("out must be [m, 8192] like the branch")
    if not store_stream:
        stream_out = None
    elif stream_out is None:
        stream_out = torch.empty((m, D), dtype=torch.float32, device=branch.device)
    elif stream_out.dtype != torch.float32 or tuple(stream_out.shape) != (m, D) or not stream_out.is_contiguous():
        raise ValueError("stream_out must be a contiguous float32 [m, 8192] tensor")
    _all_on(branch, stream_in=stream_in, alpha=alpha, beta=beta, post_w=post_w, pre_w=pre_w, out=out,
            stream_out=stream_out)
    flags = (1 if post_input_scale else 0) | (2 if pre_input_scale else 0)
    _call(branch, _load().nrc_draft_boundary, _ptr(branch), m, D, _ptr(stream_in), sk, _ptr(alpha), _ptr(beta),
          _ptr(post_w), pk, _ptr(pre_w), qk, post_eps, pre_eps, post_center, pre_center, flags, _ptr(stream_out),
          _ptr(out), _stream(stream, branch))
    return stream_out, out


def context_hidden_norm(x, hidden_w, pre_w, L, hidden_eps=1e-6, pre_eps=1e-6, hidden_center=0.0, pre_center=0.0,
                        h=None, r=None, stream=None):
    """Pre-pass of the fused path: (h [T, 8192] bf16, r [T] float32)."""
    import torch

    _bf16(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, 8192]")
    T, D = x.shape
    if hidden_w is not None:
        _bf16(hidden_w, "hidden_w")
        if tuple(hidden_w.shape) != (D,):
            raise ValueError("hidden_w must be [D]")
    if pre_w is not None:
        _bf16(pre_w, "pre_w")
        if tuple(pre_w.shape) != (L, D):
            raise ValueError("pre_w must be [L, D]")
    _all_on(x, hidden_w=hidden_w, pre_w=pre_w)
    if h is None:
        h = torch.empty((T, D), dtype=torch.bfloat16, device=x.device)
    if r is None:
        r = torch.empty((T,), dtype=torch.float32, device=x.device)
    _bf16(h, "h")
    if tuple(h.shape) != (T, D) or r.dtype != torch.float32 or tuple(r.shape) != (T,) or not r.is_contiguous():
        raise ValueError("h must be [T, D] bf16 and r [T] float32")
    _same_device(h, x, "h")
    _same_device(r, x, "r")
    _call(x, _load().nrc_context_hidden_norm, _ptr(x), T, D, _ptr(hidden_w), _ptr(pre_w), L, hidden_eps, pre_eps,
          hidden_center, pre_center, _ptr(h), _ptr(r), _stream(stream, x))
    return h, r


def context_kv_project_fused(h, r, pre_w, w_kv, pre_center=0.0, out=None, stream=None, split=True):
    """kv[l] = bf16((h * |r|) * (pre_w[l] + pre_center)) . w_kv[l]; equal to
    context_norms followed by context_kv_project with the same `split`
    (small T: the summation split over several workgroups, with a workspace
    from torch's allocator; split=False keeps the one-pass kernel)."""
    import torch

    _bf16(h, "h")
    _bf16(w_kv, "w_kv")
    if h.dim() != 2 or w_kv.dim() != 3:
        raise ValueError("h must be [T, D] and w_kv [L, D, N]")
    T, D = h.shape
    L, Dw, N = w_kv.shape
    if Dw != D:
        raise ValueError("w_kv must be [L, D, N]")
    if pre_w is not None:
        _bf16(pre_w, "pre_w")
        if tuple(pre_w.shape) != (L, D):
            raise ValueError("pre_w must be [L, D]")
    if r.dtype != torch.float32 or tuple(r.shape) != (T,) or not r.is_contiguous():
        raise ValueError("r must be a contiguous float32 [T]")
    _same_device(r, h, "r")
    _same_device(w_kv, h, "w_kv")
    if pre_w is not None:
        _same_device(pre_w, h, "pre_w")
    if out is None:
        out = torch.empty((L, T, N), dtype=torch.bfloat16, device=h.device)
    else:
        _bf16(out, "out")
        _same_device(out, h, "out")
        if tuple(out.shape) != (L, T, N):
            raise ValueError("out must be [L, T, N]")
    lib = _load()
    need = lib.nrc_context_kv_project_workspace_bytes(L, T, D, N) if split else 0
    if need < 0:
        _check(need)
    if need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=h.device)
        if stream is not None:
            ws.record_stream(stream)  # the allocator may reuse it only after this stream's work
        _call(h, lib.nrc_context_kv_project_fused_split, _ptr(h), _ptr(r), _ptr(pre_w), pre_center, _ptr(w_kv),
              _ptr(out), L, T, D, N, _ptr(ws), need, _stream(stream, h))
    else:
        _call(h, lib.nrc_context_kv_project_fused, _ptr(h), _ptr(r), _ptr(pre_w), pre_center, _ptr(w_kv), _ptr(out), L,
              T, D, N, _stream(stream, h))
    return out


def _project_operands(normed, w_kv, out, w_layout):
    """Shape checks of the projection; returns L, T, D, N, the layout code and out."""
    import torch

    _bf16(normed, "normed")
    _bf16(w_kv, "w_kv")
    _same_device(w_kv, normed, "w_kv")
    if normed.dim() != 3:
        raise ValueError("normed must be [L, T, D]")
    L, T, D = normed.shape
    if w_layout == "dn":
        if w_kv.dim() != 3 or w_kv.shape[0] != L or w_kv.shape[1] != D:
            raise ValueError("w_kv must be [L, D, N]")
        N = w_kv.shape[2]
    elif w_layout == "nd":
        if w_kv.dim() != 3 or w_kv.shape[0] != L or w_kv.shape[2] != D:
            raise ValueError("w_kv must be [L, N, D]")
        N = w_kv.shape[1]
    else:
        raise ValueError("w_layout is 'dn' or 'nd'")
    if out is None:
        out = torch.empty((L, T, N), dtype=torch.bfloat16, device=normed.device)
    else:
        _bf16(out, "out")
        _same_device(out, normed, "out")
        if tuple(out.shape) != (L, T, N):
            raise ValueError("out must be [L, T, N]")
    return L, T, D, N, (0 if w_layout == "dn" else 1), out


def context_kv_project(normed, w_kv, out=None, stream=None, w_layout="dn", split=True):
    """[L, T, D] x [L, D, N] -> [L, T, N] bf16 (FP32 accumulation).
    w_layout "nd": w_kv is stored [L, N, D] (the pages' storage). split: for
    shapes with too few output tiles to fill the GPU (small T) the summation
    axis is split over several workgroups, with a workspace from torch's
    allocator (split=False keeps the one-pass kernel)."""
    import torch

    L, T, D, N, layout, out = _project_operands(normed, w_kv, out, w_layout)
    lib = _load()
    need = lib.nrc_context_kv_project_workspace_bytes(L, T, D, N) if split else 0
    if need < 0:
        _check(need)
    if need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=normed.device)
        if stream is not None:
            ws.record_stream(stream)  # the allocator may reuse it only after this stream's work
        _call(normed, lib.nrc_context_kv_project_split, _ptr(normed), _ptr(w_kv), layout, _ptr(out), L, T, D, N,
              _ptr(ws), need, _stream(stream, normed))
    elif w_layout == "dn":
        _call(normed, lib.nrc_context_kv_project, _ptr(normed), _ptr(w_kv), _ptr(out), L, T, D, N,
              _stream(stream, normed))
    else:
        _call(normed, lib.nrc_context_kv_project_ex, _ptr(normed), _ptr(w_kv), 1, _ptr(out), L, T, D, N,
              _stream(stream, normed))
    return out


def context_kv_project_noalloc(normed, w_kv, out, stream=None, w_layout="dn"):
    """context_kv_project for callers that cannot allocate: the split form's
    partial sums go to the library's per-GPU scratch (no workspace, no
    allocation by the library or here; `out` is required). Same bits as
    context_kv_project; raises NrcError for a split needing more scratch
    than the library holds. Calls that overlap on one GPU race."""
    if out is None:
        raise ValueError("context_kv_project_noalloc writes into a caller-owned out")
    L, T, D, N, layout, out = _project_operands(normed, w_kv, out, w_layout)
    _call(normed, _load().nrc_context_kv_project_noalloc, _ptr(normed), _ptr(w_kv), layout, _ptr(out), L, T, D, N,
          _stream(stream, normed))
    return out


def context_kv_project_timed(normed, w_kv, out=None, stream=None, w_layout="dn"):
    """The one-pass projection with per-workgroup clock stamps (a diagnostic;
    the call synchronizes the device to read them). Returns (out, clocks):
    clocks holds 'workgroups', 'stamps' (CPU int64 [workgroups, 4]: shader
    clock at start, constant clock at start, shader clock at end, constant
    clock at end), 'wall_khz' (the constant clock's rate) and 'shader_ghz'
    (each workgroup's mean shader clock over its lifetime, GHz)."""
    import ctypes
    import torch

    L, T, D, N, layout, out = _project_operands(normed, w_kv, out, w_layout)
    lib = _load()
    n = 8 * torch.cuda.get_device_properties(normed.device).multi_processor_count
    stamps = torch.zeros(n, dtype=torch.int64, device=normed.device)
    wg, khz = ctypes.c_int32(0), ctypes.c_int32(0)
    _call(normed, lib.nrc_context_kv_project_timed, _ptr(normed), _ptr(w_kv), layout, _ptr(out), L, T, D, N,
          _ptr(stamps), n, ctypes.byref(wg), ctypes.byref(khz), _stream(stream, normed))
    torch.cuda.synchronize(normed.device)
    st = stamps[: 4 * wg.value].view(-1, 4).cpu()
    ds = (st[:, 2] - st[:, 0]).double()
    dr = (st[:, 3] - st[:, 1]).double()
    ghz = (ds / dr * khz.value / 1e6) if wg.value else torch.empty(0, dtype=torch.float64)
    return out, {"workgroups": wg.value, "stamps": st, "wall_khz": khz.value, "shader_ghz": ghz}


def kv_views(kv, H):
    """k, v views [L, T, H, 64] of a projection output [L, T, 2 H 64]."""
    L, T, N = kv.shape
    v5 = kv.view(L, T, 2, H, HEAD_DIM)
    return v5[:, :, 0], v5[:, :, 1]


def _store_operands(kv_ref, L, T, H, positions, slots, cos_sin, caches, rows):
    """Checks of the store's operands against the K/V source kv_ref ([L, T, ...]
    on one device); returns the host pointer arrays and sizes the C ABI takes:
    (slot_arr, cache_arr, n_rows, num_blocks, block_size, max_position)."""
    import torch

    # Per-layer pointers: a contiguous stacked tensor is addressed by its
    # layer stride (no per-layer views); lists and other tensors layer by layer.
    if isinstance(caches, torch.Tensor) and caches.dim() == 5 and caches.is_contiguous():
        _bf16(caches, "cache")
        _same_device(caches, kv_ref, "caches")
        if caches.shape[0] != L:
            raise ValueError("one cache and one slot mapping per layer")
        if caches.shape[2] != H or caches.shape[4] != 2 * HEAD_DIM:
            raise ValueError("caches must be [num_blocks, H, block_size, 128]")
        nb, bs = caches.shape[1], caches.shape[3]
        c_base, c_step = caches.data_ptr(), caches.stride(0) * 2
        cache_ptrs = [c_base + i * c_step for i in range(L)]
    else:
        cache_list = list(caches) if not isinstance(caches, torch.Tensor) else [caches[i] for i in range(caches.shape[0])]
        if len(cache_list) != L:
            raise ValueError("one cache and one slot mapping per layer")
        c0 = cache_list[0]
        if c0.dim() != 4 or c0.shape[1] != H or c0.shape[3] != 2 * HEAD_DIM:
            raise ValueError("caches must be [num_blocks, H, block_size, 128]")
        nb, _, bs, _ = c0.shape
        for c in cache_list:
            _bf16(c, "cache")
            _same_device(c, kv_ref, "caches")
            if c.shape != c0.shape:
                raise ValueError("all caches must have one shape")
        cache_ptrs = [c.data_ptr() for c in cache_list]
    if isinstance(slots, torch.Tensor) and slots.dim() == 1:
        # one mapping shared by every layer: each layer's pointer is the same array
        if slots.dtype != torch.int64 or not slots.is_contiguous():
            raise ValueError("slots must be contiguous int64 [rows] tensors of one length")
        _same_device(slots, kv_ref, "slots")
        slot_len = slots.shape[0]
        slot_ptrs = [slots.data_ptr()] * L
    elif isinstance(slots, torch.Tensor) and slots.dim() == 2 and slots.is_contiguous():
        if slots.dtype != torch.int64:
            raise ValueError("slots must be contiguous int64 [rows] tensors of one length")
        if slots.shape[0] != L:
            raise ValueError("one cache and one slot mapping per layer")
        _same_device(slots, kv_ref, "slots")
        slot_len = slots.shape[1]
        s_base, s_step = slots.data_ptr(), slots.stride(0) * 8
        slot_ptrs = [s_base + i * s_step for i in range(L)]
    else:
        slot_list = list(slots) if not isinstance(slots, torch.Tensor) else [slots[i] for i in range(slots.shape[0])]
        if len(slot_list) != L:
            raise ValueError("one cache and one slot mapping per layer")
        for s in slot_list:
            if (not isinstance(s, torch.Tensor) or s.dtype != torch.int64 or s.dim() != 1 or not s.is_contiguous()
                    or s.shape[0] != slot_list[0].shape[0]):
                raise ValueError("slots must be contiguous int64 [rows] tensors of one length")
            _same_device(s, kv_ref, "slots")
        slot_len = slot_list[0].shape[0]
        slot_ptrs = [s.data_ptr() for s in slot_list]
    n_rows = slot_len if rows is None else int(rows)
    if n_rows < 0 or n_rows > slot_len:
        raise ValueError(f"rows = {n_rows} must lie in [0, {slot_len}] (the slot mapping's length)")
    if n_rows > T:
        raise ValueError(f"rows = {n_rows} exceeds the {T} rows of kv")
    if cos_sin is not None:
        _bf16(cos_sin, "cos_sin")
        _same_device(cos_sin, kv_ref, "cos_sin")
        if cos_sin.dim() != 2 or cos_sin.shape[1] != HEAD_DIM:
            raise ValueError("cos_sin must be [max_position, 64]")
        if positions is None or positions.dtype != torch.int64 or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int64 tensor")
        _same_device(positions, kv_ref, "positions")
        if positions.shape[0] < n_rows:
            raise ValueError("positions shorter than the inserted rows")
    slot_arr = (_vp * L)(*slot_ptrs)
    cache_arr = (_vp * L)(*cache_ptrs)
    max_pos = 0 if cos_sin is None else cos_sin.shape[0]
    return slot_arr, cache_arr, n_rows, nb, bs, max_pos


def context_kv_store_ex(kv, positions, slots, cos_sin, caches, H, eps=1e-6, k=None, v=None, stream=None):
    """The store with per-layer slot lists and strided cache views, in place.

    slots   a list of L entries: a contiguous int64 [rows_l] tensor (its
            first rows_l rows are inserted) or None (the layer stores nothing)
    caches  a list of L [num_blocks, H, block_size, 128] bf16 views of one
            shape and stride, unit last stride (any block / head / page
            strides that are multiples of 8), or None where slots is None
    Other arguments as context_kv_store."""
    import torch

    if k is None:
        _bf16(kv, "kv")
        k, v = kv_views(kv, H)
    for name, t in (("k", k), ("v", v)):
        _bf16(t, name, contiguous=False)
        if t.dim() != 4 or t.shape[2] != H or t.shape[3] != HEAD_DIM or t.stride(3) != 1 or t.stride(2) != HEAD_DIM:
            raise ValueError(f"{name} must be an [L, T, H, 64] view with unit last stride and head stride 64")
    L, T = k.shape[0], k.shape[1]
    _same_device(v, k, "v")
    slot_list, cache_list = list(slots), list(caches)
    if len(slot_list) != L or len(cache_list) != L:
        raise ValueError("one cache and one slot list (or None) per layer")
    live = [c for s, c in zip(slot_list, cache_list) if s is not None]
    if not live:
        return
    c0 = live[0]
    if c0.dim() != 4 or c0.shape[1] != H or c0.shape[3] != 2 * HEAD_DIM or c0.stride(3) != 1:
        raise ValueError("caches must be [num_blocks, H, block_size, 128] views with unit last stride")
    for c in live:
        if c is None or c.dtype != torch.bfloat16 or not c.is_cuda:
            raise ValueError("every layer with slots needs a bf16 device cache")
        _same_device(c, k, "caches")
        if c.shape != c0.shape or c.stride() != c0.stride():
            raise ValueError("all caches must have one shape and one stride")
    nb, _, bs, _ = c0.shape
    rows = []
    for s in slot_list:
        if s is None:
            rows.append(0)
            continue
        if not isinstance(s, torch.Tensor) or s.dtype != torch.int64 or s.dim() != 1 or not s.is_contiguous():
            raise ValueError("slots must be contiguous int64 [rows] tensors")
        _same_device(s, k, "slots")
        rows.append(s.shape[0])
    if cos_sin is not None:
        _bf16(cos_sin, "cos_sin")
        _same_device(cos_sin, k, "cos_sin")
        if cos_sin.dim() != 2 or cos_sin.shape[1] != HEAD_DIM:
            raise ValueError("cos_sin must be [max_position, 64]")
        if positions is None or positions.dtype != torch.int64 or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int64 tensor")
        _same_device(positions, k, "positions")
        if positions.shape[0] < max(rows):
            raise ValueError("positions shorter than the inserted rows")
    slot_arr = (_vp * L)(*[None if s is None else s.data_ptr() for s in slot_list])
    cache_arr = (_vp * L)(*[None if (s is None or c is None) else c.data_ptr()
                            for s, c in zip(slot_list, cache_list)])
    row_arr = (ctypes.c_int64 * L)(*rows)
    max_pos = 0 if cos_sin is None else cos_sin.shape[0]
    _call(k, _load().nrc_context_kv_store_ex, _ptr(k), _ptr(v), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
          _ptr(positions) if cos_sin is not None else None, slot_arr, row_arr, T, _ptr(cos_sin), max_pos, cache_arr, nb,
          bs, c0.stride(0), c0.stride(2), c0.stride(1), H, L, eps, _stream(stream, k))


def context_kv_store(kv, positions, slots, cos_sin, caches, H, eps=1e-6, rows=None, k=None, v=None,
                     stream=None):
    """K-norm + GPT-J RoPE + paged insert, in place on `caches`.

    kv       [L, T, 2 H 64] bf16 projection output (or pass k, v views
             [L, T, H, 64] with unit last stride and head stride 64)
    positions [T] int64 (unused without cos_sin)
    slots    [rows] int64 tensor (one mapping shared by every layer), an
             [L, rows] int64 tensor or a list of L [rows] int64 tensors
    rows     the first `rows` rows are inserted (default: the mapping's
             length; at most that length and T)
    cos_sin  [max_position, 64] bf16 or None (RoPE off)
    caches   [L, num_blocks, H, block_size, 128] bf16 tensor or a list of L
             [num_blocks, H, block_size, 128] tensors
    """
    import torch

    if k is None:
        _bf16(kv, "kv")
        if kv.dim() != 3 or kv.shape[2] != 2 * H * HEAD_DIM:
            raise ValueError("kv must be [L, T, 2 H 64]")
        # K and V are the two halves of each contiguous kv row
        L, T = kv.shape[0], kv.shape[1]
        k_ptr = kv.data_ptr()
        v_ptr = k_ptr + H * HEAD_DIM * 2
        k_ls = v_ls = kv.stride(0)
        k_rs = v_rs = kv.stride(1)
    else:
        for name, t in (("k", k), ("v", v)):
            _bf16(t, name, contiguous=False)
            if t.dim() != 4 or t.shape[2] != H or t.shape[3] != HEAD_DIM or t.stride(3) != 1 or t.stride(2) != HEAD_DIM:
                raise ValueError(f"{name} must be an [L, T, H, 64] view with unit last stride and head stride 64")
        L, T = k.shape[0], k.shape[1]
        _same_device(v, k, "v")
        k_ptr, v_ptr = k.data_ptr(), v.data_ptr()
        k_ls, k_rs, v_ls, v_rs = k.stride(0), k.stride(1), v.stride(0), v.stride(1)
    kv_ref = kv if k is None else k
    slot_arr, cache_arr, n_rows, nb, bs, max_pos = _store_operands(kv_ref, L, T, H, positions, slots, cos_sin,
                                                                  caches, rows)
    _call(kv_ref, _load().nrc_context_kv_store, ctypes.c_void_p(k_ptr), ctypes.c_void_p(v_ptr), k_ls, k_rs, v_ls, v_rs,
          _ptr(positions) if cos_sin is not None else None, slot_arr, n_rows, T, _ptr(cos_sin), max_pos, cache_arr, nb,
          bs, H, L, eps, _stream(stream, kv_ref))


def context_kv_project_store(normed, w_kv, positions, slots, cos_sin, caches, eps=1e-6, rows=None, out=None,
                             stream=None, w_layout="dn"):
    """context_kv_project (split=True) then context_kv_store on its output,
    in one call: same kv and cache bits. Where the shape splits the
    summation (small T), the store's kernel adds the slices itself, writing
    kv and inserting each row in the same pass. H = N / 128. Returns kv."""
    import torch

    L, T, D, N, layout, out = _project_operands(normed, w_kv, out, w_layout)
    if N % (2 * HEAD_DIM):
        raise ValueError("N must be 2 H 64")
    H = N // (2 * HEAD_DIM)
    slot_arr, cache_arr, n_rows, nb, bs, max_pos = _store_operands(out, L, T, H, positions, slots, cos_sin, caches,
                                                                  rows)
    lib = _load()
    need = lib.nrc_context_kv_project_workspace_bytes(L, T, D, N)
    if need < 0:
        _check(need)
    ws = None
    if need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=normed.device)
        if stream is not None:
            ws.record_stream(stream)
    _call(normed, lib.nrc_context_kv_project_store, _ptr(normed), _ptr(w_kv), layout, _ptr(out), L, T, D, N, _ptr(ws),
          need, _ptr(positions) if cos_sin is not None else None, slot_arr, n_rows, _ptr(cos_sin), max_pos, cache_arr,
          nb, bs, eps, _stream(stream, normed))
    return out


def check_scalars(x, want_bf16=True, want_rsqrt=True, stream=None):
    """Diagnostic: the library's device bf16 rounding and 1/sqrt applied to
    a float32 GPU tensor; returns (bf16 bits as int16 tensor, float32 tensor)."""
    import torch

    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 GPU tensor")
    bf = torch.empty(x.shape, dtype=torch.int16, device=x.device) if want_bf16 else None
    rs = torch.empty_like(x) if want_rsqrt else None
    _call(x, _load().nrc_check_scalars, _ptr(x), _ptr(bf), _ptr(rs), x.numel(), _stream(stream, x))
    return bf, rs


def check_bf16_pair(x, stream=None):
    """Diagnostic: the paired hardware bf16 conversion the norms use on
    NaN-free rows, applied to a float32 GPU tensor (bits as int16)."""
    import torch

    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 GPU tensor")
    out = torch.empty(x.shape, dtype=torch.int16, device=x.device)
    _call(x, _load().nrc_check_bf16_pair, _ptr(x), _ptr(out), x.numel(), _stream(stream, x))
    return out


TWIN_NORMS_STORES, TWIN_PLAIN_STORES, TWIN_READS_ONLY, TWIN_WRITES_ONLY = 0, 1, 2, 3


def traffic_twin(x, L, mode, out=None, per_cu=1, stream=None):
    """Diagnostic: the norms' HBM traffic (read x [T, 8192], write it to L
    rows of out [L, T, 8192]) in the norms' access pattern, no arithmetic;
    mode TWIN_* as in nrc.h. Returns out."""
    import torch

    _bf16(x, "x")
    T = x.shape[0]
    if tuple(x.shape) != (T, HIDDEN):
        raise ValueError("x must be [T, 8192]")
    if out is None and mode != TWIN_READS_ONLY:
        out = torch.empty((L, T, HIDDEN), dtype=torch.bfloat16, device=x.device)
    if out is not None:
        _bf16(out, "out")
        _same_device(out, x, "out")
        if tuple(out.shape) != (L, T, HIDDEN):
            raise ValueError("out must be [L, T, 8192]")
    sink = None
    if mode == TWIN_READS_ONLY:
        n = per_cu * torch.cuda.get_device_properties(x.device).multi_processor_count * 1024
        sink = torch.empty(n, dtype=torch.int32, device=x.device)
    _call(x, _load().nrc_traffic_twin, _ptr(x), T, L, mode, per_cu, _ptr(out), _ptr(sink),
          0 if sink is None else sink.numel(), _stream(stream, x))
    return out


def _empty(shape, dtype, device, stream):
    """An uninitialized tensor of the call's stream: as under
    torch.cuda.stream(stream) when one is given, so that its memory is not one that
    another stream still uses."""
    torch = _torch or _get_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the operands on {device}")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _fits32(v, name):
    """Raise unless v is an integer of 32 bits (ctypes would cut it)."""
    if not isinstance(v, int) or not -0x80000000 <= v <= 0x7FFFFFFF:
        raise ValueError(f"{name} must be an integer of 32 bits, not {v!r}")


ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_PASS_OUTSIDE = 1


def _dtype_code(dtype, name, table=False):
    torch = _torch or _get_torch()
    if dtype == torch.bfloat16:
        return 0
    if dtype == torch.float32:
        return 2
    if dtype == torch.float16 and not table:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float32{'' if table else ' or float16'}, not {dtype}")


def rope_table(count, rotary_dim, base=10000.0, scaling="none", factor=1.0, original_max=0, low=1.0, high=32.0,
               magnitude=1.0, width=None, start=0, dtype=None, device=None, out=None, stream=None):
    """The cos/sin table [count, width] of positions start .. start + count - 1
    (bf16 unless dtype is float32): cos of width / 2 pairs, then sin.

    rotary_dim  the elements that turn; width (default rotary_dim) adds pairs
                that do not (64 with a smaller rotary_dim lets context_kv_store
                rotate a part of the head)
    scaling     "none"; "linear" (angles divided by factor); "base" (base
                times factor^(R / (R - 2))); "bands" and "ramp" (slow pairs
                divided, fast ones kept, those between `low` and `high` turns over
                original_max in between: by their turns, or by their index;
                the ramp's upper index is held to the last pair)
    magnitude   factor of cos and sin
    """
    torch = _torch or _get_torch()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling is one of {', '.join(ROPE_SCALINGS)}")
    width = rotary_dim if width is None else width
    if not -1 << 63 <= start < 1 << 63:  # (ctypes would cut it)
        raise ValueError("start does not fit 64 bits")
    _fits32(rotary_dim, "rotary_dim")
    _fits32(width, "width")
    if out is None:
        if count < 0 or width < 0:
            raise ValueError("count and width must not be negative")
        device = torch.device("cuda") if device is None else torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"the table is made on a GPU, not on {device}")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        out = _empty((count, width), torch.bfloat16 if dtype is None else dtype, device, stream)
    elif not out.is_cuda or not out.is_contiguous() or tuple(out.shape) != (count, width):
        raise ValueError("out must be a contiguous device tensor [count, width]")
    elif dtype is not None and out.dtype != dtype or device is not None and torch.device(device) not in (
            out.device, torch.device(out.device.type)):
        raise ValueError("out is of another dtype or device than asked for")
    code = _dtype_code(out.dtype, "the table", table=True)
    _call(out, _load().nrc_rope_table, start, count, rotary_dim, width, base, ROPE_SCALINGS[scaling], factor,
          original_max, low, high, magnitude, _ptr(out), code, _stream(stream, out))
    return out


_rotation = None  # the rotation as a torch.autograd.Function, once an x that requires grad has needed it


def _get_rotation():
    global _rotation
    import torch

    class Rotation(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, cos_sin, layout, inverse, stream):
            ctx.save_for_backward(positions, cos_sin)
            ctx.layout, ctx.inverse = layout, inverse
            return rope_rotate(x, positions, cos_sin, layout, inverse, stream=stream)

        @staticmethod
        def backward(ctx, grad):
            positions, cos_sin = ctx.saved_tensors
            if grad.stride(2) != 1:  # (of a sum: one value for all)
                grad = grad.clone(memory_format=torch.contiguous_format)
            # the map is linear and orthogonal up to the table's magnitude: its transposed is the turn by the negative
            # angles, and rows that came through as they were pass their gradient
            back = rope_rotate(grad, positions, cos_sin, ctx.layout, not ctx.inverse)
            return back, None, None, None, None, None

    _rotation = Rotation
    return Rotation


def rope_rotate(x, positions, cos_sin, layout="interleaved", inverse=False, out=None, stream=None):
    """x [T, H, d] (bf16, float16 or float32; any row and head strides) with the
    first R = cos_sin.shape[1] elements of each head turned by its row's
    position; the rest is copied.

    positions  [T] int64; a row outside the table is left as it is in a given
               out, and comes out as it went in otherwise
    cos_sin    [max_position, R] bf16 or float32 (rope_table)
    layout     "interleaved" (pairs 2j, 2j + 1, as context_kv_store turns its
               keys) or "half" (pairs j, j + R / 2)
    inverse    turn back: the gradient of the rotation
    out        x itself, or a tensor apart from it (default: a new one)
    An x that requires grad gets its gradient (by the inverse, on the current
    stream of the forward call); it takes no out, and cos_sin gets none.
    """
    torch = _torch or _get_torch()
    code = _dtype_code(x.dtype, "x")
    dev = x.get_device()
    if dev < 0:
        raise TypeError("x must be a GPU tensor")
    shape, st = x.shape, x.stride()
    if len(shape) != 3 or st[2] != 1 and shape[2] != 1:
        raise ValueError("x must be [T, H, d] with unit last stride")
    T, H, d = shape
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout is 'interleaved' or 'half'")
    _at(positions, dev, "positions")
    _at(cos_sin, dev, "cos_sin")
    tcode = _dtype_code(cos_sin.dtype, "cos_sin", table=True)
    table = cos_sin.shape
    if len(table) != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous [max_position, R]")
    if positions.dtype != torch.int64 or positions.shape != (T,) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int64 [T] tensor")
    if (x.requires_grad or cos_sin.requires_grad) and torch.is_grad_enabled():
        if cos_sin.requires_grad:
            raise ValueError("cos_sin gets no gradient: detach it")
        if out is not None:
            raise ValueError("an x that requires grad takes no out: detach it, or call under torch.no_grad()")
        return (_rotation or _get_rotation()).apply(x, positions, cos_sin, layout, inverse, stream)
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
        ost, flags = (H * d, d), ROPE_PASS_OUTSIDE
    else:
        ost, flags = out.stride(), 0
        if out.dtype != x.dtype or out.shape != shape or ost[2] != 1:
            raise ValueError("out must be shaped like x, of its dtype, with unit last stride")
        _at(out, dev, "out")
    _call(x, _load().nrc_rope_rotate_ex, x.data_ptr(), code, T, H, d, st[0], st[1], positions.data_ptr(),
          cos_sin.data_ptr(), tcode, table[0], table[1], ROPE_LAYOUTS[layout], 1 if inverse else 0, out.data_ptr(), ost[0],
          ost[1], flags, _stream(stream, x))
    return out


def _at(t, dev, name):
    """Raise unless t is a tensor on GPU `dev`."""
    torch = _torch or _get_torch()
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        where = "not a tensor" if not isinstance(t, torch.Tensor) else str(t.device)
        raise ValueError(f"{name} must be a tensor on cuda:{dev} ({where})")


def _int32(t, name, dev, shape):
    torch = _torch or _get_torch()
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype == torch.int32 and t.shape == shape
            and t.is_contiguous()):
        return
    _at(t, dev, name)
    raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor")


def _paged_operands(cache, tables):
    """Checks of one layer's cache view and its block tables; the GPU, and the
    C ABI's arguments from `cache` to `B`."""
    torch = _torch or _get_torch()
    dev = cache.get_device()
    if cache.dtype != torch.bfloat16 or dev < 0:
        raise TypeError(f"cache must be a bfloat16 GPU tensor, not {cache.dtype} on {cache.device}")
    shape, st = cache.shape, cache.stride()
    if len(shape) != 4 or shape[3] != 2 * HEAD_DIM or st[3] != 1:
        raise ValueError("cache must be a [num_blocks, H, block_size, 128] view with unit last stride")
    _at(tables, dev, "tables")
    if tables.dtype != torch.int32 or tables.dim() != 2:
        raise ValueError("tables must be an int32 [B, blocks] tensor")
    B, width = tables.shape
    tst = tables.stride()
    if width > 1 and tst[1] != 1:
        raise ValueError("tables must have unit last stride")
    nb, H, bs, _ = shape
    # (one of a kind has no stride)
    return dev, (cache.data_ptr(), nb, bs, st[0] if nb > 1 else 0, st[2] if bs > 1 else 0, st[1] if H > 1 else 0, H,
                 tables.data_ptr(), tst[0], width, B)


def _query_operands(q, cache, tables, ctx_lens, q_starts, max_nodes, max_ctx, tree_mask, scale, softcap):
    """Checks shared by the attention and its received weights; the GPU, T, Hq, H,
    B, max_ctx and the C ABI's arguments from `q` to `softcap`."""
    torch = _torch or _get_torch()
    dev, paged = _paged_operands(cache, tables)
    bs, H, width, B = paged[2], paged[6], paged[9], paged[10]
    _fits32(max_nodes, "max_nodes")
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q must be bfloat16, not {q.dtype}")
    _at(q, dev, "q")
    shape, st = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != HEAD_DIM or st[2] != 1:
        raise ValueError("q must be [T, Hq, 64] with unit last stride")
    T, Hq, _ = shape
    _int32(ctx_lens, "ctx_lens", dev, (B,))
    _int32(q_starts, "q_starts", dev, (B + 1,))
    mask, words = None, 0
    if tree_mask is not None:
        _at(tree_mask, dev, "tree_mask")
        if tree_mask.dtype != torch.int64 or tree_mask.dim() != 2 or not tree_mask.is_contiguous():
            raise ValueError("tree_mask must be a contiguous int64 [T, words] tensor")
        rows, words = tree_mask.shape
        if rows != T or words == 0:
            raise ValueError("tree_mask must have T rows of a word at least")
        if T:
            mask = tree_mask.data_ptr()
        else:
            words = 0  # (no row to read)
    if max_ctx is None:
        max_ctx = width * bs
    elif not 0 <= max_ctx < 1 << 63:  # (ctypes would cut it)
        raise ValueError("max_ctx must not be negative and fit 64 bits")
    return dev, T, Hq, H, B, max_ctx, (
        q.data_ptr(), st[0] if T > 1 else 0, st[1] if Hq > 1 else 0, T, Hq, *paged, ctx_lens.data_ptr(),
        q_starts.data_ptr(), max_nodes, max_ctx, mask, words, HEAD_DIM ** -0.5 if scale is None else scale, softcap)


ATTENTION_FILL_OUT, ATTENTION_FILL_LSE = 1, 2


def context_tree_attention(q, cache, tables, ctx_lens, q_starts, max_nodes, max_ctx=None, tree_mask=None, scale=None,
                           softcap=0.0, out=None, lse=None, stream=None):
    """Drafted tokens attending to the cache of one layer -> (out [T, Hq, 64]
    bf16, lse [T, Hq] float32).

    q         [T, Hq, 64] bf16, every sequence's nodes one after the other;
              query head i reads KV head i // (Hq // H)
    cache     [num_blocks, H, block_size, 128] bf16 (context_kv_store), any
              strides that are multiples of 8
    tables    [B, blocks] int32: the sequences' blocks
    ctx_lens  [B] int32: keys before the nodes; node i's K and V are key
              ctx_lens + i, stored before the call
    q_starts  [B + 1] int32: sequence b's rows of q
    max_nodes most nodes of a sequence; max_ctx most of ctx_lens (default: what
              the tables hold)
    tree_mask [T, words] int64: bit j set, the row sees node j of its
              sequence; None: a chain (each node sees those up to itself)
    scale     factor of the scores (1/8); softcap: scores become
              softcap tanh(score / softcap) when it is not 0 (2^-10 .. 2^10)
    The weights are rounded to bf16 for the product with V.
    A row that sees no key gets 0 and -inf; so does, in an output that is not
    given, a row of no sequence or past max_nodes (in a given one it stays as it
    is). The keys of long contexts are split
    over workgroups, with a workspace from torch's allocator."""
    torch = _torch or _get_torch()
    dev, T, Hq, H, B, max_ctx, args = _query_operands(q, cache, tables, ctx_lens, q_starts, max_nodes, max_ctx,
                                                      tree_mask, scale, softcap)
    flags = 0
    if out is None:
        out = _empty((T, Hq, HEAD_DIM), torch.bfloat16, q.device, stream)
        flags = ATTENTION_FILL_OUT
    else:
        _at(out, dev, "out")
        if out.dtype != torch.bfloat16 or out.shape != (T, Hq, HEAD_DIM) or not out.is_contiguous():
            raise ValueError("out must be a contiguous bfloat16 [T, Hq, 64]")
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, stream)
        flags |= ATTENTION_FILL_LSE
    else:
        _float_lse(lse, dev, (T, Hq))
    lib = _load()
    # the split follows the device's size: asked with q's GPU as the current device
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            need = lib.nrc_context_tree_attention_workspace_bytes(B, T, Hq, H, max_nodes, max_ctx)
    else:
        need = lib.nrc_context_tree_attention_workspace_bytes(B, T, Hq, H, max_nodes, max_ctx)
    if need < 0:
        _check(need)
    ws = _empty((need,), torch.uint8, q.device, stream) if need > 0 else None
    _call(q, lib.nrc_context_tree_attention_ex, *args, out.data_ptr(), lse.data_ptr(),
          None if ws is None else ws.data_ptr(), need, flags, _stream(stream, q))
    return out, lse


def _float_lse(lse, dev, shape):
    torch = _torch or _get_torch()
    if (isinstance(lse, torch.Tensor) and lse.get_device() == dev and lse.dtype == torch.float32 and lse.shape == shape
            and lse.is_contiguous()):
        return
    _at(lse, dev, "lse")
    raise ValueError("lse must be a contiguous float32 [T, Hq] tensor")


def _cells(t, name, dev, dtype, shape):
    """A [B, H, width] tensor of per-cell values with unit last stride; its strides."""
    torch = _torch or _get_torch()
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _at(t, dev, name)
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor")
    st = t.stride()
    if shape[2] > 1 and st[2] != 1:
        raise ValueError(f"{name} must have unit last stride")
    return st


def context_attention_mass(q, cache, tables, ctx_lens, q_starts, lse, max_nodes, max_ctx=None, tree_mask=None,
                           scale=None, softcap=0.0, weights=None, decay=1.0, width=None, out=None, stream=None):
    """decay * weights + the attention weight each cached cell receives from
    the rows of q, [B, H, width] float32; 0 past each sequence's keys.

    lse      [T, Hq] float32 from context_tree_attention on the same operands
    weights  [B, H, width] float32 (any batch and head strides) or None (0)
    width    cells a head (default: weights' or out's, else what the tables hold)
    out      weights itself, or a tensor apart from it (default: a new one)
    Other arguments as context_tree_attention."""
    torch = _torch or _get_torch()
    dev, T, Hq, H, B, max_ctx, args = _query_operands(q, cache, tables, ctx_lens, q_starts, max_nodes, max_ctx,
                                                      tree_mask, scale, softcap)
    _float_lse(lse, dev, (T, Hq))
    if width is None:
        given = weights if weights is not None else out
        width = tables.shape[1] * cache.shape[2] if given is None or given.dim() != 3 else given.shape[2]
    if width < 0:
        raise ValueError("width must not be negative")
    shape = (B, H, width)
    w, wst = None, (0, 0)
    if weights is not None:
        wst = _cells(weights, "weights", dev, torch.float32, shape)
        w = weights.data_ptr()
    if out is None:
        out = _empty(shape, torch.float32, q.device, stream)
        ost = (H * width, width)
    else:
        ost = _cells(out, "out", dev, torch.float32, shape)
    _call(q, _load().nrc_context_attention_mass, *args, lse.data_ptr(), w, wst[0], wst[1], decay, out.data_ptr(), ost[0],
          ost[1], width, _stream(stream, q))
    return out


def context_kv_evict(cache, tables, lens, weights, positions, ends, budget, sinks=0, recent=0, new_weights=None,
                     new_positions=None, new_lens=None, stream=None):
    """Keep, in place, the `budget` cells of every (sequence, KV head) with the
    most weight -> (new_weights [B, H, budget] float32, new_positions
    [B, H, budget] int32, new_lens [B] int32).

    cache, tables  as context_tree_attention; no block in two tables
    lens       [B] int32: cells of each sequence
    weights    [B, H, width] float32, positions [B, H, width] int32 (any batch
               and head strides), width >= every length
    ends       [B] int32: one past the newest token's position
    sinks, recent  positions below sinks, and from ends - recent on, come first
    Equal weights: the lower index stays, among more protected cells than the
    budget too (the newest go: recent <= budget - sinks keeps them). Kept cells past the new length move
    into the holes before it; weights and positions follow them, into tensors
    apart from the given ones."""
    torch = _torch or _get_torch()
    dev, paged = _paged_operands(cache, tables)
    H, B = paged[6], paged[10]
    _fits32(budget, "budget")
    _fits32(sinks, "sinks")
    _fits32(recent, "recent")
    if budget < 1:
        raise ValueError("budget must be at least 1")
    _int32(lens, "lens", dev, (B,))
    _int32(ends, "ends", dev, (B,))
    if not isinstance(weights, torch.Tensor) or weights.dim() != 3:
        raise ValueError("weights must be a float32 [B, H, width] tensor")
    width = weights.shape[2]
    wst = _cells(weights, "weights", dev, torch.float32, (B, H, width))
    pst = _cells(positions, "positions", dev, torch.int32, (B, H, width))
    lib = _load()
    need = lib.nrc_context_kv_evict_workspace_bytes(B, H, width, budget)
    if need < 0:
        _check(need)
    device, shape = cache.device, (B, H, budget)
    if new_weights is None:
        new_weights = _empty(shape, torch.float32, device, stream)
    else:
        _cells(new_weights, "new_weights", dev, torch.float32, shape)
    if new_positions is None:
        new_positions = _empty(shape, torch.int32, device, stream)
    else:
        _cells(new_positions, "new_positions", dev, torch.int32, shape)
    if not new_weights.is_contiguous() or not new_positions.is_contiguous():
        raise ValueError("new_weights and new_positions must be contiguous")
    if new_lens is None:
        new_lens = _empty((B,), torch.int32, device, stream)
    else:
        _int32(new_lens, "new_lens", dev, (B,))
    ws = _empty((need,), torch.uint8, device, stream) if need > 0 else None
    _call(cache, lib.nrc_context_kv_evict, *paged, lens.data_ptr(), weights.data_ptr(), wst[0], wst[1],
          positions.data_ptr(), pst[0], pst[1], width, ends.data_ptr(), sinks, recent, budget, new_weights.data_ptr(),
          new_positions.data_ptr(), new_lens.data_ptr(), None if ws is None else ws.data_ptr(), need,
          _stream(stream, cache))
    return new_weights, new_positions, new_lens


def context_kv_chain(x, hidden_w, pre_w, w_kv, positions, slots, cos_sin, caches, H, hidden_eps=1e-6,
                     pre_eps=1e-6, k_eps=1e-6, fused=False, workspace=None, kv=None, stream=None, split=True):
    """The whole chain, in place on `caches`; returns kv [L, T, N].

    fused=False (the faster form on MI355X at H = 8): norms into `workspace`
    ([L, T, 8192] bf16) -> projection and store (one call with split=True). fused=True: pre-pass (h, r)
    -> fused projection -> store, without the [L, T, 8192] intermediate;
    `workspace` may be a tuple (h [T, 8192] bf16, r [T] float32). Both forms
    write the same bits for the same `split`; for small T split=True splits
    the summation (see context_kv_project), which changes the rounding
    within the projection's tolerance."""
    L = w_kv.shape[0]
    if fused:
        h, r = workspace if workspace is not None else (None, None)
        h, r = context_hidden_norm(x, hidden_w, pre_w, L, hidden_eps, pre_eps, h=h, r=r, stream=stream)
        kv = context_kv_project_fused(h, r, pre_w, w_kv, out=kv, stream=stream, split=split)
    else:
        normed = context_norms(x, hidden_w, pre_w, L, hidden_eps, pre_eps, out=workspace, stream=stream)
        if split:
            # the projection and the store in one call (same bits as the two)
            if w_kv.shape[2] != 2 * H * HEAD_DIM:
                raise ValueError("w_kv must be [L, D, 2 H 64]")
            return context_kv_project_store(normed, w_kv, positions, slots, cos_sin, caches, k_eps, out=kv,
                                            stream=stream)
        kv = context_kv_project(normed, w_kv, out=kv, stream=stream, split=split)
    context_kv_store(kv, positions, slots, cos_sin, caches, H, k_eps, stream=stream)
    return kv
