"""Python binding of libwanvae.so (include/wanvae.h): argument marshalling only.

Every function here forwards to the C entry point of the same name; all the
work runs in the library's CUDA kernels.  torch is used for device memory
and streams.  There is no fallback: if the library is missing or a call
fails, an exception is raised.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwanvae.so")

(OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT,
 ERR_UNDRAINED) = range(8)
BF16, F32, E4M3, E2M1 = 0, 1, 2, 3

# Every exported symbol of include/wanvae.h.
EXPORTS = (
    "wanvae_status_string", "wanvae_version", "wanvae_rmsnorm_silu", "wanvae_causal_conv3d",
    "wanvae_resblock_workspace_size", "wanvae_resblock_forward",
    "wanvae_resblock_forward_profiled", "wanvae_sync_status", "wanvae_set_wait_limit_ns",
    "wanvae_launch_count", "wanvae_resblock_forward_static", "wanvae_upsample2d_workspace_size",
    "wanvae_upsample2d_conv", "wanvae_set_kernel_variant", "wanvae_time_upsample_workspace_size",
    "wanvae_time_upsample_conv", "wanvae_upsample3d_workspace_size", "wanvae_upsample3d",
    "wanvae_frame_attention_workspace_size", "wanvae_frame_attention",
    "wanvae_resblock_forward_host_workspace_size", "wanvae_resblock_forward_host",
    "wanvae_packed_attention", "wanvae_kv_cache_append", "wanvae_kv_cache_gather",
    "wanvae_paged_attention_workspace_size", "wanvae_paged_attention",
    "wanvae_gated_residual_norm", "wanvae_kv_cache_write", "wanvae_kv_pages_extend",
    "wanvae_kv_pages_release", "wanvae_qk_norm_rotate",
)

# Size of the library's own workspace used by resblock_forward_static.
STATIC_WORKSPACE_BYTES = 32 << 20


class WanvaeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("W", ctypes.c_int64)]


class ResblockParams(ctypes.Structure):
    _fields_ = [
        ("c_in", ctypes.c_int64), ("c_out", ctypes.c_int64), ("eps", ctypes.c_float),
        ("gamma1", ctypes.c_void_p), ("gamma2", ctypes.c_void_p),
        ("wA", ctypes.c_void_p), ("bA", ctypes.c_void_p),
        ("wB", ctypes.c_void_p), ("bB", ctypes.c_void_p),
        ("wS", ctypes.c_void_p), ("bS", ctypes.c_void_p),
    ]


class ResblockCache(ctypes.Structure):
    _fields_ = [("convA_in", ctypes.c_void_p), ("convB_in", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("n_kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("dt", ctypes.c_int), ("k_off", ctypes.c_void_p), ("v_off", ctypes.c_void_p)]


class KvPagePoolDesc(ctypes.Structure):
    _fields_ = [("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int64)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.POINTER(ctypes.c_double)), ("n_axes", ctypes.c_int64),
                ("pairs", ctypes.c_int64 * 4), ("interleaved", ctypes.c_int)]


_lib = None


def load(path=LIB_PATH):
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with video_vae_causal_gb300.build")
    L = ctypes.CDLL(path)
    vp, i64, ci, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int
    L.wanvae_status_string.argtypes = [st]
    L.wanvae_status_string.restype = ctypes.c_char_p
    L.wanvae_version.argtypes = []
    L.wanvae_version.restype = ci
    L.wanvae_rmsnorm_silu.argtypes = [vp, vp, vp, ci, i64, i64, ctypes.c_float, vp]
    L.wanvae_rmsnorm_silu.restype = st
    L.wanvae_causal_conv3d.argtypes = [vp, vp, vp, vp, Dims, i64, i64, ci, vp, vp]
    L.wanvae_causal_conv3d.restype = st
    L.wanvae_resblock_workspace_size.argtypes = [Dims, i64, i64]
    L.wanvae_resblock_workspace_size.restype = ctypes.c_size_t
    L.wanvae_resblock_forward.argtypes = [ctypes.POINTER(ResblockParams), vp, vp, Dims,
                                          ctypes.POINTER(ResblockCache), vp, ctypes.c_size_t, vp]
    L.wanvae_resblock_forward.restype = st
    L.wanvae_resblock_forward_profiled.argtypes = [
        ctypes.POINTER(ResblockParams), vp, vp, Dims, ctypes.POINTER(ResblockCache), vp,
        ctypes.c_size_t, ctypes.POINTER(vp), vp]
    L.wanvae_resblock_forward_profiled.restype = st
    L.wanvae_sync_status.argtypes = [vp]
    L.wanvae_sync_status.restype = st
    L.wanvae_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.wanvae_set_wait_limit_ns.restype = None
    L.wanvae_resblock_forward_host_workspace_size.argtypes = [Dims, i64, i64, i64]
    L.wanvae_resblock_forward_host_workspace_size.restype = ctypes.c_size_t
    L.wanvae_resblock_forward_host.argtypes = [ctypes.POINTER(ResblockParams), vp, vp, Dims, i64,
                                               vp, ctypes.c_size_t, vp, vp, vp]
    L.wanvae_resblock_forward_host.restype = st
    L.wanvae_set_kernel_variant.argtypes = [ci, ci, ci, ci, ci]
    L.wanvae_set_kernel_variant.restype = None
    L.wanvae_launch_count.argtypes = []
    L.wanvae_launch_count.restype = ctypes.c_uint64
    L.wanvae_resblock_forward_static.argtypes = [ctypes.POINTER(ResblockParams), vp, vp, Dims,
                                                 ctypes.POINTER(ResblockCache), vp]
    L.wanvae_resblock_forward_static.restype = st
    L.wanvae_upsample2d_workspace_size.argtypes = [i64, i64]
    L.wanvae_upsample2d_workspace_size.restype = ctypes.c_size_t
    L.wanvae_upsample2d_conv.argtypes = [vp, vp, vp, vp, Dims, i64, i64, vp, ctypes.c_size_t, vp]
    L.wanvae_upsample2d_conv.restype = st
    L.wanvae_time_upsample_workspace_size.argtypes = [i64, i64]
    L.wanvae_time_upsample_workspace_size.restype = ctypes.c_size_t
    L.wanvae_time_upsample_conv.argtypes = [vp, vp, vp, vp, Dims, i64, i64, vp, ctypes.c_size_t,
                                            vp]
    L.wanvae_time_upsample_conv.restype = st
    L.wanvae_upsample3d_workspace_size.argtypes = [Dims, i64, i64, i64]
    L.wanvae_upsample3d_workspace_size.restype = ctypes.c_size_t
    L.wanvae_upsample3d.argtypes = [vp, vp, vp, vp, vp, vp, Dims, i64, i64, i64, vp,
                                    ctypes.c_size_t, vp]
    L.wanvae_upsample3d.restype = st
    L.wanvae_frame_attention_workspace_size.argtypes = [Dims, i64]
    L.wanvae_frame_attention_workspace_size.restype = ctypes.c_size_t
    L.wanvae_frame_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, Dims, i64, ctypes.c_float, vp,
                                         ctypes.c_size_t, vp]
    L.wanvae_frame_attention.restype = st
    cache, f32 = ctypes.POINTER(KvCacheDesc), ctypes.c_float
    L.wanvae_packed_attention.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, i64,
                                          i64, i64, i64, i64, f32, ci, vp]
    L.wanvae_packed_attention.restype = st
    L.wanvae_kv_cache_append.argtypes = [cache, vp, i64, vp, i64, vp, vp, i64, vp, i64, i64, vp]
    L.wanvae_kv_cache_append.restype = st
    L.wanvae_kv_cache_gather.argtypes = [cache, vp, i64, vp, i64, i64, vp, i64, vp, i64, vp]
    L.wanvae_kv_cache_gather.restype = st
    L.wanvae_paged_attention_workspace_size.argtypes = [i64, i64, i64]
    L.wanvae_paged_attention_workspace_size.restype = ctypes.c_size_t
    L.wanvae_paged_attention.argtypes = [vp, i64, cache, vp, vp, i64, i64, i64, f32, vp, i64, vp,
                                         ctypes.c_size_t, vp]
    L.wanvae_paged_attention.restype = st
    L.wanvae_gated_residual_norm.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, ci, i64, i64, f32,
                                             f32, vp]
    L.wanvae_gated_residual_norm.restype = st
    L.wanvae_kv_cache_write.argtypes = [cache, vp, i64, vp, i64, vp, i64, vp]
    L.wanvae_kv_cache_write.restype = st
    pool = ctypes.POINTER(KvPagePoolDesc)
    L.wanvae_kv_pages_extend.argtypes = [pool, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    L.wanvae_kv_pages_extend.restype = st
    L.wanvae_kv_pages_release.argtypes = [pool, vp, vp, vp, i64, i64, vp, vp, vp]
    L.wanvae_kv_pages_release.restype = st
    L.wanvae_qk_norm_rotate.argtypes = [vp, i64, vp, i64, vp, vp, ctypes.POINTER(RotaryDesc), vp, vp,
                                        i64, vp, i64, ci, i64, i64, i64, i64, f32, vp]
    L.wanvae_qk_norm_rotate.restype = st
    _lib = L
    return L


def status_string(status):
    return load().wanvae_status_string(int(status)).decode()


def _check(status, where):
    if status != OK:
        raise WanvaeError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dims(shape):
    B, T, H, W = shape[:4]
    return Dims(B, T, H, W)


def version():
    return int(load().wanvae_version())


def launch_count():
    return int(load().wanvae_launch_count())


def set_wait_limit_ns(ns):
    load().wanvae_set_wait_limit_ns(int(ns))


def set_kernel_variant(pair=-1, halo=-1, wide=-1, narrow=-1, fuse_norm=-1):
    """Force kernel variants for later calls (0 or 1 each; -1 = automatic)."""
    load().wanvae_set_kernel_variant(int(pair), int(halo), int(wide), int(narrow),
                                     int(fuse_norm))


def sync_status(stream=None):
    """Synchronise the stream; raise WanvaeError(ERR_TIMEOUT) if a kernel of
    the library gave up a bounded wait."""
    _check(load().wanvae_sync_status(_stream(stream)), "wanvae_sync_status")


def rmsnorm_silu(x, gamma, y=None, eps=1e-12, stream=None):
    """SiLU(RMS_norm(x)) over the last axis of x (bf16 or fp32, contiguous)."""
    dt = {torch.bfloat16: BF16, torch.float32: F32}[x.dtype]
    if y is None:
        y = torch.empty_like(x)
    C = x.shape[-1]
    st = load().wanvae_rmsnorm_silu(_ptr(x), _ptr(y), _ptr(gamma), dt, x.numel() // C, C,
                                    float(eps), _stream(stream))
    _check(st, "wanvae_rmsnorm_silu")
    return y


def causal_conv3d(x, w, bias=None, y=None, cache=None, stream=None):
    """CausalConv3d of NDHWC bf16 x [B,T,H,W,c_in] with w [c_out,k,k,k,c_in]."""
    c_out, k = w.shape[0], w.shape[1]
    if y is None:
        y = torch.empty(x.shape[:4] + (c_out,), dtype=torch.bfloat16, device=x.device)
    st = load().wanvae_causal_conv3d(_ptr(x), _ptr(w), _ptr(bias), _ptr(y), _dims(x.shape),
                                     x.shape[4], c_out, k, _ptr(cache), _stream(stream))
    _check(st, "wanvae_causal_conv3d")
    return y


def upsample2d_conv(x, w, bias=None, y=None, workspace=None, stream=None):
    """Nearest 2x upsampling in H and W, then a 3x3 conv with bias, per frame.
    x [B,T,H,W,c_in] bf16, w [c_out,3,3,c_in] bf16 -> y [B,T,2H,2W,c_out]."""
    B, T, H, W, c_in = x.shape
    c_out = w.shape[0]
    if y is None:
        y = torch.empty((B, T, 2 * H, 2 * W, c_out), dtype=torch.bfloat16, device=x.device)
    L = load()
    if workspace is None:
        n = int(L.wanvae_upsample2d_workspace_size(c_in, c_out))
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    st = L.wanvae_upsample2d_conv(_ptr(x), _ptr(w), _ptr(bias), _ptr(y), _dims(x.shape), c_in,
                                  c_out, _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "wanvae_upsample2d_conv")
    return y


def time_upsample_conv(x, w, bias=None, y=None, workspace=None, stream=None):
    """Nearest 2x upsampling in T, then a causal 3x1x1 conv with bias (the
    temporal half of upsample3d).  x [B,T,H,W,c_in] bf16, w [c_out,3,c_in]
    bf16 -> y [B,2T,H,W,c_out]."""
    B, T, H, W, c_in = x.shape
    c_out = w.shape[0]
    if y is None:
        y = torch.empty((B, 2 * T, H, W, c_out), dtype=torch.bfloat16, device=x.device)
    L = load()
    if workspace is None:
        n = int(L.wanvae_time_upsample_workspace_size(c_in, c_out))
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    st = L.wanvae_time_upsample_conv(_ptr(x), _ptr(w), _ptr(bias), _ptr(y), _dims(x.shape), c_in,
                                     c_out, _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "wanvae_time_upsample_conv")
    return y


def upsample3d(x, w_t, b_t, w_s, b_s, y=None, workspace=None, stream=None):
    """upsample3d: the temporal half (w_t [c_mid,3,c_in]) then the spatial
    upsampler (w_s [c_out,3,3,c_mid]).  x [B,T,H,W,c_in] -> [B,2T,2H,2W,c_out]."""
    B, T, H, W, c_in = x.shape
    c_mid, c_out = w_t.shape[0], w_s.shape[0]
    if y is None:
        y = torch.empty((B, 2 * T, 2 * H, 2 * W, c_out), dtype=torch.bfloat16, device=x.device)
    L = load()
    if workspace is None:
        n = int(L.wanvae_upsample3d_workspace_size(_dims(x.shape), c_in, c_mid, c_out))
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    st = L.wanvae_upsample3d(_ptr(x), _ptr(w_t), _ptr(b_t), _ptr(w_s), _ptr(b_s), _ptr(y),
                             _dims(x.shape), c_in, c_mid, c_out, _ptr(workspace),
                             workspace.numel(), _stream(stream))
    _check(st, "wanvae_upsample3d")
    return y


def frame_attention(x, gamma, wqkv, bqkv=None, wo=None, bo=None, y=None, workspace=None,
                    eps=1e-12, stream=None):
    """The mid-block attention: y = x + Wo softmax(q k^T / sqrt(C)) v + bo per
    frame, [q; k; v] = Wqkv RMS_norm(x) + bqkv.  x [B,T,H,W,C] bf16, gamma fp32
    [C], wqkv bf16 [3C,C], bqkv fp32 [3C], wo bf16 [C,C], bo fp32 [C]."""
    B, T, H, W, C = x.shape
    if y is None:
        y = torch.empty_like(x)
    L = load()
    if workspace is None:
        n = int(L.wanvae_frame_attention_workspace_size(_dims(x.shape), C))
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    st = L.wanvae_frame_attention(_ptr(x), _ptr(gamma), _ptr(wqkv), _ptr(bqkv), _ptr(wo),
                                  _ptr(bo), _ptr(y), _dims(x.shape), C, eps, _ptr(workspace),
                                  workspace.numel(), _stream(stream))
    _check(st, "wanvae_frame_attention")
    return y


def resblock_workspace_size(dims, c_in, c_out):
    return int(load().wanvae_resblock_workspace_size(_dims(dims), c_in, c_out))


def make_params(p, eps=1e-12):
    """ResblockParams from a dict of device tensors (gamma1, wA, bA, gamma2,
    wB, bB and optionally wS, bS).  Keep the dict alive while it is used."""
    c_out, c_in = p["wA"].shape[0], p["wA"].shape[-1]
    return ResblockParams(c_in, c_out, eps, p["gamma1"].data_ptr(), p["gamma2"].data_ptr(),
                          p["wA"].data_ptr(), p["bA"].data_ptr(), p["wB"].data_ptr(),
                          p["bB"].data_ptr(),
                          p["wS"].data_ptr() if p.get("wS") is not None else None,
                          p["bS"].data_ptr() if p.get("bS") is not None else None)


def make_workspace(dims, c_in, c_out, device="cuda"):
    n = resblock_workspace_size(dims, c_in, c_out)
    return torch.empty(n, dtype=torch.uint8, device=device)


def resblock_forward(x, params, y=None, cache=None, workspace=None, stream=None, events=None):
    """ResidualBlock forward of NDHWC bf16 x.

    params: a ResblockParams or a dict of device tensors.  cache: None for
    full-T, or a (convA_in, convB_in) pair of bf16 [B,2,H,W,C] tensors updated
    in place.  events: optional list of 4 torch.cuda.Event recorded around
    the kernels (see wanvae_resblock_forward_profiled)."""
    keep_alive = params  # the dict's tensors must outlive the allocations below
    if isinstance(params, dict):
        params = make_params(params)
    B, T, H, W, c_in = x.shape
    if y is None:
        y = torch.empty((B, T, H, W, params.c_out), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = make_workspace(x.shape, c_in, params.c_out, device=x.device)
    cs = None
    if cache is not None:
        cs = ctypes.byref(ResblockCache(cache[0].data_ptr(), cache[1].data_ptr()))
    L = load()
    if events is None:
        st = L.wanvae_resblock_forward(ctypes.byref(params), _ptr(x), _ptr(y), _dims(x.shape), cs,
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    else:
        for e in events:
            if not e.cuda_event:  # torch creates the CUDA event lazily
                e.record()
        ev = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
        st = L.wanvae_resblock_forward_profiled(ctypes.byref(params), _ptr(x), _ptr(y),
                                                _dims(x.shape), cs, _ptr(workspace),
                                                workspace.numel(), ev, _stream(stream))
    _check(st, "wanvae_resblock_forward")
    del keep_alive
    return y


def resblock_forward_host_workspace_size(dims, c_in, c_out, chunk_frames):
    return int(load().wanvae_resblock_forward_host_workspace_size(_dims(dims), c_in, c_out,
                                                                   chunk_frames))


def resblock_forward_host(x_host, params, y_host, chunk_frames, workspace, streams):
    """Whole-clip ResidualBlock forward of a clip in host memory (x_host, y_host:
    CPU bf16 tensors, pinned for the copies to overlap), as chunks of
    chunk_frames frames carried by the feat_cache and pipelined over
    streams = (compute, copy_in, copy_out).  Returns once enqueued; y_host is
    complete when streams[2] has drained."""
    keep_alive = params
    if isinstance(params, dict):
        params = make_params(params)
    sc, si, so = (ctypes.c_void_p(s.cuda_stream) for s in streams)
    st = load().wanvae_resblock_forward_host(ctypes.byref(params), _ptr(x_host), _ptr(y_host),
                                             _dims(x_host.shape), int(chunk_frames),
                                             _ptr(workspace), workspace.numel(), sc, si, so)
    _check(st, "wanvae_resblock_forward_host")
    del keep_alive
    return y_host


def resblock_forward_static(x, params, y, cache=None, stream=None):
    """resblock_forward with the library's own device workspace instead of a
    caller buffer, for callers that cannot allocate device memory where they
    run the block.  y must be given (nothing is allocated here either)."""
    keep_alive = params
    if isinstance(params, dict):
        params = make_params(params)
    cs = None
    if cache is not None:
        cs = ctypes.byref(ResblockCache(cache[0].data_ptr(), cache[1].data_ptr()))
    st = load().wanvae_resblock_forward_static(ctypes.byref(params), _ptr(x), _ptr(y),
                                               _dims(x.shape), cs, _stream(stream))
    _check(st, "wanvae_resblock_forward_static")
    del keep_alive
    return y


# ------------------------------------------------------------------ sequences
# These calls are short enough for their own overhead to count (a decoding
# step's kernels take a few microseconds each), so the checks ask each tensor
# for as little as they need.
def _fit(where, ok):
    """Refuse a call whose tensors do not fit it."""
    if not ok:
        raise WanvaeError(ERR_INVALID_ARG, where)


def _on_device(where, first, *tensors):
    """The current device's index, if every tensor (None: absent) lies there: its
    context is the one that the library launches in."""
    here = first.get_device()
    _fit(where, here >= 0 and here == torch.cuda.current_device())
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise WanvaeError(ERR_INVALID_ARG, where)
    return here


def _raw(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(where, stream, device):
    if stream is None:
        return _current_raw_stream(device)
    _fit(where, stream.device_index == device)
    return stream.cuda_stream


def _heads(where, t, dtype=torch.bfloat16):
    """Token stride of [tokens, heads, D] whose tokens are each contiguous."""
    if t.dtype != dtype or t.dim() != 3:
        raise WanvaeError(ERR_INVALID_ARG, where)
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if (h > 1 and sh != d) or (d > 1 and sd != 1):
        raise WanvaeError(ERR_INVALID_ARG, where)
    return sn if n > 1 else h * d  # (one token's stride means nothing)


def _ints(where, t, *shape):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise WanvaeError(ERR_INVALID_ARG, where)


def _on_stream(stream, make, *args, **kw):
    """make(..) out of the memory of the stream that the call works on: a block of the
    current stream's may still be in use there."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _result(stream, make, *args, **kw):
    """_on_stream for what is returned: its memory is not reused before the current stream
    is done with it."""
    t = _on_stream(stream, make, *args, **kw)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream())
    return t


def packed_attention(q, k, v, cu_q, cu_k=None, out=None, causal=True, scale=None, stream=None):
    """Attention over packed sequences of different lengths.  q [Tq, Hq, D], k
    and v [Tk, Hkv, D] bf16 (tokens may be strided, as slices of one projection
    are), cu_q and cu_k int32 [n + 1] offsets on the device (cu_k: cu_q unless
    given); causal: the last query of a sequence sees all of its keys.  Rows of
    `out` behind the last sequence are left as they were."""
    where = "wanvae_packed_attention"
    dev = _on_device(where, q, k, v, cu_q, cu_k, out)
    if out is None:
        out = _result(stream, torch.empty, q.shape, dtype=torch.bfloat16, device=q.device)
    n = cu_q.numel() - 1
    _ints(where, cu_q, n + 1)
    if cu_k is None:
        cu_k = cu_q
    else:
        _ints(where, cu_k, n + 1)
    qs, ks, vs, os_ = _heads(where, q), _heads(where, k), _heads(where, v), _heads(where, out)
    shape, kshape = q.shape, k.shape
    _fit(where, out.shape == shape and v.shape == kshape and shape[2] == kshape[2])
    Tq, Hq, D = shape
    st = load().wanvae_packed_attention(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, out.data_ptr(), os_,
        cu_q.data_ptr(), cu_k.data_ptr(), n, Tq, kshape[0], Hq, kshape[1], D,
        D ** -0.5 if scale is None else scale, 1 if causal else 0, _raw_stream(where, stream, dev))
    _check(st, where)
    return out


class KVCache:
    """A paged key-value cache over the caller's tensors: k and v
    [n_pages, Hkv, page_size, D], bf16; or float8_e4m3fn with k_exp and v_exp
    [n_pages, Hkv, page_size] (float8_e8m0fnu or uint8), one scale a row; or, in 4 bits,
    uint8 [n_pages, Hkv, page_size, D / 2] (two elements a byte, as include/wanvae.h lays
    them out) with k_exp and v_exp, and k_off and v_off uint8
    [n_pages, Hkv, page_size, D / 32]."""

    def __init__(self, k, v, k_exp=None, v_exp=None, k_off=None, v_off=None):
        where = "wanvae_kv_cache"
        _fit(where, k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and
             k.is_contiguous() and v.is_contiguous())
        kinds = {torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3, torch.uint8: E2M1}
        _fit(where, k.dtype in kinds)
        dt = kinds[k.dtype]
        n, self.heads, self.page_size, self.head_dim = k.shape
        if dt == E2M1:
            self.head_dim *= 2
        for e in (k_exp, v_exp):
            _fit(where, (e is not None) == (dt != BF16))
            _fit(where, e is None or (e.element_size() == 1 and e.is_contiguous() and
                                      e.shape == k.shape[:3]))
        for o in (k_off, v_off):
            _fit(where, (o is not None) == (dt == E2M1))
            _fit(where, o is None or (o.dtype == torch.uint8 and o.is_contiguous() and
                                      o.shape == (*k.shape[:3], self.head_dim // 32)))
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.k_off, self.v_off = k_off, v_off
        self.desc = KvCacheDesc(_raw(k), _raw(v), _raw(k_exp), _raw(v_exp), n, self.page_size,
                                self.heads, self.head_dim, dt, _raw(k_off), _raw(v_off))
        self.ref = ctypes.byref(self.desc)
        self.device = k.get_device()
        _fit(where, all(t is None or t.get_device() == self.device for t in self.tensors()))

    def tensors(self):
        held = self.k, self.v, self.k_exp, self.v_exp
        return held if self.k_off is None else (*held, self.k_off, self.v_off)


def make_kv_cache(n_pages, page_size, n_kv_heads, head_dim, dtype=torch.float8_e4m3fn,
                  device="cuda"):
    """An empty paged cache, in 8 bits (float8_e4m3fn), bf16, or 4 bits (uint8)."""
    rows = (n_pages, n_kv_heads, page_size)
    width = head_dim // 2 if dtype == torch.uint8 else head_dim
    k, v = (torch.zeros((*rows, width), dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype,
                        device=device).view(dtype) for _ in range(2))
    if dtype not in (torch.float8_e4m3fn, torch.uint8):
        return KVCache(k, v)
    # (the scales that rows of zeros are written with: 1, in 4 bits the smallest)
    zeros = 127 - 94 if dtype == torch.uint8 else 127
    ke, ve = (torch.full(rows, zeros, dtype=torch.uint8, device=device)
              .view(torch.float8_e8m0fnu) for _ in range(2))
    if dtype != torch.uint8:
        return KVCache(k, v, ke, ve)
    ko, vo = (torch.zeros((*rows, head_dim // 32), dtype=torch.uint8, device=device)
              for _ in range(2))
    return KVCache(k, v, ke, ve, ko, vo)


def kv_cache_append(cache, k, v, lens, page_table, cu_new=None, stream=None):
    """New rows k, v [T, Hkv, D] bf16 into the cache: the last positions of
    sequences whose lengths with them are lens (int32 [n], device).  cu_new
    int32 [n + 1]: sequence s has rows cu_new[s] .. cu_new[s + 1] - 1; None: one
    row a sequence.  page_table int32 [n, max_pages]."""
    where = "wanvae_kv_cache_append"
    dev = _on_device(where, k, v, lens, page_table, cu_new)
    ks, vs = _heads(where, k), _heads(where, v)
    T = k.shape[0]
    shape = (T, cache.heads, cache.head_dim)
    _fit(where, k.shape == shape and v.shape == shape and page_table.dim() == 2 and
         cache.device == dev)
    n, max_pages = page_table.shape
    _ints(where, lens, n)
    _ints(where, page_table, n, max_pages)
    if cu_new is not None:
        _ints(where, cu_new, n + 1)
    st = load().wanvae_kv_cache_append(cache.ref, k.data_ptr(), ks, v.data_ptr(), vs,
                                       lens.data_ptr(), page_table.data_ptr(), max_pages,
                                       _raw(cu_new), n, T, _raw_stream(where, stream, dev))
    _check(st, where)


def kv_cache_write(cache, k, v, slots, stream=None):
    """New rows k, v [T, Hkv, D] bf16 into the cache, row i into slot slots[i] (int64 [T],
    device, as kv_pages_extend gives them); below 0: not written."""
    where = "wanvae_kv_cache_write"
    dev = _on_device(where, k, v, slots)
    ks, vs = _heads(where, k), _heads(where, v)
    T = k.shape[0]
    shape = (T, cache.heads, cache.head_dim)
    _fit(where, k.shape == shape and v.shape == shape and cache.device == dev and
         slots.dtype == torch.int64 and slots.shape == (T,) and slots.is_contiguous())
    st = load().wanvae_kv_cache_write(cache.ref, k.data_ptr(), ks, v.data_ptr(), vs,
                                      slots.data_ptr(), T, _raw_stream(where, stream, dev))
    _check(st, where)


class KVPagePool:
    """The free pages of a cache over the caller's tensors: free int32 [n_pages], a stack of
    which the first n_free[0] (int32 [1]) are free.  A page is free or one sequence's: pages
    that several sequences read stay out of the pool (it counts no users)."""

    def __init__(self, free, n_free, page_size):
        where = "wanvae_kv_page_pool"
        _fit(where, free.dim() == 1)
        _ints(where, free, free.shape[0])
        _ints(where, n_free, 1)
        self.free, self.n_free, self.page_size = free, n_free, page_size
        self.desc = KvPagePoolDesc(_raw(free), _raw(n_free), free.shape[0], page_size)
        self.ref = ctypes.byref(self.desc)
        self.device = free.get_device()
        _fit(where, n_free.get_device() == self.device)


def make_kv_page_pool(n_pages, page_size, device="cuda"):
    """A pool of n_pages pages, all free; page 0 is taken first."""
    free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)
    return KVPagePool(free, torch.full((1,), n_pages, dtype=torch.int32, device=device), page_size)


def kv_pages_extend(pool, lens, n_new, page_table, total=None, lens_out=None, n_free_out=None,
                    cu_new=None, taken=None, positions=None, slots=None, stream=None):
    """Pages for n_new more tokens (int32 [n]) of sequences of lens positions (int32 [n]),
    off the pool and into page_table (int32 [n, max_pages]), and where the new tokens, packed
    into a batch of `total` rows, go: returns (lens_out, cu_new, taken, positions, slots)
    (include/wanvae.h).  lens_out and n_free_out: lens and the pool's count, in place,
    unless given.  total: positions' rows unless given."""
    where = "wanvae_kv_pages_extend"
    dev = _on_device(where, lens, n_new, page_table, lens_out, n_free_out, cu_new, taken,
                     positions, slots)
    _fit(where, page_table.dim() == 2 and pool.device == dev and
         (total is not None or positions is not None))
    n, max_pages = page_table.shape
    if total is None:
        total = positions.shape[0]

    def out(t, size, dtype=torch.int32):
        if t is None:
            return _result(stream, torch.empty, size, dtype=dtype, device=lens.device)
        _fit(where, t.dtype == dtype and t.shape == (size,) and t.is_contiguous())
        return t

    lens_out = lens if lens_out is None else lens_out
    n_free_out = pool.n_free if n_free_out is None else n_free_out
    cu_new, taken, positions = out(cu_new, n + 1), out(taken, n), out(positions, total)
    slots = out(slots, total, torch.int64)
    for t in (lens, n_new, lens_out):
        _ints(where, t, n)
    _ints(where, n_free_out, 1)
    _ints(where, page_table, n, max_pages)
    st = load().wanvae_kv_pages_extend(
        pool.ref, lens.data_ptr(), n_new.data_ptr(), page_table.data_ptr(), max_pages, n, total,
        lens_out.data_ptr(), n_free_out.data_ptr(), cu_new.data_ptr(), taken.data_ptr(),
        positions.data_ptr(), slots.data_ptr(), _raw_stream(where, stream, dev))
    _check(st, where)
    return lens_out, cu_new, taken, positions, slots


def kv_pages_release(pool, lens, done, page_table, lens_out=None, n_free_out=None, stream=None):
    """The pages of the sequences that are done (uint8 or bool [n], device) back to the pool;
    returns their lengths, 0 for those.  lens_out and n_free_out as for kv_pages_extend."""
    where = "wanvae_kv_pages_release"
    dev = _on_device(where, lens, done, page_table, lens_out, n_free_out)
    _fit(where, page_table.dim() == 2 and pool.device == dev)
    n, max_pages = page_table.shape
    lens_out = lens if lens_out is None else lens_out
    n_free_out = pool.n_free if n_free_out is None else n_free_out
    for t in (lens, lens_out):
        _ints(where, t, n)
    _ints(where, n_free_out, 1)
    _ints(where, page_table, n, max_pages)
    _fit(where, done.dtype in (torch.uint8, torch.bool) and done.shape == (n,) and
         done.is_contiguous())
    st = load().wanvae_kv_pages_release(
        pool.ref, lens.data_ptr(), done.data_ptr(), page_table.data_ptr(), max_pages, n,
        lens_out.data_ptr(), n_free_out.data_ptr(), _raw_stream(where, stream, dev))
    _check(st, where)
    return lens_out


class Rotary:
    """Which elements of a head turn with a token's position: pairs[a] pairs with position a
    (one number: one position a token), by inv_freq radians a position each (one for each
    pair in all; unless given theta ** (-i / pairs[a]) for the i-th pair of an axis).
    interleaved: the elements of a pair are neighbours, else half the turned elements apart."""

    def __init__(self, pairs, theta=10000.0, interleaved=False, inv_freq=None):
        where = "wanvae_rotary"
        self.pairs = [int(pairs)] if isinstance(pairs, int) else [int(n) for n in pairs]
        _fit(where, 1 <= len(self.pairs) <= 4 and min(self.pairs) >= 0)
        if inv_freq is None:
            inv_freq = [theta ** (-i / n) for n in self.pairs for i in range(n)]
        inv_freq = [float(f) for f in inv_freq]
        _fit(where, len(inv_freq) == sum(self.pairs))
        self.inv_freq = (ctypes.c_double * max(1, len(inv_freq)))(*inv_freq)
        self.interleaved = bool(interleaved)
        self.desc = RotaryDesc(self.inv_freq, len(self.pairs),
                               (ctypes.c_int64 * 4)(*self.pairs), 1 if interleaved else 0)
        self.ref = ctypes.byref(self.desc)


def qk_norm_rotate(q, k, positions, rotary, gamma_q=None, gamma_k=None, q_out=None, k_out=None,
                   eps=1e-12, stream=None):
    """RMS_norm of every head of q [T, Hq, D] and k [T, Hkv, D] (bf16 or fp32, tokens may be
    strided; k None: queries alone) and their rotation by positions (int32 [T] or
    [T, axes], device).  gamma_q, gamma_k fp32 [D]; None: no norm.  Returns (q_out, k_out);
    they may be q and k."""
    where = "wanvae_qk_norm_rotate"
    dev = _on_device(where, q, k, positions, gamma_q, gamma_k, q_out, k_out)
    dtype = q.dtype
    _fit(where, dtype == torch.bfloat16 or dtype == torch.float32)
    _fit(where, k is not None or (k_out is None and gamma_k is None))
    qs = _heads(where, q, dtype)
    T, Hq, D = q.shape
    if q_out is None:
        q_out = _result(stream, torch.empty, q.shape, dtype=dtype, device=q.device)
    _fit(where, q_out.shape == q.shape)
    qos = _heads(where, q_out, dtype)
    ks = kos = Hk = 0
    if k is not None:
        ks, Hk = _heads(where, k, dtype), k.shape[1]
        if k_out is None:
            k_out = _result(stream, torch.empty, k.shape, dtype=dtype, device=q.device)
        _fit(where, k.shape == (T, Hk, D) and k_out.shape == k.shape)
        kos = _heads(where, k_out, dtype)
    axes = len(rotary.pairs)
    if positions.dim() == 1:
        _fit(where, axes == 1)
        _ints(where, positions, T)
    else:
        _ints(where, positions, T, axes)
    for g in (gamma_q, gamma_k):
        if g is not None and (g.dtype != torch.float32 or g.shape != (D,) or
                              not g.is_contiguous()):
            raise WanvaeError(ERR_INVALID_ARG, where)
    st = load().wanvae_qk_norm_rotate(
        q.data_ptr(), qs, _raw(k), ks, _raw(gamma_q), _raw(gamma_k), rotary.ref,
        positions.data_ptr(), q_out.data_ptr(), qos, _raw(k_out), kos,
        BF16 if dtype == torch.bfloat16 else F32, T, Hq, Hk, D, eps,
        _raw_stream(where, stream, dev))
    _check(st, where)
    return q_out, k_out


def kv_cache_gather(cache, page_table, cu, k=None, v=None, total=None, stream=None):
    """The cache read back, packed: positions 0 .. of sequence s to the rows
    cu[s] .. cu[s + 1] - 1 of k and v [total, Hkv, D] bf16 (cu int32 [n + 1],
    device).  Without k and v, `total` rows are allocated."""
    where = "wanvae_kv_cache_gather"
    dev = _on_device(where, page_table, cu, k, v)
    if k is None or v is None:
        _fit(where, k is None and v is None and total is not None)
        k, v = (_result(stream, torch.empty, (total, cache.heads, cache.head_dim),
                        dtype=torch.bfloat16, device=page_table.device) for _ in range(2))
    ks, vs = _heads(where, k), _heads(where, v)
    T = k.shape[0]
    shape = (T, cache.heads, cache.head_dim)
    _fit(where, k.shape == shape and v.shape == shape and page_table.dim() == 2 and
         cache.device == dev)
    n, max_pages = page_table.shape
    _ints(where, cu, n + 1)
    _ints(where, page_table, n, max_pages)
    st = load().wanvae_kv_cache_gather(cache.ref, page_table.data_ptr(), max_pages, cu.data_ptr(),
                                       n, T, k.data_ptr(), ks, v.data_ptr(), vs,
                                       _raw_stream(where, stream, dev))
    _check(st, where)
    return k, v


def paged_attention_workspace_size(n_heads, n_kv_heads, head_dim):
    return int(load().wanvae_paged_attention_workspace_size(n_heads, n_kv_heads, head_dim))


def make_paged_attention_workspace(q, cache):
    """A workspace for paged_attention of q's heads over the cache."""
    n = paged_attention_workspace_size(q.shape[1], cache.heads, cache.head_dim)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def paged_attention(q, cache, lens, page_table, out=None, workspace=None, scale=None,
                    stream=None):
    """Attention of one new token for each sequence, q [n, Hq, D] bf16, over the
    first lens[s] positions of the cache (lens int32 [n], page_table int32
    [n, max_pages], device); zeros where lens[s] is 0."""
    where = "wanvae_paged_attention"
    dev = _on_device(where, q, lens, page_table, out, workspace)
    if out is None:
        out = _result(stream, torch.empty, q.shape, dtype=torch.bfloat16, device=q.device)
    if workspace is None:
        workspace = _on_stream(stream, make_paged_attention_workspace, q, cache)
    _fit(where, workspace.is_contiguous())
    qs, os_ = _heads(where, q), _heads(where, out)
    shape = q.shape
    n, Hq, D = shape
    _fit(where, out.shape == shape and D == cache.head_dim and page_table.dim() == 2 and
         cache.device == dev)
    max_pages = page_table.shape[1]
    _ints(where, lens, n)
    _ints(where, page_table, n, max_pages)
    st = load().wanvae_paged_attention(q.data_ptr(), qs, cache.ref, lens.data_ptr(),
                                       page_table.data_ptr(), max_pages, n, Hq,
                                       D ** -0.5 if scale is None else scale, out.data_ptr(), os_,
                                       workspace.data_ptr(), workspace.nbytes,
                                       _raw_stream(where, stream, dev))
    _check(st, where)
    return out


def gated_residual_norm(x, f, gamma_post=None, gate=None, gamma_pre=None, tokens_per_gate=1,
                        residual_scale=1.0, y=None, n=None, eps=1e-12, stream=None):
    """y = x + residual_scale * gate * RMS_norm(f; gamma_post) and, with
    gamma_pre, n = RMS_norm(y; gamma_pre), over the last axis of x and f (bf16
    or fp32, contiguous).  gate fp32 [G, C]: token i has row i // tokens_per_gate.
    Returns (y, n); n is None without gamma_pre."""
    where = "wanvae_gated_residual_norm"
    dev = _on_device(where, x, f, gamma_post, gate, gamma_pre, y, n)
    if y is None:
        y = _result(stream, torch.empty_like, x)
    if n is None and gamma_pre is not None:
        n = _result(stream, torch.empty_like, x)
    shape, dtype = x.shape, x.dtype
    _fit(where, (dtype == torch.bfloat16 or dtype == torch.float32) and x.is_contiguous())
    for t in (f, y, n):
        if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_contiguous()):
            raise WanvaeError(ERR_INVALID_ARG, where)
    C = shape[-1]
    tokens = x.numel() // C if C else 0
    for t in (gamma_post, gamma_pre):
        if t is not None and (t.dtype != torch.float32 or t.shape != (C,) or
                              not t.is_contiguous()):
            raise WanvaeError(ERR_INVALID_ARG, where)
    if gate is not None:
        _fit(where, gate.dtype == torch.float32 and gate.is_contiguous() and gate.dim() == 2 and
             gate.shape[1] == C and tokens_per_gate >= 1 and
             gate.shape[0] * tokens_per_gate >= tokens)
    st = load().wanvae_gated_residual_norm(
        x.data_ptr(), f.data_ptr(), _raw(gamma_post), _raw(gate), tokens_per_gate,
        _raw(gamma_pre), y.data_ptr(), _raw(n), BF16 if dtype == torch.bfloat16 else F32,
        tokens, C, residual_scale, eps, _raw_stream(where, stream, dev))
    _check(st, where)
    return y, n
