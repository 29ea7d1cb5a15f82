"""ctypes binding of libcc3d.so (the C ABI in include/cc3d.h).

Argument marshalling only: every step of the computation runs in the CUDA
library.  The raw entry points keep the C names (``cc3d_plan_create``,
``cc3d_forward``, ``rmsnorm_silu``, ``cc3d_block_create``,
``cc3d_resblock_forward``, ...).  ``Plan`` and ``Block`` wrap them for
torch tensors: they pass ``data_ptr()`` and the current CUDA stream, nothing
else.  Loading fails loudly when the library is missing -- there is no CPU
path.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libcc3d.so")

(OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_ALIAS, ERR_OOM, ERR_CUDA, ERR_TIMEOUT,
 ERR_TOO_LARGE) = range(9)
BF16, FP32, FP8_E4M3 = 0, 1, 2
EPI_BIAS, EPI_BIAS_RESIDUAL, EPI_BIAS_RMS_SILU, EPI_BIAS_RMS = 0, 1, 2, 3
ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3
VARIANT_NONE, VARIANT_UMMA, VARIANT_THIN, VARIANT_FP32 = 0, 1, 2, 3

_STATUS_NAMES = {0: "CC3D_OK", 1: "CC3D_ERR_INVALID_ARG", 2: "CC3D_ERR_UNSUPPORTED",
                 3: "CC3D_ERR_ALIGNMENT", 4: "CC3D_ERR_ALIAS", 5: "CC3D_ERR_OOM",
                 6: "CC3D_ERR_CUDA", 7: "CC3D_ERR_TIMEOUT", 8: "CC3D_ERR_TOO_LARGE"}


class Cc3dError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)} "
                         f"({lib().cc3d_status_string(status).decode()})")


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "n", "c_in", "c_out", "h", "w", "max_t", "kt", "kh", "kw", "pad_h", "pad_w",
        "stride_t", "stride_h", "stride_w", "dil_t", "dil_h", "dil_w", "groups", "dtype")] + [
        ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("epi", ctypes.c_int),
        ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("w_scale", ctypes.c_void_p),
        ("x_scale", ctypes.c_float)]


class Stats(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64), ("rejected", ctypes.c_uint64),
                ("tiles", ctypes.c_uint64), ("variant", ctypes.c_int), ("tile_h", ctypes.c_int),
                ("tile_w", ctypes.c_int), ("n_tile", ctypes.c_int), ("k_chunk", ctypes.c_int),
                ("k_split", ctypes.c_int), ("mma_ctas", ctypes.c_int),
                ("w_resident", ctypes.c_int), ("row_ctas", ctypes.c_int),
                ("one_frame_mma_ctas", ctypes.c_int), ("one_frame_n_tile", ctypes.c_int),
                ("second_tile_calls", ctypes.c_uint64)]


class HostCall(ctypes.Structure):
    _fields_ = [("x_host", ctypes.c_void_p), ("t", ctypes.c_int), ("cache_in", ctypes.c_void_p),
                ("cache_out", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("y_host", ctypes.c_void_p)]


# name -> (restype, argtypes)
_VP, _I = ctypes.c_void_p, ctypes.c_int
SIGNATURES = {
    "cc3d_plan_create": (_I, [ctypes.POINTER(Desc), ctypes.POINTER(_VP)]),
    "cc3d_plan_destroy": (_I, [_VP]),
    "cc3d_forward": (_I, [_VP, _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "cc3d_forward_host": (_I, [_VP, ctypes.POINTER(HostCall), _I, _VP]),
    "rmsnorm_silu": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP]),
    "rms_norm": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP]),
    "cc3d_quantize_e4m3": (_I, [_VP, ctypes.c_size_t, ctypes.c_float, _VP, _VP]),
    "cc3d_block_create": (_I, [_I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP,
                               ctypes.POINTER(_VP)]),
    "cc3d_block_create2": (_I, [_I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                ctypes.POINTER(_VP)]),
    "cc3d_block_destroy": (_I, [_VP]),
    "cc3d_resblock_forward": (_I, [_VP, _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP]),
    "cc3d_resblock_forward_fused": (_I, [_VP, _VP, _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                         _VP, _VP, _VP]),
    "cc3d_sync_status": (_I, [_VP]),
    "cc3d_get_stats": (_I, [_VP, ctypes.POINTER(Stats)]),
    "cc3d_status_string": (ctypes.c_char_p, [_I]),
    "cc3d_launch_count": (ctypes.c_uint64, []),
    "cc3d_forward_noalloc": (_I, [ctypes.POINTER(Desc), _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP,
                                  _VP]),
    "cc3d_add_rms_norm": (_I, [_VP, _VP]),
    "cc3d_linear": (_I, [_VP, _VP]),
    "cc3d_attention": (_I, [_VP, _VP]),
    "cc3d_kv_append": (_I, [_VP, _VP]),
}

_lib = None


def lib():
    """Load libcc3d.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m video_vae_causal_implicit_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def check(status, where):
    if status != OK:
        raise Cc3dError(status, where)


# Raw C entry points, same names as the header.
def cc3d_plan_create(desc, out):
    return lib().cc3d_plan_create(ctypes.byref(desc), ctypes.byref(out))


def cc3d_plan_destroy(plan):
    return lib().cc3d_plan_destroy(plan)


def cc3d_forward(plan, x, t, cache_in, y, cache_out, residual, next_cache_in, next_cache_out,
                 stream):
    return lib().cc3d_forward(plan, x, t, cache_in, y, cache_out, residual, next_cache_in,
                              next_cache_out, stream)


def cc3d_forward_host(plan, calls, ncalls, stream):
    return lib().cc3d_forward_host(plan, calls, ncalls, stream)


def rmsnorm_silu(x, gamma, beta, n, t, h, w, c, y, cache_in, cache_out, stream):
    return lib().rmsnorm_silu(x, gamma, beta, n, t, h, w, c, y, cache_in, cache_out, stream)


def rms_norm(x, gamma, beta, n, t, h, w, c, y, cache_in, cache_out, stream):
    return lib().rms_norm(x, gamma, beta, n, t, h, w, c, y, cache_in, cache_out, stream)


def cc3d_block_create(n, c, h, w, max_t, w1, b1, g1, w2, b2, g2, out):
    return lib().cc3d_block_create(n, c, h, w, max_t, w1, b1, g1, w2, b2, g2, ctypes.byref(out))


def cc3d_block_create2(n, c_in, c_out, h, w, max_t, w1, b1, g1, w2, b2, g2, w_sc, b_sc, out):
    return lib().cc3d_block_create2(n, c_in, c_out, h, w, max_t, w1, b1, g1, w2, b2, g2, w_sc,
                                    b_sc, ctypes.byref(out))


def cc3d_block_destroy(block):
    return lib().cc3d_block_destroy(block)


def cc3d_resblock_forward(block, x, t, cache1_in, cache2_in, y, cache1_out, cache2_out, stream):
    return lib().cc3d_resblock_forward(block, x, t, cache1_in, cache2_in, y, cache1_out,
                                       cache2_out, stream)


def cc3d_resblock_forward_fused(block, x, a0_in, t, cache1_in, cache2_in, y, cache1_out,
                                cache2_out, g_next, a0_next, a0_next_cache_in, a0_next_cache_out,
                                stream):
    return lib().cc3d_resblock_forward_fused(block, x, a0_in, t, cache1_in, cache2_in, y,
                                             cache1_out, cache2_out, g_next, a0_next,
                                             a0_next_cache_in, a0_next_cache_out, stream)


def cc3d_sync_status(stream):
    return lib().cc3d_sync_status(stream)


def cc3d_get_stats(plan, out):
    return lib().cc3d_get_stats(plan, ctypes.byref(out))


def cc3d_status_string(status):
    return lib().cc3d_status_string(status).decode()


def cc3d_launch_count():
    return int(lib().cc3d_launch_count())


def cc3d_forward_noalloc(desc, x, t, cache_in, y, cache_out, residual, next_cache_in,
                         next_cache_out, stream):
    """The conv without a plan and without device allocation (scratch is a
    fixed array inside the library; see include/cc3d.h)."""
    return lib().cc3d_forward_noalloc(ctypes.byref(desc), x, t, cache_in, y, cache_out, residual,
                                      next_cache_in, next_cache_out, stream)


# ---- torch conveniences (pointers + current stream only) --------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Plan:
    """A causal conv plan.  ``weight`` is [C_out, C_in, kt, kh, kw] on the
    device (bf16, or fp32 for dtype=FP32); bias/gamma/beta fp32 [C_out]."""

    def __init__(self, weight, bias=None, *, n=1, h, w, max_t, epi=EPI_BIAS, gamma=None,
                 beta=None, dtype=BF16, pad=None, stride_t=1, stride_hw=1, w_scale=None,
                 x_scale=0.0):
        co, ci, kt, kh, kw = (int(s) for s in weight.shape)
        d = Desc()
        d.n, d.c_in, d.c_out, d.h, d.w, d.max_t = n, ci, co, h, w, max_t
        d.kt, d.kh, d.kw = kt, kh, kw
        d.pad_h, d.pad_w = pad if pad is not None else (kh // 2, kw // 2)
        d.stride_t = stride_t
        d.stride_h = d.stride_w = stride_hw
        d.dil_t = d.dil_h = d.dil_w = 1
        d.groups = 1
        d.dtype = dtype
        weight = weight.contiguous()
        d.weight = weight.data_ptr()
        d.bias = bias.data_ptr() if bias is not None else None
        d.epi = epi
        d.gamma = gamma.data_ptr() if gamma is not None else None
        d.beta = beta.data_ptr() if beta is not None else None
        d.w_scale = w_scale.data_ptr() if w_scale is not None else None
        d.x_scale = float(x_scale)
        self.desc = d
        self.handle = ctypes.c_void_p()
        check(cc3d_plan_create(d, self.handle), "cc3d_plan_create")

    def forward(self, x, y, t=None, cache_in=None, cache_out=None, residual=None,
                next_cache_in=None, next_cache_out=None, stream=None):
        t = int(x.shape[1]) if t is None else t
        check(cc3d_forward(self.handle, _ptr(x), t, _ptr(cache_in), _ptr(y), _ptr(cache_out),
                           _ptr(residual), _ptr(next_cache_in), _ptr(next_cache_out),
                           _stream(stream)), "cc3d_forward")
        return y

    def forward_host(self, calls, stream=None):
        """cc3d_forward_host: ``calls`` is a list of dicts with x_host and
        y_host (host tensors, pinned for overlap) and optionally t,
        cache_in, cache_out, residual (device tensors)."""
        arr = (HostCall * len(calls))()
        for i, c in enumerate(calls):
            arr[i].x_host = c["x_host"].data_ptr()
            arr[i].t = int(c.get("t", c["x_host"].shape[1]))
            for k in ("cache_in", "cache_out", "residual"):
                v = c.get(k)
                setattr(arr[i], k, v.data_ptr() if v is not None else None)
            arr[i].y_host = c["y_host"].data_ptr()
        check(cc3d_forward_host(self.handle, arr, len(calls), _stream(stream)),
              "cc3d_forward_host")

    def stats(self):
        s = Stats()
        check(cc3d_get_stats(self.handle, s), "cc3d_get_stats")
        return s

    def close(self):
        if self.handle:
            cc3d_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Block:
    """Residual block, 3x3x3 convs, from C_in = w1.shape[1] to C_out =
    w1.shape[0] channels; w_sc [C_out, C_in, 1, 1, 1] (+ b_sc) is the
    1x1x1 conv_shortcut (None: the identity shortcut, C_in == C_out).

    In a chain of blocks, ``forward(..., g_next=next_block.g1, a0_next=A)``
    also writes the next block's first activation SiLU(RMS_norm(y; g_next))
    to A (from this block's conv2 epilogue), and the next block takes it as
    ``forward(y, ..., a0_in=A)``, skipping its own first norm."""

    def __init__(self, w1, b1, g1, w2, b2, g2, *, n=1, h, w, max_t, w_sc=None, b_sc=None):
        self.c_out, self.c_in = int(w1.shape[0]), int(w1.shape[1])
        self.c = self.c_out
        keep = [None if t is None else t.contiguous() for t in (w1, b1, g1, w2, b2, g2, w_sc, b_sc)]
        self.g1 = keep[2].float().contiguous()  # (the previous block's g_next)
        self.handle = ctypes.c_void_p()
        check(cc3d_block_create2(n, self.c_in, self.c_out, h, w, max_t,
                                 *(_ptr(t) for t in keep), self.handle),
              "cc3d_block_create2")

    def forward(self, x, y, t=None, cache1_in=None, cache2_in=None, cache1_out=None,
                cache2_out=None, stream=None, a0_in=None, g_next=None, a0_next=None,
                a0_next_cache_in=None, a0_next_cache_out=None):
        t = int(x.shape[1]) if t is None else t
        if a0_in is None and g_next is None and a0_next is None:
            check(cc3d_resblock_forward(self.handle, _ptr(x), t, _ptr(cache1_in),
                                        _ptr(cache2_in), _ptr(y), _ptr(cache1_out),
                                        _ptr(cache2_out), _stream(stream)),
                  "cc3d_resblock_forward")
            return y
        check(cc3d_resblock_forward_fused(self.handle, _ptr(x), _ptr(a0_in), t, _ptr(cache1_in),
                                          _ptr(cache2_in), _ptr(y), _ptr(cache1_out),
                                          _ptr(cache2_out), _ptr(g_next), _ptr(a0_next),
                                          _ptr(a0_next_cache_in), _ptr(a0_next_cache_out),
                                          _stream(stream)),
              "cc3d_resblock_forward_fused")
        return y

    def close(self):
        if self.handle:
            cc3d_block_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rms_silu(x, gamma, y, beta=None, cache_in=None, cache_out=None, stream=None):
    n, t, h, w, c = (int(s) for s in x.shape)
    check(rmsnorm_silu(_ptr(x), _ptr(gamma), _ptr(beta), n, t, h, w, c, _ptr(y), _ptr(cache_in),
                       _ptr(cache_out), _stream(stream)), "rmsnorm_silu")
    return y


def rms(x, gamma, y, beta=None, cache_in=None, cache_out=None, stream=None):
    """The RMS_norm alone (no SiLU)."""
    n, t, h, w, c = (int(s) for s in x.shape)
    check(rms_norm(_ptr(x), _ptr(gamma), _ptr(beta), n, t, h, w, c, _ptr(y), _ptr(cache_in),
                   _ptr(cache_out), _stream(stream)), "rms_norm")
    return y


def quantize_e4m3(x, scale, q, stream=None):
    """q (uint8, same element count as the bf16 tensor x) = E4M3(x / scale)."""
    check(lib().cc3d_quantize_e4m3(_ptr(x), x.numel(), float(scale), _ptr(q), _stream(stream)),
          "cc3d_quantize_e4m3")
    return q


# ---- transformer operators ---------------------------------------------------------
#
# The C calls see addresses only, so these wrappers check what the addresses
# stand for: type, device (the current one), shape and strides.  A small call
# takes as long as its checks, so each is one expression and the reasons are
# worked out only for a tensor that fails it.

# The calls' argument structs as the C compiler lays them out (packing one is
# a third of the time that as many ctypes arguments take)
_NORM_CALL = struct.Struct("@8Pq2i2f")
_LINEAR_CALL = struct.Struct("@7P5q4if4x")
_ATTN_CALL = struct.Struct("@11if6P12q")
_KV_CALL = struct.Struct("@9i6P12q")

_torch = None  # torch and the types of the operators, on first use
_B16 = _F32 = _B8 = _I32 = ()


def _load_torch():
    global _torch, _B16, _F32, _B8, _I32
    import torch
    _B16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
    _B8 = (torch.float8_e4m3fn, torch.uint8)
    _torch = torch


def _current(t, name, stream):
    """(device index, raw stream) of a call whose first tensor is `t`."""
    if _torch is None:
        _load_torch()
    dev = t.get_device()
    if dev < 0 or dev != _torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if stream is None:
        return dev, _torch._C._cuda_getCurrentRawStream(dev)
    return dev, stream.cuda_stream


def _refuse(t, name, dtypes, dev, shape):
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: strides {t.stride()} of shape {tuple(t.shape)}; contiguous "
                     "elements (or rows, where rows may be strided) expected")


def _flat(t, name, dtypes, dev, shape):
    """The address of a contiguous tensor, checked (None: 0)."""
    if t is None:
        return 0
    if (t.dtype not in dtypes or t.get_device() != dev or t.shape != shape
            or not t.is_contiguous()):
        _refuse(t, name, dtypes, dev, shape)
    return t.data_ptr()


def _rows(t, name, dtypes, dev, shape):
    """(address, distance of rows) of a matrix with contiguous rows, checked."""
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != shape or len(shape) != 2:
        _refuse(t, name, dtypes, dev, shape)
    step, one = t.stride()
    if one != 1 and shape[1] > 1:
        _refuse(t, name, dtypes, dev, shape)
    # (the distance of a single row is free: any legal one will do)
    return t.data_ptr(), step if shape[0] > 1 else shape[1]


def linear(x, weight, y, *, bias=None, residual=None, act=ACT_NONE, x_scales=None, w_scales=None,
           x_scale=0.0, stream=None):
    """y = act(x @ weight.T (scaled) + bias) + residual (cc3d_linear).

    x [m, k] and weight [n, k] are bf16, or both E4M3 codes (float8_e4m3fn or
    uint8) with w_scales [n] and x_scales [m] (or one x_scale); bias fp32 [n];
    residual and y bf16 [m, n] (y may be the residual).  Rows may be strided."""
    dev, st = _current(x, "x", stream)
    fp8 = x.dtype in _B8
    ops = _B8 if fp8 else _B16
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x [m, k] and weight [n, k] expected")
    m, k = x.shape
    n = weight.shape[0]
    px, ldx = _rows(x, "x", ops, dev, x.shape)
    pw, ldw = _rows(weight, "weight", ops, dev, (n, k))
    py, ldy = _rows(y, "y", _B16, dev, (m, n))
    pr, ldr = _rows(residual, "residual", _B16, dev, (m, n)) if residual is not None else (0, 0)
    check((_lib or lib()).cc3d_linear(
        _LINEAR_CALL.pack(px, pw, _flat(bias, "bias", _F32, dev, (n,)), pr, py,
                          _flat(x_scales, "x_scales", _F32, dev, (m,)),
                          _flat(w_scales, "w_scales", _F32, dev, (n,)), ldx, ldw, ldr, ldy, m, n,
                          k, FP8_E4M3 if fp8 else BF16, act, x_scale), st), "cc3d_linear")
    return y


def add_rms_norm(x, gamma, *, residual=None, beta=None, eps=0.0, silu=False, h=None, y=None,
                 q=None, scales=None, scale=0.0, stream=None):
    """RMS norm of x (+ residual) over the last dimension, with an output in
    16 bits (y), in E4M3 (q, with row scales written to `scales` or one given
    `scale`), and the sum itself (h); see cc3d_add_rms_norm.  Outputs are the
    tensors given; returns None."""
    dev, st = _current(x, "x", stream)
    shape = x.shape
    c = shape[-1]
    rows = x.numel() // c if c else 0
    check((_lib or lib()).cc3d_add_rms_norm(
        _NORM_CALL.pack(_flat(x, "x", _B16, dev, shape),
                        _flat(residual, "residual", _B16, dev, shape),
                        _flat(gamma, "gamma", _F32, dev, (c,)),
                        _flat(beta, "beta", _F32, dev, (c,)), _flat(h, "h", _B16, dev, shape),
                        _flat(y, "y", _B16, dev, shape), _flat(q, "q", _B8, dev, shape),
                        _flat(scales, "scales", _F32, dev, shape[:-1]) if scales is not None else 0,
                        rows, c, 1 if silu else 0, eps, scale), st), "cc3d_add_rms_norm")


def _heads(t, name, dev, shape, frame):
    """(address, strides of sequences, tokens and heads) of a [n, tokens,
    heads, d] bf16 tensor with a contiguous last dimension, checked."""
    if t.dtype not in _B16 or t.get_device() != dev or t.shape != shape or len(shape) != 4:
        _refuse(t, name, _B16, dev, shape)
    a, b, c, one = t.stride()
    if (one != 1 and shape[3] > 1) or shape[1] % frame:
        if shape[1] % frame == 0:
            _refuse(t, name, _B16, dev, shape)
        raise ValueError(f"{name}: {shape[1]} tokens are not whole frames of {frame}")
    return t.data_ptr(), a, b, c


def _lengths(n, frame, total, q_frames, k_frames, dev):
    if frame < 1:
        raise ValueError(f"frame: {frame}")
    if k_frames is None:
        if total is None:
            raise ValueError("total or k_frames is needed")
    elif total is None:
        total = 0
    return (total, _flat(q_frames, "q_frames", _I32, dev, (n,)),
            _flat(k_frames, "k_frames", _I32, dev, (n,)))


def attention(q, k, v, o, *, frame=1, window=0, sinks=0, ring=0, total=None, q_frames=None,
              k_frames=None, scale=0.0, stream=None):
    """Attention in a sliding window of frames with sink frames
    (cc3d_attention): q and o [n, t * frame, heads, d], k and v caches
    [n, slots * frame, kv_heads, d], bf16, any strides with a contiguous last
    dimension.  total: frames of every sequence, this chunk included, or
    k_frames (int32 [n], device) one count each; window 0: unlimited."""
    dev, st = _current(q, "q", stream)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q [n, tokens, heads, d] and k [n, tokens, kv_heads, d] expected")
    n, qt, heads, d = q.shape
    _, kt, kv_heads, _ = k.shape
    total, pqf, pkf = _lengths(n, frame, total, q_frames, k_frames, dev)
    cache = (n, kt, kv_heads, d)
    pq, q0, q1, q2 = _heads(q, "q", dev, q.shape, frame)
    pk, k0, k1, k2 = _heads(k, "k", dev, cache, frame)
    pv, v0, v1, v2 = _heads(v, "v", dev, cache, frame)
    po, o0, o1, o2 = _heads(o, "o", dev, q.shape, frame)
    check((_lib or lib()).cc3d_attention(
        _ATTN_CALL.pack(n, heads, kv_heads, d, frame, qt // frame, kt // frame, window, sinks,
                        ring, total, scale, pqf, pkf, pq, pk, pv, po, q0, q1, q2, k0, k1, k2, v0,
                        v1, v2, o0, o1, o2), st), "cc3d_attention")
    return o


def kv_append(k, v, k_cache, v_cache, *, frame=1, sinks=0, ring=0, total=None, q_frames=None,
              k_frames=None, stream=None):
    """A chunk's keys and values [n, t * frame, kv_heads, d] into the caches
    [n, slots * frame, kv_heads, d] (cc3d_kv_append); frame counts as in
    attention, the chunk included."""
    dev, st = _current(k, "k", stream)
    if k.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("k and k_cache [n, tokens, kv_heads, d] expected")
    n, kt, heads, d = k.shape
    ct = k_cache.shape[1]
    total, pqf, pkf = _lengths(n, frame, total, q_frames, k_frames, dev)
    cache = (n, ct, heads, d)
    pk, k0, k1, k2 = _heads(k, "k", dev, k.shape, frame)
    pv, v0, v1, v2 = _heads(v, "v", dev, k.shape, frame)
    pkc, kc0, kc1, kc2 = _heads(k_cache, "k_cache", dev, cache, frame)
    pvc, vc0, vc1, vc2 = _heads(v_cache, "v_cache", dev, cache, frame)
    check((_lib or lib()).cc3d_kv_append(
        _KV_CALL.pack(n, heads, d, frame, kt // frame, ct // frame, sinks, ring, total, pqf, pkf,
                      pk, pv, pkc, pvc, k0, k1, k2, v0, v1, v2, kc0, kc1, kc2, vc0, vc1, vc2),
        st), "cc3d_kv_append")


def sync_status(stream=None):
    check(cc3d_sync_status(_stream(stream)), "cc3d_sync_status")
