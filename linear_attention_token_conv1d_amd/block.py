"""The operators around the mixer in a hybrid block.

As in the package itself, these functions only marshal arguments, here in
C++ (csrc/binding.cpp: a call of one token takes less time than its checks
would in Python): torch-level properties (device, dtype, strides) are checked
there, everything else by the library, and every step of the computation runs
in its HIP kernels.  A call's tensors lie on one GPU; the call runs on torch's
current stream of that GPU, which need not be the current device.

The ctypes structs are those of include/gdn.h, for callers that make the C
calls themselves.
"""
from __future__ import annotations

import collections
import ctypes
import math

import torch

from . import BF16, F32, GdnError, _c_void_p, lib

_DT = {torch.float32: F32, torch.bfloat16: BF16}
_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class NormArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", _i32), ("weight_dtype", _i32), ("order", _i32),
                ("activation", _i32), ("heads", _i32), ("width", _i32), ("eps", _f32), ("scale", _f32),
                ("weight_offset", _f32), ("tokens", _i64), ("x", _c_void_p), ("weight", _c_void_p),
                ("gate", _c_void_p), ("residual", _c_void_p), ("y", _c_void_p), ("sum", _c_void_p),
                ("x_stride", _i64), ("gate_stride", _i64), ("residual_stride", _i64), ("y_stride", _i64),
                ("sum_stride", _i64)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", _i32), ("weight_dtype", _i32), ("order", _i32),
                ("activation", _i32), ("heads", _i32), ("width", _i32), ("eps", _f32), ("scale", _f32),
                ("weight_offset", _f32), ("tokens", _i64), ("x", _c_void_p), ("weight", _c_void_p),
                ("gate", _c_void_p), ("dy", _c_void_p), ("d_sum", _c_void_p), ("dx", _c_void_p),
                ("d_residual", _c_void_p), ("dgate", _c_void_p), ("dweight", _c_void_p), ("x_stride", _i64),
                ("gate_stride", _i64), ("dy_stride", _i64), ("d_sum_stride", _i64), ("dx_stride", _i64),
                ("d_residual_stride", _i64), ("dgate_stride", _i64), ("workspace", _c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", _i32), ("layout", _i32), ("inverse", _i32),
                ("position_bits", _i32), ("h_q", _i32), ("h_k", _i32), ("d", _i32), ("rot", _i32), ("mscale", _f32),
                ("tokens", _i64), ("q", _c_void_p), ("k", _c_void_p), ("positions", _c_void_p), ("inv_freq", _c_void_p),
                ("q_out", _c_void_p), ("k_out", _c_void_p), ("q_stride", _i64), ("k_stride", _i64),
                ("q_out_stride", _i64), ("k_out_stride", _i64)]


class CacheStoreArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("io_dtype", _i32), ("n_seqs", _i32), ("h_kv", _i32), ("d", _i32),
                ("page_size", _i32), ("pages", _i32), ("max_pages", _i32), ("tokens", _i64), ("k", _c_void_p),
                ("v", _c_void_p), ("k_stride", _i64), ("v_stride", _i64), ("k_cache", _c_void_p), ("v_cache", _c_void_p),
                ("k_scale", _c_void_p), ("v_scale", _c_void_p), ("page_table", _c_void_p), ("lens", _c_void_p),
                ("cu_seqlens", _c_void_p)]


class CacheAttentionArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("io_dtype", _i32), ("n_seqs", _i32), ("h_q", _i32), ("h_kv", _i32),
                ("d", _i32), ("page_size", _i32), ("pages", _i32), ("max_pages", _i32), ("causal", _i32),
                ("window", _i32), ("scale", _f32), ("tokens", _i64), ("q", _c_void_p), ("gate", _c_void_p),
                ("o", _c_void_p), ("q_stride", _i64), ("gate_stride", _i64), ("o_stride", _i64), ("lse", _c_void_p),
                ("k_cache", _c_void_p), ("v_cache", _c_void_p), ("k_scale", _c_void_p), ("v_scale", _c_void_p),
                ("page_table", _c_void_p), ("lens", _c_void_p), ("cu_seqlens", _c_void_p), ("workspace", _c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


def declare(L):
    """Argument types of this module's entry points in the loaded library."""
    for name, argt in (("gdn_rms_norm", NormArgs), ("gdn_rms_norm_backward", NormBwdArgs), ("gdn_rope", RopeArgs),
                       ("gdn_cache_store", CacheStoreArgs), ("gdn_cache_attention", CacheAttentionArgs)):
        f = getattr(L, name)
        f.argtypes = [ctypes.POINTER(argt), _c_void_p]
        f.restype = ctypes.c_int
    for name, argt in (("gdn_rms_norm_backward_workspace_size", NormBwdArgs),
                       ("gdn_cache_attention_workspace_size", CacheAttentionArgs)):
        f = getattr(L, name)
        f.argtypes = [ctypes.POINTER(argt)]
        f.restype = ctypes.c_size_t


_native = None


def _bound():
    """The compiled binding (raises GdnError when it, or libgdn.so, is missing)."""
    global _native
    if _native is None:
        lib()
        try:
            from . import _binding
        except ImportError as e:
            raise GdnError(f"_binding.so is not built or does not load ({e}); run python -m linear_attention_token_conv1d_amd._build")
        _binding.init(GdnError, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch._C._cuda_setDevice)
        _native = _binding
    return _native


def rms_norm(x, weight=None, gate=None, residual=None, order="pre", activation="silu", scale=1.0, eps=1e-6,
             weight_offset=0.0, out=None, sum_out=None):
    """RMS norm over the last dimension of x [T, D] or [T, H, D] (bf16 or fp32,
    token stride free), fused with the residual sum and the output gate.

    order="pre":  h = residual + scale * x; returns (y, h) with a residual, y
    without one, where y = norm(h) * (weight + weight_offset) * act(gate).
    order="post": returns y = residual + scale * norm(x) * (weight + weight_offset) * act(gate).

    weight [D] (bf16 or fp32), gate and residual (like x) are optional;
    activation is "silu" or "sigmoid".  out and sum_out may be given, also as
    the input they replace (in place)."""
    return (_native or _bound()).rms_norm(x, weight, gate, residual, order, activation, scale, eps, weight_offset, out, sum_out)


def rms_norm_backward(x, dy, weight=None, gate=None, d_sum=None, residual=False, order="pre", activation="silu",
                      scale=1.0, eps=1e-6, weight_offset=0.0, dx=None, dgate=None, workspace=None):
    """Gradients of rms_norm: returns (dx, dresidual, dweight, dgate).

    x is what was normed: the forward call's x, or the sum h that it returned
    (residual=True, or d_sum, the gradient that reaches h from its other uses,
    say so).  dx is the gradient of the forward call's x; dresidual that of
    the residual (None without one; in the post order it is dy itself and
    None here; with scale 1 it is the same tensor as dx).  dweight is fp32
    [D] (None without a weight), dgate like x (None without a gate)."""
    return (_native or _bound()).rms_norm_backward(x, dy, weight, gate, d_sum, residual, order, activation, scale, eps, weight_offset, dx,
                                                   dgate, workspace)


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=None, low=1.0, high=32.0, device=None):
    """Radians a position for each of the rot / 2 pairs of a rotated head, fp64
    [rot / 2], and the factor on the cosines and sines (rope's inv_freq and
    mscale).

    scaling=None: base^(-2 i / rot).  For contexts `factor` times longer:
    "linear" divides every frequency by factor; "ntk" raises the base so that
    the slowest pair is divided by it and the fastest keeps its frequency;
    "by_parts" keeps pairs that turn more than `high` times over the original
    context, divides those that turn less than `low` times, blends between,
    and returns the factor 0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise GdnError(f"rot must be even and positive, got {rot}")
    if not factor >= 1.0:
        raise GdnError(f"factor must be at least 1, got {factor}")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    f = float(base) ** (-2 * i / rot)
    m = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if not original or not 0 < low < high:
            raise GdnError("by_parts needs the original context length and 0 < low < high")
        turns = original * f / (2 * math.pi)
        kept = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * kept + f / factor * (1 - kept)
        m = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise GdnError(f"scaling must be None, 'linear', 'ntk' or 'by_parts', got {scaling!r}")
    return f.to(device) if device is not None else f, m


def rope(q, positions, inv_freq, k=None, layout="half", mscale=1.0, out=None, k_out=None):
    """Rotary positions on the heads of q [T, H, d], and of k [T, H_k, d] in the
    same launch (bf16 or fp32, token stride free): returns q' or (q', k').

    positions [T] (int32 or int64) are the tokens' positions, inv_freq
    [rot / 2] fp64 the radians a position of each pair (rope_frequencies);
    rot may be less than d: the rest of a head passes through.  layout "half"
    pairs elements i and i + rot / 2, "interleaved" 2 i and 2 i + 1.  out and
    k_out may be q and k themselves (in place)."""
    return (_native or _bound()).rope(q, positions, inv_freq, k, layout, mscale, False, out, k_out)


def rope_backward(dq, positions, inv_freq, k=None, layout="half", mscale=1.0, out=None, k_out=None):
    """Gradients of rope's inputs given those of its outputs (dq, and k: that of
    k'): the rotation by the opposite angle.  Arguments as in rope."""
    return (_native or _bound()).rope(dq, positions, inv_freq, k, layout, mscale, True, out, k_out)


FP8 = torch.float8_e4m3fn
KVCache = collections.namedtuple("KVCache", "k v k_scale v_scale")


def kv_cache(pages, h_kv, d, page_size=64, device="cuda"):
    """An empty pool of pages: e4m3 keys [pages, h_kv, page_size, d] and values
    [pages, h_kv, d, page_size], and their fp32 scales [pages, h_kv]."""
    def new(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)

    return KVCache(new(pages, h_kv, page_size, d, dtype=torch.uint8).view(FP8), new(pages, h_kv, d, page_size, dtype=torch.uint8).view(FP8),
                   new(pages, h_kv, dtype=torch.float32), new(pages, h_kv, dtype=torch.float32))


def cache_store(k, v, cache, page_table, lens, cu_seqlens=None):
    """Store new keys and values [T, H_kv, d] (bf16 or fp32, token stride free)
    in the pages of `cache` (kv_cache), in place.

    page_table [N, M] int32 names the pages of each sequence, lens [N] int32
    the tokens it held before.  cu_seqlens [N + 1] int32 are the offsets of
    each sequence's new tokens; without it each has T / N.  Each page and head
    gets the least power of two as its scale that holds its largest value; a
    page that holds older tokens keeps a larger scale, or has them rounded
    anew by the new one.  Tokens behind the table or on a page outside the
    pool (say -1) are not stored."""
    (_native or _bound()).cache_store(k, v, cache, page_table, lens, cu_seqlens)


def cache_attention(q, cache, page_table, lens, cu_seqlens=None, scale=None, causal=True, window=0, gate=None, out=None,
                    return_lse=False, workspace=None):
    """Attention of each sequence's newest tokens q [T, H_q, d] over its pages of
    `cache`, where their own keys and values lie already (cache_store).

    lens [N] int32 counts the tokens in the cache, the new ones among them;
    cu_seqlens [N + 1] int32 are the offsets of the new tokens (T / N each
    without it).  scale is d^-1/2 by default.  causal: a token sees positions
    up to its own; window > 0: only those above its own minus window.  gate
    (like q) multiplies the output by its sigmoid.  Returns o like q, or
    (o, lse [T, H_q] fp32) with return_lse; a token that sees nothing gives
    zeros and -inf.  Rows behind the last sequence of a padded batch are not
    written."""
    return (_native or _bound()).cache_attention(q, cache, page_table, lens, cu_seqlens, scale, causal, window, gate, out, return_lse,
                                                 workspace)


def cache_attention_workspace_size(tokens, n_seqs, max_pages, h_q, h_kv, d, page_size=64, ragged=False, dtype=torch.bfloat16,
                                   causal=True, window=0):
    """Bytes of workspace that cache_attention needs with these arguments (0: none), for a caller that keeps one."""
    a = CacheAttentionArgs(struct_size=ctypes.sizeof(CacheAttentionArgs), io_dtype=_DT[dtype], n_seqs=n_seqs, h_q=h_q, h_kv=h_kv, d=d, page_size=page_size,
                           max_pages=max_pages, tokens=tokens, cu_seqlens=1 if ragged else None, causal=int(bool(causal)), window=window)
    return lib().gdn_cache_attention_workspace_size(a)
