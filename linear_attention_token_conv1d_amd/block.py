"""The operators around the mixer in a hybrid block.

As in the package itself, these functions only marshal arguments: torch-level
properties (device, dtype, strides) are checked here, everything else by the
library, and every step of the computation runs in its HIP kernels.  A call's
tensors lie on one GPU; the call runs on torch's current stream of that GPU,
which need not be the current device.
"""
from __future__ import annotations

import collections
import ctypes
import math

import torch

from . import BF16, F32, GdnError, _c_void_p, lib

ACT = {"silu": 1, "sigmoid": 2}
ORDER = {"pre": 0, "post": 1}
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


_SIZE = {c: ctypes.sizeof(c) for c in (NormArgs, NormBwdArgs, RopeArgs, CacheStoreArgs, CacheAttentionArgs)}
_stream_of = torch._C._cuda_getCurrentRawStream
_device_now = torch._C._cuda_getDevice
_entries = {}


def _entry(name):
    f = _entries.get(name)
    if f is None:
        f = _entries[name] = getattr(lib(), name)
    return f


def _run(name, args, index):
    """Call an entry point on the current stream of GPU `index`."""
    f = _entry(name)
    if index == _device_now():
        status = f(args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            status = f(args, _stream_of(index))
    if status:
        L = lib()
        raise GdnError(f"{name}: {L.gdn_status_string(status).decode()}: {L.gdn_last_error().decode()}")


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdnError(f"{name} must be a GPU tensor")
    return t.get_device()


def _wrong(t, name, index, shape, dtype):
    """What is wrong with a tensor that is not on GPU `index`, or not of this dtype or shape."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        return GdnError(f"{name} must be on the same GPU as the call's other tensors")
    if t.dtype != dtype:
        return GdnError(f"{name} must be {dtype}, got {t.dtype}")
    return GdnError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _tensor(t, name, index, shape, dtype):
    """An optional contiguous tensor of exactly this shape and dtype on GPU `index`: its address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        raise _wrong(t, name, index, shape, dtype)
    if not t.is_contiguous():
        raise GdnError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, index, shape, dtype):
    """An optional [T, H, d] or [T, d] tensor, token stride free: its address and token stride."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        raise _wrong(t, name, index, shape, dtype)
    if t.is_contiguous():
        return t.data_ptr(), shape[1] if len(shape) == 2 else shape[1] * shape[2]
    s = t.stride()
    # a stride over one element says nothing about the layout
    if (s[-1] != 1 and shape[-1] > 1) or (len(s) == 3 and s[1] != shape[2] and shape[1] > 1):
        raise GdnError(f"{name} must have contiguous heads inside a token")
    return t.data_ptr(), s[0]


def _norm_shape(x):
    index = _gpu(x, "x")
    if x.dtype not in _DT:
        raise GdnError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    if x.dim() not in (2, 3):
        raise GdnError("x must be [T, D] or [T, H, D]")
    return index, x.shape, (x.shape[1] if x.dim() == 3 else 1), x.shape[-1]


def _norm_how(weight, gate, order, activation):
    if order not in ORDER:
        raise GdnError(f"order must be 'pre' or 'post', got {order!r}")
    if gate is not None and activation not in ACT:
        raise GdnError(f"activation must be 'silu' or 'sigmoid', got {activation!r}")
    if weight is not None and (not isinstance(weight, torch.Tensor) or weight.dtype not in _DT):
        raise GdnError("weight must be a torch.bfloat16 or torch.float32 tensor")
    return ORDER[order], ACT[activation] if gate is not None else 0


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
    index, shape, heads, width = _norm_shape(x)
    order, act = _norm_how(weight, gate, order, activation)
    dt = x.dtype
    y = torch.empty_like(x) if out is None else out
    sums = residual is not None and order == 0
    if sums and sum_out is None:
        sum_out = torch.empty_like(residual)
    if not sums and sum_out is not None:
        raise GdnError("sum_out goes with a residual in the pre order")
    px, sx = _rows(x, "x", index, shape, dt)
    pg, sg = _rows(gate, "gate", index, shape, dt)
    pr, sr = _rows(residual, "residual", index, shape, dt)
    py, sy = _rows(y, "out", index, shape, dt)
    ps, ss = _rows(sum_out, "sum_out", index, shape, dt)
    pw = _tensor(weight, "weight", index, (width,), weight.dtype) if weight is not None else None
    a = NormArgs(_SIZE[NormArgs], _DT[dt], F32 if weight is None else _DT[weight.dtype], order, act, heads, width,
                 eps, scale, weight_offset, shape[0], px, pw, pg, pr, py, ps, sx, sg, sr, sy, ss)
    _run("gdn_rms_norm", a, index)
    return (y, sum_out) if sums else y


def rms_norm_backward(x, dy, weight=None, gate=None, d_sum=None, residual=False, order="pre", activation="silu",
                      scale=1.0, eps=1e-6, weight_offset=0.0, dx=None, dgate=None, workspace=None):
    """Gradients of rms_norm: returns (dx, dresidual, dweight, dgate).

    x is what was normed: the forward call's x, or the sum h that it returned
    (residual=True, or d_sum, the gradient that reaches h from its other uses,
    say so).  dx is the gradient of the forward call's x; dresidual that of
    the residual (None without one; in the post order it is dy itself and
    None here; with scale 1 it is the same tensor as dx).  dweight is fp32
    [D] (None without a weight), dgate like x (None without a gate)."""
    index, shape, heads, width = _norm_shape(x)
    order, act = _norm_how(weight, gate, order, activation)
    dt, dev = x.dtype, x.device
    residual = residual or d_sum is not None
    if residual and order == 1:
        raise GdnError("residual and d_sum belong to the pre order: in the post order the residual's gradient is dy")
    if order == 0 and not residual and scale != 1.0:
        raise GdnError("the pre order scales x only where it is added to a residual")
    dx = torch.empty_like(x) if dx is None else dx
    dres = None
    if residual:
        dres = dx if scale == 1.0 else torch.empty_like(x)
    if gate is not None and dgate is None:
        dgate = torch.empty_like(gate)
    px, sx = _rows(x, "x", index, shape, dt)
    pg, sg = _rows(gate, "gate", index, shape, dt)
    pd, sd = _rows(dy, "dy", index, shape, dt)
    pu, su = _rows(d_sum, "d_sum", index, shape, dt)
    po, so = _rows(dx, "dx", index, shape, dt)
    pr, sr = (None, 0) if dres is dx else _rows(dres, "dresidual", index, shape, dt)
    pz, sz = _rows(dgate, "dgate", index, shape, dt)
    dweight = pw = None
    if weight is not None:
        pw = _tensor(weight, "weight", index, (width,), weight.dtype)
        dweight = torch.empty(width, dtype=torch.float32, device=dev)
    a = NormBwdArgs(_SIZE[NormBwdArgs], _DT[dt], F32 if weight is None else _DT[weight.dtype], order, act, heads,
                    width, eps, scale, weight_offset, shape[0], px, pw, pg, pd, pu, po, pr, pz,
                    None if dweight is None else dweight.data_ptr(), sx, sg, sd, su, so, sr, sz)
    if dweight is not None:
        workspace = _workspace(workspace, _entry("gdn_rms_norm_backward_workspace_size")(a), index, dev)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _run("gdn_rms_norm_backward", a, index)
    return dx, dres, dweight, dgate


def _workspace(given, need, index, dev):
    """The caller's workspace where it is large enough, else a new one."""
    if given is not None:
        if not isinstance(given, torch.Tensor) or given.get_device() != index or given.dtype != torch.uint8:
            raise GdnError("workspace must be a torch.uint8 tensor on the call's GPU")
        if given.numel() >= need and given.is_contiguous():
            return given
    return torch.empty(need, dtype=torch.uint8, device=dev)


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


ROPE_LAYOUT = {"half": 0, "interleaved": 1}


def _heads(t, name, index, dtype):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise GdnError(f"{name} must be a [T, H, d] tensor")
    return _rows(t, name, index, t.shape, dtype)


def _rope(q, positions, inv_freq, k, layout, mscale, inverse, out, k_out):
    index = _gpu(q, "q")
    if q.dtype not in _DT:
        raise GdnError(f"q must be torch.bfloat16 or torch.float32, got {q.dtype}")
    if layout not in ROPE_LAYOUT:
        raise GdnError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    dt = q.dtype
    pq, sq = _heads(q, "q", index, dt)
    T, h_q, d = q.shape
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int64, torch.int32):
        raise GdnError("positions must be a torch.int32 or torch.int64 tensor")
    pp = _tensor(positions, "positions", index, (T,), positions.dtype)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise GdnError("inv_freq must be a [rot / 2] tensor")
    pf = _tensor(inv_freq, "inv_freq", index, inv_freq.shape, torch.float64)
    y = torch.empty_like(q) if out is None else out
    py, sy = _rows(y, "out", index, q.shape, dt)
    h_k, pk, sk, pz, sz, z = 0, None, 0, None, 0, None
    if k is not None:
        pk, sk = _heads(k, "k", index, dt)
        if k.shape[0] != T or k.shape[2] != d:
            raise GdnError(f"k must be [{T}, H, {d}], got {list(k.shape)}")
        h_k = k.shape[1]
        z = torch.empty_like(k) if k_out is None else k_out
        pz, sz = _rows(z, "k_out", index, k.shape, dt)
    elif k_out is not None:
        raise GdnError("k_out goes with k")
    a = RopeArgs(_SIZE[RopeArgs], _DT[dt], ROPE_LAYOUT[layout], inverse, 64 if positions.dtype == torch.int64 else 32,
                 h_q, h_k, d, 2 * inv_freq.shape[0], mscale, T, pq, pk, pp, pf, py, pz, sq, sk, sy, sz)
    _run("gdn_rope", a, index)
    return y if k is None else (y, z)


def rope(q, positions, inv_freq, k=None, layout="half", mscale=1.0, out=None, k_out=None):
    """Rotary positions on the heads of q [T, H, d], and of k [T, H_k, d] in the
    same launch (bf16 or fp32, token stride free): returns q' or (q', k').

    positions [T] (int32 or int64) are the tokens' positions, inv_freq
    [rot / 2] fp64 the radians a position of each pair (rope_frequencies);
    rot may be less than d: the rest of a head passes through.  layout "half"
    pairs elements i and i + rot / 2, "interleaved" 2 i and 2 i + 1.  out and
    k_out may be q and k themselves (in place)."""
    return _rope(q, positions, inv_freq, k, layout, mscale, 0, out, k_out)


def rope_backward(dq, positions, inv_freq, k=None, layout="half", mscale=1.0, out=None, k_out=None):
    """Gradients of rope's inputs given those of its outputs (dq, and k: that of
    k'): the rotation by the opposite angle.  Arguments as in rope."""
    return _rope(dq, positions, inv_freq, k, layout, mscale, 1, out, k_out)


FP8 = torch.float8_e4m3fn
KVCache = collections.namedtuple("KVCache", "k v k_scale v_scale")


def kv_cache(pages, h_kv, d, page_size=64, device="cuda"):
    """An empty pool of pages: e4m3 keys [pages, h_kv, page_size, d] and values
    [pages, h_kv, d, page_size], and their fp32 scales [pages, h_kv]."""
    def new(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)

    return KVCache(new(pages, h_kv, page_size, d, dtype=torch.uint8).view(FP8), new(pages, h_kv, d, page_size, dtype=torch.uint8).view(FP8),
                   new(pages, h_kv, dtype=torch.float32), new(pages, h_kv, dtype=torch.float32))


def _cache(cache, index, h_kv, d):
    if len(cache) != 4 or not isinstance(cache[0], torch.Tensor) or cache[0].dim() != 4:
        raise GdnError("cache must be (k [pages, h_kv, page_size, d], v, k_scale, v_scale)")
    k, v, ks, vs = cache
    pages, h, page = k.shape[:3]
    if h != h_kv or k.shape[3] != d:
        raise GdnError(f"the cache holds {h} heads of {k.shape[3]}, not {h_kv} of {d}")
    return (pages, page, _tensor(k, "cache.k", index, k.shape, FP8), _tensor(v, "cache.v", index, (pages, h, d, page), FP8),
            _tensor(ks, "cache.k_scale", index, (pages, h), torch.float32), _tensor(vs, "cache.v_scale", index, (pages, h), torch.float32))


def _sequences(page_table, lens, cu_seqlens, index, tokens):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise GdnError("page_table must be [n_seqs, max_pages]")
    n, width = page_table.shape
    pt = _tensor(page_table, "page_table", index, page_table.shape, torch.int32)
    pl = _tensor(lens, "lens", index, (n,), torch.int32)
    if pl is None:
        raise GdnError("lens is required")
    pc = _tensor(cu_seqlens, "cu_seqlens", index, (n + 1,), torch.int32)
    if pc is None and n and tokens % n:
        raise GdnError(f"without cu_seqlens every sequence has the same number of new tokens: {tokens} over {n} sequences")
    return n, width, pt, pl, pc


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
    index = _gpu(k, "k")
    if k.dtype not in _DT:
        raise GdnError(f"k must be torch.bfloat16 or torch.float32, got {k.dtype}")
    pk, sk = _heads(k, "k", index, k.dtype)
    T, h, d = k.shape
    pv, sv = _rows(v, "v", index, k.shape, k.dtype)
    pages, page, pkc, pvc, pks, pvs = _cache(cache, index, h, d)
    n, width, pt, pl, pc = _sequences(page_table, lens, cu_seqlens, index, T)
    a = CacheStoreArgs(_SIZE[CacheStoreArgs], _DT[k.dtype], n, h, d, page, pages, width, T, pk, pv, sk, sv, pkc, pvc, pks, pvs,
                       pt, pl, pc)
    _run("gdn_cache_store", a, index)


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
    index = _gpu(q, "q")
    if q.dtype not in _DT:
        raise GdnError(f"q must be torch.bfloat16 or torch.float32, got {q.dtype}")
    dt = q.dtype
    pq, sq = _heads(q, "q", index, dt)
    T, h_q, d = q.shape
    if not isinstance(cache[0], torch.Tensor) or cache[0].dim() != 4:
        raise GdnError("cache must be (k [pages, h_kv, page_size, d], v, k_scale, v_scale)")
    h = cache[0].shape[1]
    pages, page, pkc, pvc, pks, pvs = _cache(cache, index, h, d)
    n, width, pt, pl, pc = _sequences(page_table, lens, cu_seqlens, index, T)
    pg, sg = _rows(gate, "gate", index, q.shape, dt)
    o = torch.empty_like(q) if out is None else out
    po, so = _rows(o, "out", index, q.shape, dt)
    lse = torch.empty((T, h_q), dtype=torch.float32, device=q.device) if return_lse else None
    a = CacheAttentionArgs(_SIZE[CacheAttentionArgs], _DT[dt], n, h_q, h, d, page, pages, width, 1 if causal else 0, window,
                           d ** -0.5 if scale is None else scale, T, pq, pg, po, sq, sg, so, None if lse is None else lse.data_ptr(), pkc,
                           pvc, pks, pvs, pt, pl, pc)
    need = _entry("gdn_cache_attention_workspace_size")(a)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, index, q.device)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _run("gdn_cache_attention", a, index)
    return (o, lse) if return_lse else o


def cache_attention_workspace_size(tokens, n_seqs, max_pages, h_q, h_kv, d, page_size=64, ragged=False, dtype=torch.bfloat16):
    """Bytes of workspace that cache_attention needs (0: none) for a caller that keeps one."""
    a = CacheAttentionArgs(struct_size=ctypes.sizeof(CacheAttentionArgs), io_dtype=_DT[dtype], n_seqs=n_seqs, h_q=h_q, h_kv=h_kv, d=d, page_size=page_size,
                           max_pages=max_pages, tokens=tokens, cu_seqlens=1 if ragged else None)
    return lib().gdn_cache_attention_workspace_size(a)
