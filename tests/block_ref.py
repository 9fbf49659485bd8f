"""Plain 64-bit forms of the operators around the mixer, for the parity tests,
and the error bound that the tests share.

Bound: an output element may be off by half a step of its type (finfo.eps / 2
relative to its value) plus the error of the fp32 arithmetic behind it, which
is counted as `terms` roundings (2^-24 each) of the sum of the absolute values
of the terms that the element is made of (`size`).
"""
import math

import torch


def close(got, ref, size, terms=64, what=""):
    """got (bf16 or fp32) against ref (fp64); size: magnitude of its terms, or a number."""
    got64 = got.detach().double().cpu()
    ref = ref.detach().double().cpu()
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    size = torch.as_tensor(size, dtype=torch.float64).cpu()
    bound = torch.finfo(got.dtype).eps / 2 * ref.abs() + terms * 2.0 ** -24 * torch.maximum(size, ref.abs())
    off = (got64 - ref).abs() - bound
    assert torch.isfinite(got64).all(), f"{what}: not finite"
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} over the bound at {divmod(int(off.argmax()), max(1, got.shape[-1]))}"


def act(name, z):
    s = torch.sigmoid(z)
    return z * s if name == "silu" else s


def slope(name, z):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s)) if name == "silu" else s * (1 - s)


def d64(t):
    return None if t is None else t.detach().double().cpu()


def rms_norm(x, weight, gate, residual, order, activation, scale, eps, offset):
    """y and the sum, in 64 bits."""
    x, w, z, res = d64(x), d64(weight), d64(gate), d64(residual)
    h = x
    if order == "pre" and res is not None:
        h = res + scale * x
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * (w + offset)
    if z is not None:
        y = y * act(activation, z)
    if order == "post":
        y = scale * y + (0 if res is None else res)
    return y, h


def rms_norm_backward(x, dy, weight, gate, d_sum, order, activation, scale, eps, offset):
    """Gradient of what was normed, of the weight and of the gate, with the magnitudes of their terms."""
    h, g, w, z, du = d64(x), d64(dy), d64(weight), d64(gate), d64(d_sum)
    g = g * scale if order == "post" else g
    w = torch.ones(h.shape[-1], dtype=torch.float64) if w is None else w + offset
    a = 1.0 if z is None else act(activation, z)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n, u = h * r, g * w * a
    dh = r * (u - n * (u * n).mean(-1, keepdim=True))
    dh_size = r * (u.abs() + n.abs() * (u * n).abs().mean(-1, keepdim=True))
    if du is not None:
        dh, dh_size = dh + du, dh_size + du.abs()
    dims = tuple(range(h.dim() - 1))
    dw, dw_size = (g * n * a).sum(dims), (g * n * a).abs().sum(dims)
    # the SiLU's slope is a difference that crosses zero: its error is relative to the factors beside it
    dz = None if z is None else (g * n * w * slope(activation, z), (g * n * w).abs())
    return dh, dh_size, dw, dw_size, dz


def rope(x, positions, inv_freq, layout, mscale, inverse):
    """Rotated heads in 64 bits, and the magnitude of their terms."""
    x = d64(x)
    angle = positions.cpu().double()[:, None] * inv_freq.cpu() * (-1 if inverse else 1)
    c, s = mscale * angle.cos()[:, None], mscale * angle.sin()[:, None]
    rot = 2 * angle.shape[1]
    even = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    odd = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    y, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., even], x[..., odd]
    y[..., even], y[..., odd] = a * c - b * s, b * c + a * s
    size[..., even] = size[..., odd] = abs(mscale) * (a.abs() + b.abs())
    return y, size


FP8 = torch.float8_e4m3fn


def decode(codes):
    """e4m3 codes' values, fp64 on the CPU."""
    return codes.cpu().view(FP8).float().double()


def lengths_of(cu, tokens, n):
    if cu is None:
        return [tokens // n] * n, [i * (tokens // n) for i in range(n)]
    cu = cu.tolist()
    return [b - a for a, b in zip(cu, cu[1:])], cu[:-1]


def _pow2(most):
    """The least power of two s >= 2^-126 with most <= 448 s."""
    s = 2.0 ** -126
    while most > 448 * s:
        s *= 2
    return s


def cache_store(k, v, cache, table, lens, cu):
    """The cache after the call, codes as bytes (CPU tensors), page by page and head by head."""
    kc, vc, ks, vs = (t.cpu().clone() for t in cache)
    kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    pages, heads, page, d = kc.shape
    new, begin = lengths_of(cu, k.shape[0], table.shape[0])
    table, lens = table.cpu(), lens.tolist()
    for n in range(len(new)):
        for first in range(lens[n] // page * page, lens[n] + new[n], page):
            if not new[n] or first // page >= table.shape[1]:
                continue
            p = int(table[n, first // page])
            if not 0 <= p < pages:
                continue
            a, b = max(lens[n] - first, 0), min(lens[n] + new[n] - first, page)
            row = begin[n] + first + a - lens[n]
            for x, codes, scales in ((k, kc, ks), (v, vc.transpose(2, 3), vs)):
                x = x[row:row + b - a].float().cpu()
                for h in range(heads):
                    f = x[:, h]
                    fine = f.abs()[f.isfinite()]
                    scale = _pow2(fine.max().item() if fine.numel() else 0.0)
                    was = scales[p, h].item()
                    if a and was > scale:
                        scale = was
                    if a and was != scale:
                        old = codes[p, h, :a].contiguous().view(FP8).float()
                        codes[p, h, :a] = (old * (was / scale)).to(FP8).view(torch.uint8)
                    y = (f.double() / scale).clamp(-448, 448)  # clamp keeps NaN
                    codes[p, h, a:b] = y.float().to(FP8).view(torch.uint8)
                    scales[p, h] = scale
    return kc, vc, ks, vs


def cache_attention(q, cache, table, lens, cu=None, scale=None, causal=True, window=0, gate=None):
    """Output and logarithm of the sum in 64 bits; the magnitude of the output's terms, an absolute error of its
    16-bit weights and the largest |score| of each row, for bounds.  Rows of no sequence stay NaN."""
    kc, vc, ks, vs = cache
    kc, vc, ks, vs = decode(kc), decode(vc), ks.cpu().double(), vs.cpu().double()
    pages, heads, page, d = kc.shape
    T, hq = q.shape[:2]
    group = hq // heads
    scale = d ** -0.5 if scale is None else scale
    q64, z = d64(q), d64(gate)
    table, lens = table.cpu(), lens.tolist()
    new, begin = lengths_of(cu, T, table.shape[0])
    o = torch.full((T, hq, d), math.nan, dtype=torch.float64)
    size, low = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((T, hq), math.nan, dtype=torch.float64)
    far = torch.zeros((T, hq), dtype=torch.float64)
    for n in range(len(new)):
        ctx = min(lens[n], table.shape[1] * page)
        at = torch.arange(max(ctx, 0))
        pid = table[n, at // page].long()
        there = (pid >= 0) & (pid < pages)
        pid = pid.clamp(0, pages - 1)
        for i in range(new[n]):
            pos = ctx - new[n] + i
            sees = there & ((at <= pos) if causal else (at >= 0))
            if window:
                sees = sees & (at > pos - window)
            t = begin[n] + i
            if not sees.any():
                o[t], lse[t] = 0.0, -math.inf
                continue
            a, p = at[sees] % page, pid[sees]
            for h in range(hq):
                kv = h // group
                key = kc[p, kv, a] * ks[p, kv, None]
                code, unit = vc[p, kv, :, a], vs[p, kv, None]
                score = scale * (key @ q64[t, h])
                far[t, h] = scale * (key.abs() @ q64[t, h].abs()).max()
                lse[t, h] = torch.logsumexp(score, 0)
                w = torch.exp(score - lse[t, h])[:, None]
                o[t, h] = (w * unit * code).sum(0)
                size[t, h] = (w * unit * code).abs().sum(0)
                low[t, h] = code.abs().sum(0) * (w * unit).max()
    if z is not None:
        s = torch.sigmoid(z)
        o, size, low = o * s, size * s, low * s
    return o, lse, size, low, far


def close_attention(got, ref, what=""):
    """o (and lse) within: half a step of the type; the weights' rounding (fp16, 2^-11 relative and 2^-25 of the
    largest, for bf16 outputs; 24 bits for fp32); the scores' error, an fp32 dot product of d terms and one
    exponential (d + 16 roundings of the largest sum of |q k|), which scales a weight by as much."""
    o, lse = got if isinstance(got, tuple) else (got, None)
    ro, rl, size, low, far = ref
    rows = ~torch.isnan(rl)
    d = o.shape[-1]
    step = 2.0 ** -24
    terms = ((d + 16) * far + 64)[..., None]
    extra = terms * step * 2 * size
    if o.dtype == torch.bfloat16:
        extra = extra + 2.0 ** -11 * size + 2.0 ** -25 * low
    else:
        extra = extra + 2.0 ** -24 * 4 * size
    ok = rows.any(-1)
    close(o.cpu()[ok], ro[ok], (extra / (64 * step))[ok], 64, what + " o")
    if lse is not None:
        l, r = lse.double().cpu()[ok], rl[ok]
        assert torch.equal(torch.isinf(l), torch.isinf(r)), what
        fine = torch.isfinite(r)
        bound = step * (terms[..., 0][ok] + 8 * r.abs())
        assert ((l - r).abs()[fine] <= bound[fine]).all(), f"{what} lse {(l - r).abs()[fine].max()}"
