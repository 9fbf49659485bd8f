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
