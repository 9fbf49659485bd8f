"""rms_norm and rms_norm_backward against their 64-bit forms: types, layouts,
both orders, gates, odd widths and strides, in-place use, graphs, streams."""
import pytest
import torch

import block_ref as ref
import linear_attention_token_conv1d_amd as gdn

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _rand(gen, shape, dtype, pad=0, scale=1.0):
    """[T, H, d] as a column slice of a buffer `pad` elements wider."""
    T, cols = shape[0], shape[1] * shape[2]
    x = (scale * torch.randn((T, cols + pad), generator=gen)).to(dtype).cuda()
    return x[:, :cols].unflatten(1, shape[1:])


SHAPES = [
    # tokens, heads, width, pad
    (1, 1, 1, 0), (3, 1, 7, 0), (1, 1, 5120, 0), (5, 48, 128, 2048), (7, 3, 64, 8), (2, 1, 1000, 0), (4, 2, 129, 3),
    (3, 5, 33, 0), (9, 1, 2049, 1), (2, 1, 16384, 0), (2, 1, 16383, 0), (300, 2, 256, 0), (2, 1, 6000, 4), (1000, 1, 8, 0),
    (3, 1, 4096, 0), (2, 1, 8192, 8), (33, 1, 1024, 0), (17, 1, 136, 0), (2, 1, 12288, 0), (3, 1, 520, 0),
    (3, 1, 4095, 0), (2, 1, 4097, 0), (70, 1, 2500, 1), (2, 4, 136, 3),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,D,pad", SHAPES)
def test_forward(T, H, D, pad, dtype):
    gen = torch.Generator().manual_seed(T * 7 + D)
    x, z, res = (_rand(gen, (T, H, D), dtype, p) for p in (pad, pad, 0))
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    for i, (order, act, weight, gate, residual, scale, offset) in enumerate([
            ("pre", "silu", w.to(dtype), z, None, 1.0, 0.0), ("pre", "sigmoid", w, None, res, 0.37, 1.0),
            ("pre", "sigmoid", w, z, res, 1.0, 0.0), ("post", "silu", w.to(dtype), None, res, 0.5, 0.0),
            ("post", "sigmoid", None, z, None, 2.0, 0.0), ("pre", "silu", None, None, None, 1.0, 0.0)]):
        got = gdn.rms_norm(x, weight, gate, residual, order, act, scale, 1e-5, offset)
        y, h = ref.rms_norm(x, weight, gate, residual, order, act, scale, 1e-5, offset)
        size = y.abs() if order == "pre" else y.abs() + (0 if residual is None else 2 * ref.d64(residual).abs())
        if residual is not None and order == "pre":
            # the sum may cancel, to zero too: its error (scale rounded to fp32, one rounding of the sum) is at most
            # 2^-24 of each of its terms, and reaches y by the factor y / h, which is that of a row of ones
            terms = ref.d64(residual).abs() + scale * ref.d64(x).abs()
            ref.close(got[1], h, terms, 2, f"sum {i}")
            r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5)
            size = size + terms * r * (ref.d64(weight) + offset).abs() * (1.0 if gate is None else ref.act(act, ref.d64(gate)).abs())
            got = got[0]
        ref.close(got, y, size, 64, f"y {i}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,D,pad", SHAPES)
def test_backward(T, H, D, pad, dtype):
    gen = torch.Generator().manual_seed(T * 11 + D)
    x, z, dy, ds = (_rand(gen, (T, H, D), dtype, p) for p in (pad, pad, 0, pad))
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    for i, (order, act, weight, gate, d_sum, residual, scale, offset) in enumerate([
            ("pre", "silu", w.to(dtype), z, None, False, 1.0, 0.0), ("pre", "sigmoid", w, None, ds, True, 0.37, 1.0),
            ("pre", "sigmoid", None, z, ds, True, 1.0, 0.0), ("post", "silu", w, z, None, False, 0.5, 0.0),
            ("pre", "silu", w, None, None, True, 2.0, 0.0), ("post", "silu", None, None, None, False, 1.0, 0.0)]):
        dx, dres, dw, dz = gdn.rms_norm_backward(x, dy, weight, gate, d_sum, residual, order, act, scale, 1e-5, offset)
        rh, sh, rw, sw, rz = ref.rms_norm_backward(x, dy, weight, gate, d_sum, order, act, scale, 1e-5, offset)
        f = scale if order == "pre" and residual else 1.0
        ref.close(dx, f * rh, f * sh, 64, f"dx {i}")
        assert (dres is None) == (not residual)
        if residual:
            ref.close(dres, rh, sh, 64, f"dresidual {i}")
        if weight is not None:
            # at most T*H/groups + log terms are added one after another
            ref.close(dw, rw, sw, 64 + T * H / 16, f"dweight {i}")
        else:
            assert dw is None
        if gate is not None:
            ref.close(dz, rz[0], rz[1], 64, f"dgate {i}")
        else:
            assert dz is None


def test_backward_against_differences():
    """The gradients are those of the loss sum(dy * y) + sum(d_sum * h): central differences of the 64-bit form."""
    gen = torch.Generator().manual_seed(2)
    T, H, D = 3, 2, 24
    x, z, dy, ds = (_rand(gen, (T, H, D), F32) for _ in range(4))
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    dx, dres, dw, dz = gdn.rms_norm_backward(x, dy, w, z, ds, True, "pre", "silu", 0.7, 1e-5, 0.25)

    def loss(h, wt, zt):
        y, _ = ref.rms_norm(h, wt, zt, None, "pre", "silu", 1.0, 1e-5, 0.25)
        return (ref.d64(dy) * y).sum() + (ref.d64(ds) * ref.d64(h)).sum()

    eps = 1e-5
    args = [ref.d64(x), ref.d64(w), ref.d64(z)]
    for k, grad in enumerate((dres, dw, dz)):
        flat = args[k].reshape(-1)
        for i in range(0, flat.numel(), 5):
            keep = flat[i].item()
            flat[i] = keep + eps
            up = loss(*args)
            flat[i] = keep - eps
            down = loss(*args)
            flat[i] = keep
            diff = ((up - down) / (2 * eps)).item()
            # differences: eps^2 of the third derivative and 2^-52 of the loss over eps, both under 1e-7 here
            assert abs(grad.reshape(-1)[i].item() - diff) < 2e-5, (k, i)
    assert torch.allclose(dx, 0.7 * dres, rtol=2.0 ** -23, atol=0)


def test_no_rows():
    x = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    assert gdn.rms_norm(x, w).shape == (0, 4, 64)
    _, _, dw, _ = gdn.rms_norm_backward(x, x, w)
    assert torch.equal(dw, torch.zeros(64, device="cuda"))


def test_zero_rows_and_extremes():
    """A row of zeros stays zero (eps keeps it finite); large rows do not overflow in fp32 sums of bf16 inputs."""
    x = torch.zeros((3, 1, 256), dtype=BF16, device="cuda")
    x[1] = 1e15
    x[2] = 1e-15
    y = gdn.rms_norm(x, eps=1e-6)
    assert torch.equal(y[0], torch.zeros_like(y[0]))
    assert torch.equal(y[1], torch.ones_like(y[1]))
    ref.close(y[2], ref.rms_norm(x, None, None, None, "pre", "silu", 1.0, 1e-6, 0.0)[0][2], 0.0, 64)
    z = torch.full((3, 1, 256), -200.0, dtype=BF16, device="cuda")
    z[1], z[2] = 200.0, -torch.inf
    for act, want in (("silu", [0.0, 200.0]), ("sigmoid", [0.0, 1.0])):
        y = gdn.rms_norm(torch.ones_like(x), gate=z, activation=act, eps=0.0)
        assert y[0].abs().max().item() <= 1e-30 and torch.all(y[1] == want[1])
        if act == "sigmoid":
            assert torch.all(y[2] == 0)


def test_in_place_and_slices():
    """Outputs over their inputs, and gradients as column slices of one buffer."""
    gen = torch.Generator().manual_seed(4)
    T, H, D = 37, 3, 128
    x, res, z = (_rand(gen, (T, H, D), BF16) for _ in range(3))
    w = torch.ones(D, dtype=BF16, device="cuda")
    y, h = gdn.rms_norm(x, w, z, res)
    x2, res2 = x.clone(), res.clone()
    y2, h2 = gdn.rms_norm(x2, w, z, res2, out=x2, sum_out=res2)
    assert y2 is x2 and h2 is res2 and torch.equal(y, y2) and torch.equal(h, h2)
    buf = torch.full((T, 2 * H * D + 5), 7.0, dtype=BF16, device="cuda")
    dx, dz = (buf[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (0, 1))
    # the slices' odd token stride rules wide loads out, so sums are taken in another order than for whole tensors
    got = gdn.rms_norm_backward(h, x, w, z, dx=dx, dgate=dz)
    assert got[0] is dx and got[3] is dz
    rh, sh, rw, sw, rz = ref.rms_norm_backward(h, x, w, z, None, "pre", "silu", 1.0, 1e-6, 0.0)
    ref.close(dx, rh, sh, 64, "dx")
    ref.close(got[2], rw, sw, 64 + T * H / 16, "dweight")
    ref.close(dz, rz[0], rz[1], 64, "dgate")
    assert torch.all(buf[:, 2 * H * D:] == 7.0)


def test_deterministic_graph_and_stream():
    gen = torch.Generator().manual_seed(5)
    T, H, D = 3000, 4, 128
    x, z, dy = (_rand(gen, (T, H, D), BF16) for _ in range(3))
    w = torch.ones(D, device="cuda")
    first = gdn.rms_norm_backward(x, dy, w, z)
    fy = gdn.rms_norm(x, w, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = gdn.rms_norm_backward(x, dy, w, z)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, again):
        assert a is None or torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gdn.rms_norm(x, w, z)
        got = gdn.rms_norm_backward(x, dy, w, z)
    for _ in range(3):
        for t in (y, *got):
            if t is not None:
                t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, fy)
        for a, b in zip(first, got):
            assert a is None or torch.equal(a, b)
        gdn.rms_norm_backward(z, x, w, dy)  # eager work between the replays


def test_refusals():
    x = torch.zeros((4, 2, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    bad = [dict(weight=w[:63]), dict(gate=x.float()), dict(residual=x[:3]), dict(order="mid"), dict(gate=x, activation="tanh"),
           dict(gate=x.transpose(0, 1)), dict(scale=2.0), dict(weight=w.half()), dict(weight=w.cpu()), dict(sum_out=x),
           dict(out=x.flatten()[64:].unfold(0, 64, 64)[:4]), dict(out=x[..., ::2]), dict(eps=-1.0)]
    for kw in bad:
        with pytest.raises(gdn.GdnError):
            gdn.rms_norm(x, **kw)
    shifted = torch.zeros(4 * 128 + 64, dtype=BF16, device="cuda")
    with pytest.raises(gdn.GdnError, match="overlap"):
        gdn.rms_norm(shifted[:512].view(4, 2, 64), out=shifted[64:].view(4, 2, 64))
    with pytest.raises(gdn.GdnError):
        gdn.rms_norm(torch.zeros((2, 16385), device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.rms_norm(x.half())
    with pytest.raises(gdn.GdnError):
        gdn.rms_norm_backward(x, x, order="post", residual=True)
    with pytest.raises(gdn.GdnError):
        gdn.rms_norm_backward(x, x, scale=0.5)


def test_offsets_beyond_32_bits():
    """Rows behind the first 2^31 elements."""
    T, D = 270000, 8192
    x = torch.empty((T, D), dtype=BF16, device="cuda")
    tail = torch.randn((5, D), generator=torch.Generator().manual_seed(9)).to(BF16).cuda()
    x[-5:] = tail
    w = torch.ones(D, dtype=BF16, device="cuda")
    y = gdn.rms_norm(x, w)
    assert torch.equal(y[-5:], gdn.rms_norm(tail, w))
    dx = gdn.rms_norm_backward(x, x, w, dx=y)[0]
    assert torch.equal(dx[-5:], gdn.rms_norm_backward(tail, tail, w)[0])


def test_small_rows_without_eps():
    """The gradient of rows so small that the third power of 1 / rms is beyond fp32."""
    gen = torch.Generator().manual_seed(10)
    x = 1e-14 * torch.randn((4, 1, 256), generator=gen).cuda()
    dy = torch.randn((4, 1, 256), generator=gen).cuda()
    dx = gdn.rms_norm_backward(x, dy, eps=0.0)[0]
    rh, sh, *_ = ref.rms_norm_backward(x, dy, None, None, None, "pre", "silu", 1.0, 0.0, 0.0)
    ref.close(dx, rh, sh, 64, "dx")


def test_more_rows_than_one_side_of_a_grid():
    """Rows of a workgroup each whose threads pass 32 bits."""
    T, D = (1 << 24) + 77, 1032
    x = torch.empty((T, D), dtype=BF16, device="cuda")
    tail = torch.randn((100, D), generator=torch.Generator().manual_seed(11)).to(BF16).cuda()
    x[-100:] = tail
    gdn.rms_norm(x, out=x)
    assert torch.equal(x[-100:], gdn.rms_norm(tail))
