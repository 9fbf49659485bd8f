"""rope and rope_backward against their 64-bit form: layouts, parts of a head,
types, odd sizes and strides, far positions, in place."""
import pytest
import torch

import block_ref as ref
import linear_attention_token_conv1d_amd as gdn

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# the angle's rounding to fp32 turns is 2^-25 of a turn (1.9e-7 rad, 3.2 roundings), sine and cosine add two, the
# products and the sum three; the hardware's sine and cosine (bf16) are off by up to 2^-20, 16 roundings, each
TERMS = {BF16: 48, F32: 16}


def _heads(gen, T, H, d, dtype, pad):
    return torch.randn((T, H * d + pad), generator=gen).to(dtype).cuda()[:, :H * d].unflatten(1, (H, d))


CASES = [
    # T, h_q, h_k, d, rot, pad, far
    (1, 24, 4, 256, 64, 0, 262144), (256, 24, 4, 256, 64, 8, 1 << 20), (37, 3, 1, 128, 128, 0, 4096), (5, 2, 2, 64, 32, 3, 100),
    (9, 1, 0, 64, 64, 0, 1 << 31), (4, 5, 2, 70, 34, 0, 9999), (3, 2, 1, 6, 2, 0, 50), (2, 1, 1, 2, 2, 1, 50), (3, 4, 4, 96, 48, 0, 1000),
    (2000, 6, 2, 64, 16, 16, 8000), (7, 2, 1, 33, 32, 0, 70000), (3, 7, 3, 512, 320, 0, 5000),
]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,h_q,h_k,d,rot,pad,far", CASES)
def test_rotation(T, h_q, h_k, d, rot, pad, far, dtype, layout):
    gen = torch.Generator().manual_seed(T + d + rot)
    q = _heads(gen, T, h_q, d, dtype, pad)
    k = _heads(gen, T, h_k, d, dtype, pad) if h_k else None
    inv, _ = gdn.rope_frequencies(rot, 1e4, device="cuda")
    pos = torch.randint(-far if far <= 100 else 0, far, (T,), generator=gen).cuda()
    pos[0] = far - 1
    if far < 1 << 31 and T % 2:
        pos = pos.to(torch.int32)
    for f, inverse in ((gdn.rope, False), (gdn.rope_backward, True)):
        got = f(q, pos, inv, k=k, layout=layout, mscale=1.25)
        got = got if k is not None else (got,)
        for y, x in zip(got, (q, k)):
            want, size = ref.rope(x, pos, inv, layout, 1.25, inverse)
            ref.close(y, want, size, TERMS[dtype], f"{layout} {inverse}")
            assert torch.equal(y[..., rot:], x[..., rot:])
    # in place
    q2, k2 = q.clone(), None if k is None else k.clone()
    got = gdn.rope(q2, pos, inv, k=k2, layout=layout, out=q2, k_out=k2)
    for y, x, z in zip(got if k is not None else (got,), (q, k), (q2, k2)):
        assert y is z
        want, size = ref.rope(x, pos, inv, layout, 1.0, False)
        ref.close(y, want, size, TERMS[dtype], f"{layout} in place")
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_gradient_is_the_transpose():
    """sum(dy * rope(x)) has the gradient rope_backward(dy): checked by the inner products of random vectors."""
    gen = torch.Generator().manual_seed(3)
    x, dy = (_heads(gen, 50, 2, 64, F32, 0) for _ in range(2))
    inv, m = gdn.rope_frequencies(48, 1e4, "by_parts", 8.0, original=512, device="cuda")
    pos = torch.arange(50, device="cuda")
    for layout in ("half", "interleaved"):
        y = gdn.rope(x, pos, inv, layout=layout, mscale=m)
        dx = gdn.rope_backward(dy, pos, inv, layout=layout, mscale=m)
        a, b = (dy.double() * y.double()).sum().item(), (dx.double() * x.double()).sum().item()
        # 6400 products of size ~1, each off by at most 16 roundings of terms of about 3
        assert abs(a - b) < 6400 * 16 * 3 * 2.0 ** -24


def test_no_tokens_graph_and_stream():
    inv, _ = gdn.rope_frequencies(64, device="cuda")
    q = torch.zeros((0, 4, 64), dtype=BF16, device="cuda")
    assert gdn.rope(q, torch.zeros(0, dtype=torch.int64, device="cuda"), inv).shape == (0, 4, 64)
    gen = torch.Generator().manual_seed(8)
    q, k = _heads(gen, 33, 4, 128, BF16, 0), _heads(gen, 33, 2, 128, BF16, 0)
    pos = torch.arange(33, device="cuda", dtype=torch.int32)
    want = gdn.rope(q, pos, inv, k=k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = gdn.rope(q, pos, inv, k=k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn.rope(q, pos, inv, k=k)
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, again):
            assert torch.equal(a, b) and torch.equal(a, c)
        gdn.rope(k, pos, inv, k=q)


def test_refusals():
    inv, _ = gdn.rope_frequencies(64, device="cuda")
    q, k = torch.zeros((4, 2, 128), dtype=BF16, device="cuda"), torch.zeros((4, 1, 128), dtype=BF16, device="cuda")
    pos = torch.arange(4, device="cuda")
    for args, kw in [((q, pos[:3], inv), {}), ((q, pos.float(), inv), {}), ((q, pos, inv.float()), {}), ((q, pos, inv), dict(k=k[:3])),
                     ((q, pos, inv), dict(k=k[..., :64])), ((q, pos, inv), dict(layout="other")), ((q.half(), pos, inv), {}),
                     ((q[..., :32], pos, inv), {}), ((q, pos.cpu(), inv), {}), ((q, pos, inv), dict(k=k.float())),
                     ((q, pos, inv), dict(k_out=k)), ((q, pos, inv), dict(k=q[:, :1], k_out=q[:, 1:])), ((q, pos, inv[:0]), {}),
                     ((q, pos, inv), dict(mscale=float("inf"))), ((q[:, 0], pos, inv), {})]:
        with pytest.raises(gdn.GdnError):
            gdn.rope(*args, **kw)


def test_offsets_beyond_32_bits():
    """Tokens behind the first 2^31 elements, and more threads than 32 bits count where pairs are single."""
    T, H, d = 2100000, 8, 130
    q = torch.empty((T, H, d), dtype=BF16, device="cuda")
    tail = torch.randn((7, H, d), generator=torch.Generator().manual_seed(9)).to(BF16).cuda()
    q[-7:] = tail
    inv, _ = gdn.rope_frequencies(64, device="cuda")
    pos = torch.arange(T, device="cuda")
    gdn.rope(q, pos, inv, out=q)
    assert torch.equal(q[-7:], gdn.rope(tail, pos[-7:], inv))
