"""cache_store and cache_attention: an e4m3 paged cache, written and read.
Codes and scales are compared bit for bit, outputs against a 64-bit form.
Every slot that holds no token, and every page that no sequence owns, is
filled with NaN codes and scales, so anything read there shows."""
import pytest
import torch

import block_ref as ref
import linear_attention_token_conv1d_amd as gdn

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = 0x7F


def pool(pages, heads, d, page):
    c = gdn.kv_cache(pages, heads, d, page)
    for t in c[:2]:
        t.view(torch.uint8).fill_(NAN)
    for t in c[2:]:
        t.fill_(float("nan"))
    return c


def tables(gen, totals, page, extra=3, width=None):
    """A random page table for sequences of these lengths: [N, M] with -1 behind their pages, pages in the pool."""
    per = [-(-t // page) for t in totals]
    pages = sum(per) + extra
    order = torch.randperm(pages, generator=gen).tolist()
    width = width or max(1, max(per))
    rows = []
    for n in per:
        rows.append([order.pop() for _ in range(n)] + [-1] * (width - n))
    return torch.tensor(rows, dtype=torch.int32).cuda(), pages


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def cu_of(new):
    return ints([sum(new[:i]) for i in range(len(new) + 1)])


def check_store(k, v, cache, table, lens, cu, what=""):
    want = ref.cache_store(k, v, cache, table, lens, cu)
    gdn.cache_store(k, v, cache, table, lens, cu)
    for name, got, exp in zip(("k", "v", "k_scale", "v_scale"), cache, want):
        got = got.cpu()
        if got.dtype == torch.float32:
            assert torch.equal(got.view(torch.int32)[~torch.isnan(exp)], exp.view(torch.int32)[~torch.isnan(exp)]), (what, name)
            assert torch.equal(torch.isnan(got), torch.isnan(exp)), (what, name)
        else:
            got = got.view(torch.uint8)
            bad = (got != exp) & ~((got & 0x7F == NAN) & (exp & 0x7F == NAN))
            assert not bad.any(), f"{what} {name}: {int(bad.sum())} codes differ, first at {bad.nonzero()[0].tolist()}"


def rand(gen, T, heads, d, dtype, pad=0, scale=1.0):
    x = scale * torch.randn((T, heads * d + pad), generator=gen) * torch.exp(0.5 * torch.randn(heads * d + pad, generator=gen))
    return x.to(dtype).cuda()[:, :heads * d].unflatten(1, (heads, d))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page,d,heads", [(16, 64, 1), (32, 128, 2), (64, 256, 4), (128, 128, 3), (256, 256, 1), (64, 64, 8)])
def test_store_in_steps(page, d, heads, dtype):
    """Packs of unequal lengths, single tokens and uniform chunks, one after another into the same pages."""
    gen = torch.Generator().manual_seed(page + d)
    steps = [[0, 70, 1, 15, 33], [1] * 5, [3] * 5, [129, 0, 2, 64, 1], [1] * 5, [0, 0, 5, 0, 0]]
    totals = [sum(s[n] for s in steps) for n in range(5)]
    table, pages = tables(gen, totals, page)
    cache, lens = pool(pages, heads, d, page), [0] * 5
    for i, new in enumerate(steps):
        T = sum(new)
        size = 1.0 if i != 4 else 300.0  # a step whose values make the scales grow
        k, v = rand(gen, T, heads, d, dtype, 8, size), rand(gen, T, heads, d, dtype, 0, 1 / size)
        cu = None if len(set(new)) == 1 else cu_of(new)
        check_store(k, v, cache, table, ints(lens), cu, f"step {i}")
        lens = [a + b for a, b in zip(lens, new)]


def test_store_values():
    """Every bf16 magnitude class, subnormal codes, ties, infinities, NaN, zeros; a scale set by others."""
    page, d = 16, 64
    table = ints([[0], [1], [2], [3], [4]])
    cache = pool(5, 1, d, page)
    x = torch.zeros((5, 16, 1, d))
    x[0, :, 0] = torch.arange(16 * d).reshape(16, d) / 16.0  # to 63.9: ties among the codes
    x[1, :, 0] = torch.randn((16, d), generator=torch.Generator().manual_seed(1)) * torch.logspace(-38, 38, d)
    x[2, 3, 0, 5], x[2, 4, 0, 6], x[2, 5, 0, 7], x[2, 6, 0, :] = float("inf"), -float("inf"), float("nan"), 3.0
    x[4, :, 0] = 1e-30 * torch.arange(d)
    for dtype in (F32, BF16):
        k = x.reshape(80, 1, d).to(dtype).cuda()
        check_store(k, -k, cache, table, ints([0] * 5), None, str(dtype))
    # older tokens keep the page's scale where it is larger, whatever it is
    cache.k_scale.fill_(0.3), cache.v_scale.fill_(1e-3)
    k = torch.ones((5, 1, d), device="cuda")
    check_store(k, 50 * k, cache, table, ints([7] * 5), None, "others' scale")


def test_store_refuses_nothing_it_cannot_place():
    """Pages outside the pool, a table that ends, lengths below zero, rows of no sequence: not stored, nothing else touched."""
    page, d = 16, 64
    gen = torch.Generator().manual_seed(5)
    cache = pool(6, 2, d, page)
    table = ints([[-1, 2], [6, 0], [4, 1]])
    k, v = rand(gen, 70, 2, d, BF16), rand(gen, 70, 2, d, BF16)
    new = [20, 20, 20]
    check_store(k, v, cache, table, ints([0, 5, 20]), cu_of(new), "outside")  # the third sequence passes the table's end
    before = [t.clone() for t in cache]
    gdn.cache_store(k, v, cache, table, ints([-3, 1 << 20, 2147483647]), cu_of(new))
    for a, b in zip(before, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    gdn.cache_store(k[:0], v[:0], cache, table, ints([0, 0, 0]))


def filled(gen, totals, heads, d, page, dtype=BF16, width=None, scales="pow2"):
    """A pool that holds random tokens of these sequences, NaN elsewhere."""
    table, pages = tables(gen, totals, page, width=width)
    cache = pool(pages, heads, d, page)
    T = sum(totals)
    gdn.cache_store(rand(gen, T, heads, d, dtype), rand(gen, T, heads, d, dtype), cache, table, ints([0] * len(totals)), cu_of(totals))
    if scales != "pow2":
        for t in cache[2:]:
            t.mul_((0.3 + torch.rand(t.shape, generator=gen)).cuda())
    return cache, table


ATTEND = [
    # new, contexts, h_q, h_kv, d, page, options
    ([1], [1], 1, 1, 64, 16, {}),
    ([1, 1, 1], [777, 64, 65], 24, 4, 256, 64, {}),
    ([1, 1], [5000, 3], 6, 1, 128, 32, dict(return_lse=True)),
    ([1] * 4, [16, 17, 1030, 300], 8, 8, 64, 16, dict(gate=True, return_lse=True)),
    ([3] * 2, [3, 200], 12, 2, 128, 128, dict(return_lse=True)),
    ([5, 0, 40, 1], [5, 9, 300, 130], 4, 2, 64, 64, dict(return_lse=True, gate=True)),
    ([70, 33], [70, 500], 2, 1, 256, 16, {}),
    ([7, 4], [3, 0], 4, 2, 64, 32, dict(return_lse=True)),  # more new tokens than there are in the cache: empty rows
    ([9, 130], [400, 140], 6, 2, 128, 256, dict(window=33, return_lse=True)),
    ([1, 1], [2000, 30], 8, 2, 64, 64, dict(window=100, causal=False, return_lse=True)),
    ([20, 4], [50, 77], 4, 4, 128, 64, dict(causal=False, return_lse=True)),
    ([1], [700], 16, 1, 256, 64, dict(scale=0.9, return_lse=True)),
    ([2, 1], [40, 0], 34, 1, 64, 16, dict(return_lse=True)),
    ([200], [330], 16, 2, 64, 32, dict(return_lse=True)),
    ([150, 2, 90], [150, 900, 91], 6, 1, 128, 64, dict(return_lse=True, gate=True, window=1)),
    ([129], [1000], 3, 3, 256, 64, dict(return_lse=True)),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(case, dtype):
    new, ctx, h_q, h_kv, d, page, how = ATTEND[case]
    gen = torch.Generator().manual_seed(case)
    cache, table = filled(gen, ctx, h_kv, d, page, dtype, scales="any" if case % 2 else "pow2")
    how = dict(how)
    T = sum(new)
    q = torch.randn((T, h_q * d + 16), generator=gen).to(dtype).cuda()[:, :h_q * d].unflatten(1, (h_q, d))
    if how.pop("gate", False):
        how["gate"] = torch.randn((T, h_q, d), generator=gen).to(dtype).cuda()
    cu = None if len(set(new)) == 1 and case % 3 else cu_of(new)
    got = gdn.cache_attention(q, cache, table, ints(ctx), cu, **how)
    how.pop("return_lse", None)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(ctx), cu, **how), f"case {case}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_of_wild_values(dtype):
    """Scales 2^24 apart from page to page, pages of zeros (scale 2^-126), scores far apart."""
    gen = torch.Generator().manual_seed(12)
    d, page, ctx = 64, 16, [160, 97]
    table, pages = tables(gen, ctx, page)
    cache = pool(pages, 1, d, page)
    k, v = rand(gen, sum(ctx), 1, d, dtype, scale=2.0), rand(gen, sum(ctx), 1, d, dtype)
    v[:16] = 0
    v[16:32] *= 2.0 ** -14
    v[32:48] *= 2.0 ** 10
    k[48:64] = 0
    gdn.cache_store(k, v, cache, table, ints([0, 0]), cu_of(ctx))
    q = 3 * torch.randn((6, 2, d), generator=gen).to(dtype).cuda()
    got = gdn.cache_attention(q, cache, table, ints(ctx), return_lse=True)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(ctx)), "wild")
    # only the page of zeros: finite, and zero
    o, lse = gdn.cache_attention(q[:2], cache, table, ints([2, 0]), return_lse=True)
    assert torch.equal(o, torch.zeros_like(o)) and torch.isfinite(lse[0]).all() and torch.isinf(lse[1]).all()


@pytest.mark.parametrize("new", [1, 40])
def test_what_is_not_seen_does_not_reach(new):
    """NaN and the largest codes in keys and values at positions that only some rows see: the others are as without."""
    gen = torch.Generator().manual_seed(13)
    d, page, ctx, heads = 128, 32, 300, 2
    cache, table = filled(gen, [ctx], heads, d, page)
    q = torch.randn((new, 4, d), generator=gen).to(BF16).cuda()
    clean = gdn.cache_attention(q, cache, table, ints([ctx]), return_lse=True)
    at = ctx - 1 - new // 2  # seen by the last new // 2 + 1 rows only
    p, slot = int(table[0, at // page]), at % page
    bad = [t.clone() for t in cache]
    bad[1].view(torch.uint8)[p, 1, 7, slot] = NAN
    o, lse = gdn.cache_attention(q, bad, table, ints([ctx]), return_lse=True)
    hidden = new - 1 - new // 2
    assert torch.equal(o[:hidden], clean[0][:hidden]) and torch.equal(lse, clean[1])
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[hidden:, 2:, 7] = True
    assert torch.equal(torch.isnan(o), hit)
    assert torch.equal(o[~hit], clean[0][~hit])
    # the same for a key: its row is NaN where it is seen
    bad = [t.clone() for t in cache]
    bad[0].view(torch.uint8)[p, 0, slot, 3] = NAN | 0x80
    o, lse = gdn.cache_attention(q, bad, table, ints([ctx]), return_lse=True)
    assert torch.equal(o[:hidden], clean[0][:hidden]) and torch.equal(o[:, 2:], clean[0][:, 2:])
    assert torch.isnan(o[hidden:, :2]).all() and torch.isnan(lse[hidden:, :2]).all()


def test_pages_outside_and_padded_rows():
    """A page outside the pool holds no tokens; rows behind the last sequence keep what they hold."""
    gen = torch.Generator().manual_seed(14)
    d, page, heads = 64, 16, 2
    ctx = [100, 90]
    cache, table = filled(gen, ctx, heads, d, page, width=9)
    table[0, 2], table[1, 0], table[1, 4] = -1, 1 << 30, cache.k.shape[0]
    new = [5, 20]
    T = 33
    q = torch.randn((T, 4, d), generator=gen).to(BF16).cuda()
    out = torch.full_like(q, 7.0)
    got = gdn.cache_attention(q, cache, table, ints(ctx), cu_of(new), out=out, return_lse=True)
    want = ref.cache_attention(q, cache, table, ints(ctx), cu_of(new))
    ref.close_attention(got, want, "outside")
    assert torch.all(out[25:] == 7.0)
    # a context that passes the table's end is cut there
    got = gdn.cache_attention(q[:2], cache, table[:, :2].contiguous(), ints([32, 100]), return_lse=True)
    ref.close_attention(got, ref.cache_attention(q[:2], cache, table[:, :2], ints([32, 32])), "table's end")
    # in place over q
    q2 = q.clone()
    assert gdn.cache_attention(q2, cache, table, ints(ctx), cu_of(new), out=q2) is q2
    assert torch.equal(q2[:25], out[:25]) and torch.equal(q2[25:], q[25:])


def test_prefill_equals_decode_and_serving_run():
    """The operators as a program uses them: norm, rope, store, attention, token by token and in chunks; a joined
    run of whole prompt and single tokens gives what one chunk gives."""
    gen = torch.Generator().manual_seed(15)
    h_q, h_kv, d, page, T, rot = 6, 2, 128, 32, 75, 32
    inv, _ = gdn.rope_frequencies(rot, 1e4, device="cuda")
    w = (1 + 0.1 * torch.randn(d, generator=gen)).cuda()
    q0, k0 = rand(gen, T, h_q, d, BF16), rand(gen, T, h_kv, d, BF16)
    v0, z0 = rand(gen, T, h_kv, d, BF16), rand(gen, T, h_q, d, BF16)
    table = ints([[2, 0, 1]])

    def run(cuts):
        cache, done, outs = pool(3, h_kv, d, page), 0, []
        for n in cuts:
            s = slice(done, done + n)
            pos = torch.arange(done, done + n, device="cuda")
            q, k = gdn.rope(gdn.rms_norm(q0[s], w), pos, inv, k=gdn.rms_norm(k0[s], w))
            gdn.cache_store(k, v0[s], cache, table, ints([done]))
            done += n
            outs.append(gdn.cache_attention(q, cache, table, ints([done]), gate=z0[s]))
        return torch.cat(outs), cache

    whole, cache = run([T])
    steps, cache2 = run([40] + [1] * 30 + [5])
    # a page filled in steps may have been rounded by a smaller scale first: the scales end up the same, the codes
    # may differ by a subnormal rounding, and earlier tokens saw the page as it was then: e4m3 steps, 2^-4 relative
    assert torch.equal(cache.k_scale, cache2.k_scale) and torch.equal(cache.v_scale, cache2.v_scale)
    a, b = cache.k.float() * cache.k_scale[..., None, None], cache2.k.float() * cache2.k_scale[..., None, None]
    live = torch.isfinite(a)
    # two roundings of a value among the subnormals: half a step each, of 2^-9 of the scale
    step = (cache.k_scale * 2.0 ** -9)[..., None, None].expand_as(a)
    assert ((a - b).abs()[live] <= (a.abs() * 2.0 ** -4 + step)[live]).all()
    ref.close_attention(whole[:1], tuple(t[:1] for t in ref.cache_attention(
        gdn.rope(gdn.rms_norm(q0[:1], w), ints([0]), inv), cache, table, ints([1]), gate=z0[:1])), "first")
    assert (whole.float() - steps.float()).abs().max() < 0.1


def test_deterministic_graph_stream_and_workspace():
    gen = torch.Generator().manual_seed(16)
    h_q, h_kv, d, page, ctx = 12, 2, 128, 64, [3000, 1500, 7, 2000]
    cache, table = filled(gen, ctx, h_kv, d, page)
    q = torch.randn((4, h_q, d), generator=gen).to(BF16).cuda()
    k, v = rand(gen, 4, h_kv, d, BF16), rand(gen, 4, h_kv, d, BF16)
    lens = ints(ctx)
    need = gdn.cache_attention_workspace_size(4, 4, table.shape[1], h_q, h_kv, d, page)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert need > 0
    want = gdn.cache_attention(q, cache, table, lens, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(gdn.cache_attention(q, cache, table, lens), want)
    torch.cuda.current_stream().wait_stream(side)
    held = lens - 1
    stored = [t.clone() for t in cache]
    gdn.cache_store(k, v, stored, table, held)
    after = gdn.cache_attention(q, stored, table, lens)
    base = [t.clone() for t in cache]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.cache_store(k, v, cache, table, held)
        got = gdn.cache_attention(q, cache, table, lens)
    for _ in range(3):
        for t, b in zip(cache, base):
            t.copy_(b)
        got.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, after)
        for t, s in zip(cache, stored):
            assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
        gdn.cache_attention(q, cache, table, lens - 3)  # eager work between the replays
    # lengths move on between replays
    lens.sub_(4), held.sub_(4)
    graph.replay()
    assert torch.equal(got, gdn.cache_attention(q, cache, table, lens))


def test_refusals():
    cache = gdn.kv_cache(4, 2, 64, 16)
    table, lens = ints([[0, 1], [2, 3]]), ints([3, 4])
    k = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    q = torch.zeros((2, 4, 64), dtype=BF16, device="cuda")
    for bad in [dict(k=k.half()), dict(v=k[:1]), dict(v=k.float()), dict(cache=cache[:3]), dict(page_table=table.long()), dict(lens=lens[:1]),
                dict(cu_seqlens=lens), dict(k=k[:, :1], v=k[:, :1]), dict(lens=lens.cpu()), dict(k=k.cpu()),
                dict(cache=(cache.v, cache.k, *cache[2:])), dict(k=k.transpose(0, 1)), dict(k=k.repeat(2, 1, 1)[:3], v=k.repeat(2, 1, 1)[:3]),
                dict(cache=(cache.k.view(torch.uint8), *cache[1:])), dict(page_table=table[0]), dict(lens=None)]:
        with pytest.raises(gdn.GdnError):
            gdn.cache_store(**{**dict(k=k, v=k, cache=cache, page_table=table, lens=lens), **bad})
    for bad in [dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(gate=q.float()), dict(scale=-1.0), dict(window=-1),
                dict(workspace=q), dict(out=q[:1]), dict(cache=gdn.kv_cache(4, 2, 64, 16)[:3]), dict(lens=ints([1])), dict(q=q.cpu())]:
        with pytest.raises(gdn.GdnError):
            gdn.cache_attention(**{**dict(q=q, cache=cache, page_table=table, lens=lens), **bad})


SHARED = [
    # contexts, new, h_q, h_kv, d, page, options: tables wide enough that the work is cut into shares
    ([3000, 17, 0, 900], 1, 24, 4, 256, 64, {}),
    ([500, 1200, 33, 64, 0, 2047], 1, 8, 8, 128, 16, dict(window=300)),
    ([700, 90], 9, 16, 8, 64, 32, dict(gate=True)),
    ([5000], 1, 6, 1, 256, 128, {}),
    ([100] * 40, 1, 8, 2, 128, 256, {}),
    ([4000, 5] * 3, 3, 1, 1, 64, 64, dict(causal=False)),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_attention_in_shares(case, dtype):
    """Contexts of unequal lengths under a table for far longer ones, pages outside the pool among them."""
    ctx, new, h_q, h_kv, d, page, how = SHARED[case]
    gen = torch.Generator().manual_seed(50 + case)
    cache, table = filled(gen, ctx, h_kv, d, page, dtype, width=8192 * 64 // page // 16 * 4)
    table[0, 1] = -1
    how = dict(how)
    q = torch.randn((len(ctx) * new, h_q, d), generator=gen).to(dtype).cuda()
    if how.pop("gate", False):
        how["gate"] = torch.randn(q.shape, generator=gen).to(dtype).cuda()
    got = gdn.cache_attention(q, cache, table, ints(ctx), return_lse=True, **how)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(ctx), **how), f"shares {case}")
    again = gdn.cache_attention(q, cache, table, ints(ctx), return_lse=True, **how)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


CHUNKS = [
    # new, contexts, h_q, h_kv, d, page, options: rows enough to share a workgroup's tiles
    ([200], [100], 4, 2, 64, 64, {}),                      # rows whose position lies before the first token
    ([100, 37], [60, 37], 40, 1, 128, 32, {}),             # 40 heads to one, empty rows among them
    ([300], [301], 3, 3, 128, 64, dict(gate=True)),        # heads that do not divide the XCDs
    ([64, 64], [64, 700], 16, 16, 64, 16, {}),
    ([130], [1500], 8, 2, 256, 128, dict(window=1)),
    ([130], [1500], 8, 2, 128, 16, dict(window=700, gate=True)),
    ([90, 80], [500, 80], 8, 2, 256, 32, dict(causal=False, window=90)),
    ([513], [1024], 2, 1, 64, 256, dict(scale=0.7)),
    ([1000], [1000], 6, 1, 128, 64, {}),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunks(case, dtype):
    """Chunks of prompts: strided queries, gates and outputs, every page size, contexts cut into pieces."""
    new, ctx, h_q, h_kv, d, page, how = CHUNKS[case]
    gen = torch.Generator().manual_seed(70 + case)
    cache, table = filled(gen, ctx, h_kv, d, page, dtype, scales="any")
    how, T = dict(how), sum(new)

    def strided():
        return torch.randn((T, h_q * d + 24), generator=gen).to(dtype).cuda()[:, 8:8 + h_q * d].unflatten(1, (h_q, d))

    q = strided()
    if how.pop("gate", False):
        how["gate"] = strided()
    out = torch.full((T + 2, h_q, d + 0), 7.0, dtype=dtype, device="cuda")
    cu = cu_of(new)
    got = gdn.cache_attention(q, cache, table, ints(ctx), cu, out=out[:T], return_lse=True, **how)
    assert got[0].data_ptr() == out.data_ptr() and torch.all(out[T:] == 7.0)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(ctx), cu, **how), f"chunk {case}")


def test_nan_in_a_chunk():
    """A NaN among the values of a chunk's own tokens reaches the rows from that token on, and a page that two tiles of
    rows share is not changed for the next."""
    gen = torch.Generator().manual_seed(80)
    d, page, T, heads = 64, 64, 300, 2
    cache, table = filled(gen, [T], heads, d, page)
    q = torch.randn((T, 4, d), generator=gen).to(BF16).cuda()
    clean = gdn.cache_attention(q, cache, table, ints([T]))
    bad = [t.clone() for t in cache]
    spots = [(10, 0, 5), (100, 1, 63), (101, 1, 0), (299, 0, 33)]
    for at, head, c in spots:
        bad[1].view(torch.uint8)[int(table[0, at // page]), head, c, at % page] = NAN
    o = gdn.cache_attention(q, bad, table, ints([T]))
    hit = torch.zeros_like(o, dtype=torch.bool)
    for at, head, c in spots:
        hit[at:, 2 * head:2 * head + 2, c] = True
    assert torch.equal(torch.isnan(o), hit) and torch.equal(o[~hit], clean[~hit])


def test_many_sequences():
    """More sequences than a wave looks at at once, most of them with no or few new tokens."""
    gen = torch.Generator().manual_seed(81)
    n, page, d = 300, 16, 64
    new = torch.randint(0, 4, (n,), generator=gen).tolist()
    new[7], new[150], new[299] = 40, 0, 9
    old = torch.randint(0, 50, (n,), generator=gen).tolist()
    total = [a + b for a, b in zip(new, old)]
    table, pages = tables(gen, total, page)
    cache = pool(pages, 1, d, page)
    k = rand(gen, sum(old), 1, d, BF16)
    check_store(k, -k, cache, table, ints([0] * n), cu_of(old), "old")
    k = rand(gen, sum(new) + 5, 1, d, BF16, scale=4.0)  # a padded batch
    check_store(k, k, cache, table, ints(old), cu_of(new), "new")
    q = torch.randn((sum(new), 2, d), generator=gen).to(BF16).cuda()
    got = gdn.cache_attention(q, cache, table, ints(total), cu_of(new), return_lse=True)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(total), cu_of(new)), "many")


def test_offsets_beyond_32_bits():
    """Pages of a pool beyond 4 GiB of codes."""
    gen = torch.Generator().manual_seed(82)
    heads, d, page, pages = 4, 256, 64, 66000
    assert pages * heads * d * page > 1 << 32
    big = gdn.KVCache(torch.empty((pages, heads, page, d), dtype=torch.uint8, device="cuda").view(FP8),
                      torch.empty((pages, heads, d, page), dtype=torch.uint8, device="cuda").view(FP8),
                      torch.empty((pages, heads), device="cuda"), torch.empty((pages, heads), device="cuda"))
    small = pool(4, heads, d, page)
    far = ints([[pages - 1, pages - 3], [pages - 2, 65537]])
    near = ints([[0, 1], [2, 3]])
    for new in (1, 100):
        T = 2 * new
        k, v = rand(gen, T, heads, d, BF16), rand(gen, T, heads, d, BF16)
        held = [0, 0] if new == 100 else [100, 100]
        q = torch.randn((T, 24, d), generator=gen).to(BF16).cuda()
        for c, t in ((big, far), (small, near)):
            if new == 1:
                gdn.cache_store(k.repeat(100, 1, 1), v.repeat(100, 1, 1), c, t, ints([0, 0]))
            gdn.cache_store(k, v, c, t, ints(held))
        lens = ints([h + new for h in held])
        assert torch.equal(gdn.cache_attention(q, big, far, lens), gdn.cache_attention(q, small, near, lens))
        for n in range(2):
            for j in range(2):
                a, b = int(far[n, j]), int(near[n, j])
                tokens = min(max(int(lens[n]) - j * page, 0), page)
                assert torch.equal(big.k[a].view(torch.uint8)[:, :tokens], small.k[b].view(torch.uint8)[:, :tokens])
                assert torch.equal(big.v[a].view(torch.uint8)[..., :tokens], small.v[b].view(torch.uint8)[..., :tokens])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,width", [([1, 1], None), ([1, 1], 40), ([1, 1], 2048), ([70, 40], None)])  # whole, pieces, shares, a chunk
@pytest.mark.parametrize("sizes", [(1e37,), (1e-22,), (1.0, 1e37), (1e37, 1.0, 1e30, 0.0), (0.0,), (0.0, 1.0)])
def test_sizes_of_values(sizes, new, width, dtype):
    """Values from the type's largest to its small ones, pages of zeros among them: e^(score - max) of what counts
    passes neither end of fp32, whatever the maximum of score + log scale is."""
    gen = torch.Generator().manual_seed(90)
    page, d, heads, ctx = 64, 64, 2, [777, 300]
    table, pages = tables(gen, ctx, page, width=width)
    cache = pool(pages, heads, d, page)
    T = sum(ctx)
    k, v = rand(gen, T, heads, d, dtype), torch.randn((T, heads, d), generator=gen)
    size = torch.tensor(sizes).repeat(-(-T // page // len(sizes)) + 1).repeat_interleave(page)[:T]
    v = (v.clamp(-3, 3) * size[:, None, None]).to(dtype).cuda()
    gdn.cache_store(k, v, cache, table, ints([0, 0]), cu_of(ctx))
    q = (2.0 * torch.randn((sum(new), 4, d), generator=gen)).to(dtype).cuda()
    cu = None if new[0] == 1 else cu_of(new)
    got = gdn.cache_attention(q, cache, table, ints(ctx), cu, return_lse=True)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(ctx), cu), str(sizes))


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [100, 60]])
def test_windows_of_any_size(new):
    """A window as wide as 32 bits allow is none at all, also for rows whose position lies before the first token."""
    gen = torch.Generator().manual_seed(91)
    cache, table = filled(gen, [1500, 50], 2, 64, 64)
    q = torch.randn((sum(new), 8, 64), generator=gen).to(BF16).cuda()
    for causal in (True, False):
        want = gdn.cache_attention(q, cache, table, ints([1500, 50]), cu_of(new), causal=causal)
        for window in (1501, 2 ** 30, 2 ** 31 - 1):
            assert torch.equal(gdn.cache_attention(q, cache, table, ints([1500, 50]), cu_of(new), causal=causal, window=window), want)


@pytest.mark.parametrize("new", [[5, 20, 0, 1], [150, 40, 0, 200]])
def test_pack_that_begins_behind_the_first_token(new):
    """Offsets that start above 0: the tokens ahead of the first sequence and behind the last are left alone."""
    gen = torch.Generator().manual_seed(92)
    page, d, skip, behind = 16, 64, 100, 30
    old = [3, 50, 7, 31]
    total = [a + b for a, b in zip(old, new)]
    cu = cu_of(new) + skip
    cu = cu.to(torch.int32)
    table, pages = tables(gen, total, page)
    cache = pool(pages, 2, d, page)
    k = rand(gen, sum(old), 2, d, BF16)
    check_store(k, -k, cache, table, ints([0] * 4), cu_of(old), "old")
    T = skip + sum(new) + behind
    k = rand(gen, T, 2, d, BF16, scale=3.0)
    check_store(k, -k, cache, table, ints(old), cu, "new")
    q = torch.randn((T, 8, d), generator=gen).to(BF16).cuda()
    out = torch.full_like(q, 7.0)
    got = gdn.cache_attention(q, cache, table, ints(total), cu, out=out, return_lse=True)
    assert torch.all(out[:skip] == 7.0) and torch.all(out[skip + sum(new):] == 7.0)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(total), cu), "offset")


@pytest.mark.parametrize("window", [1, 63, 64, 65, 300, 1000])
@pytest.mark.parametrize("new,h_q", [([1] * 3, 4), ([5, 0, 9], 2), ([1] * 3, 40), ([60, 33, 1], 6), ([300, 1, 131], 2)])
def test_windows_in_long_tables(new, h_q, window):
    """Windows well inside long contexts and longer tables: pieces are cut for the window's keys."""
    gen = torch.Generator().manual_seed(93)
    ctx = [2000, 1, 1537]
    cache, table = filled(gen, ctx, 2, 64, 32, width=400)
    q = torch.randn((sum(new), h_q, 64), generator=gen).to(BF16).cuda()
    cu = None if len(set(new)) == 1 else cu_of(new)
    need = gdn.cache_attention_workspace_size(sum(new), 3, 400, h_q, 2, 64, 32, cu is not None, window=window)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda") if need else None
    got = gdn.cache_attention(q, cache, table, ints(ctx), cu, window=window, return_lse=True, workspace=ws)
    ref.close_attention(got, ref.cache_attention(q, cache, table, ints(ctx), cu, window=window), f"window {window}")


def test_graphs_that_share_a_workspace():
    """Two captured calls (shares, and pieces of a chunk) with one workspace, replayed in turn with eager work between."""
    gen = torch.Generator().manual_seed(94)
    ctx, d, page = [900, 1500], 64, 64
    cache, table = filled(gen, ctx, 2, d, page, width=2048)
    calls = []
    for new in ([1, 1], [120, 7]):
        q = torch.randn((sum(new), 8, d), generator=gen).to(BF16).cuda()
        calls.append((q, None if new == [1, 1] else cu_of(new), torch.empty_like(q)))
    need = [gdn.cache_attention_workspace_size(q.shape[0], 2, 2048, 8, 2, d, page, cu is not None) for q, cu, _ in calls]
    assert min(need) > 0
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    want = [gdn.cache_attention(q, cache, table, ints(ctx), cu) for q, cu, _ in calls]
    lens, graphs = ints(ctx), []
    torch.cuda.synchronize()
    for q, cu, out in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.cache_attention(q, cache, table, lens, cu, out=out, workspace=ws)
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1) if turn % 2 else (1, 0):
            calls[i][2].fill_(float("nan"))
            graphs[i].replay()
        for i in range(2):
            assert torch.equal(calls[i][2], want[i]), (turn, i)
        ws.fill_(0xFF)
        gdn.cache_attention(calls[0][0], cache, table, lens, None, workspace=ws)
        torch.cuda.synchronize()
