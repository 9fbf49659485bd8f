"""Cases and plain forms of the operators that stand around the Gated DeltaNet mixer in a hybrid block:

  norm    rms_norm / rms_norm_backward: RMS norm fused with residual sum, residual scale and output gate
  rope    rope / rope_backward: rotary positions on the attention layer's q and k
  store   cache_store: new keys and values into the pages of an 8-bit cache (e4m3, one scale a page and head)
  attend  cache_attention: attention of the newest queries over that cache

A pass of a plain form is elementary torch in float32; `exact` is the definition in float64.  Shapes are those of
the repository's 9B and 27B layers (widths 5120, heads of 128; 24 query and 4 KV heads of 256 with a quarter of
each head rotated, 256 decoding sequences) and generic ones.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
FP8_MAX = 448.0


def listed():
    return [
        # the residual sum and norm ahead of a mixer for one decoding sequence: latency alone
        norm("norm_one_token", tokens=1, width=5120, residual=True),
        # the mixer's output norm and SiLU gate in a decode step of 256 sequences, 48 heads of 128
        norm("norm_gate_decode", tokens=256, heads=48, width=128, gate="silu", pad=2048),
        # residual sum and norm of a long prompt
        norm("norm_residual_prompt", tokens=16384, width=5120, residual=True, scale=0.5),
        # training: gradients of the output norm and gate of the 9B layer at 8192 tokens
        norm("norm_gate_backward", tokens=8192, heads=32, width=128, gate="silu", backward=True),
        # one decode step of 256 sequences, a quarter of each head rotated, positions up to 262144
        rope("rope_decode", tokens=256, far=262144),
        # a 65536-token prompt
        rope("rope_prompt", tokens=65536, far=65536),
        # training: the whole head rotated, neighbouring elements paired, fp32, an odd number of tokens
        rope("rope_backward", tokens=8191, far=8191, h_q=16, h_k=16, d=64, rot=64, layout="interleaved", dtype="f32",
             backward=True),
        # one new token for each of 256 sequences
        store("store_decode", seqs=256, tokens=256, old=1024),
        # a pack of 8 prompts of unequal lengths that continue short ones
        store("store_prompt", seqs=8, tokens=65536, ragged=True, old=500),
        # one new token of one sequence
        attend("attend_one_token", seqs=1, tokens=1, ctx_min=777, ctx_max=777),
        # a decode step of 64 sequences with long contexts of unequal lengths, output gate
        attend("attend_decode", seqs=64, tokens=64, ctx_min=4096, ctx_max=32768, gate=True),
        # a chunk of 4096 tokens of a prompt of which 4001 are cached already
        attend("attend_chunk", seqs=1, tokens=4096, ctx_min=8097, ctx_max=8097),
    ]


def norm(name=None, tokens=1, heads=1, width=5120, gate="", residual=False, order="pre", scale=1.0, pad=0, dtype="bf16",
         backward=False):
    return _case(name, op="norm", tokens=tokens, heads=heads, width=width, gate=gate, residual=residual, order=order,
                 scale=scale, pad=pad, dtype=dtype, backward=backward)


def rope(name=None, tokens=1, far=4096, h_q=24, h_k=4, d=256, rot=64, layout="half", dtype="bf16", backward=False,
         base=1e7, mscale=1.0):
    return _case(name, op="rope", tokens=tokens, far=far, h_q=h_q, h_k=h_k, d=d, rot=rot, layout=layout, dtype=dtype,
                 backward=backward, base=base, mscale=mscale)


def store(name=None, seqs=1, tokens=1, ragged=False, old=0, h_k=4, d=256, page=64, dtype="bf16", lens=1):
    return _case(name, op="store", seqs=seqs, tokens=tokens, ragged=ragged, old=old, h_k=h_k, d=d, page=page,
                 dtype=dtype, lens=lens)


def attend(name=None, seqs=1, tokens=1, ragged=False, ctx_min=1, ctx_max=1, h_q=24, h_k=4, d=256, page=64, causal=True,
           window=0, gate=False, lse=False, dtype="bf16", lens=1):
    return _case(name, op="attend", seqs=seqs, tokens=tokens, ragged=ragged, ctx_min=ctx_min, ctx_max=ctx_max, h_q=h_q,
                 h_k=h_k, d=d, page=page, causal=causal, window=window, gate=gate, lse=lse, dtype=dtype, lens=lens)


def _case(name, **fields):
    return dict({} if name is None else {"name": name}, **fields)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "store", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        heads = rng.choice([1, 1, rng.randint(2, 48)])
        width = _log(rng, 64, 8192) if heads == 1 else rng.choice([64, 128, 256, rng.randint(33, 300)])
        most = (40 if dtype == "bf16" else 20) * (1 << 20)
        order = rng.choice(["pre", "pre", "post"])
        residual = order == "post" or rng.random() < 0.5
        return norm(tokens=_log(rng, 1, most // (heads * width)), heads=heads, width=width,
                    gate=rng.choice(["", "silu", "sigmoid"]), residual=residual, order=order,
                    scale=round(rng.uniform(0.1, 1.5), 3) if residual else 1.0, pad=rng.choice([0, 0, 8 * rng.randint(1, 64), 3]),
                    dtype=dtype, backward=rng.random() < 0.5)
    if op == "rope":
        d = rng.choice([64, 128, 256, 2 * rng.randint(20, 100)])
        h_k = rng.randint(1, 8)
        h_q = h_k * rng.randint(1, 6)
        return rope(tokens=_log(rng, 1, 40 * (1 << 20) // ((h_q + h_k) * d)), far=_log(rng, 128, 1 << 20), h_q=h_q, h_k=h_k, d=d,
                    rot=rng.choice([d, d // 4 * 2, 2 * rng.randint(4, d // 2)]), layout=rng.choice(["half", "interleaved"]),
                    dtype=dtype, backward=rng.random() < 0.4, base=rng.choice([1e4, 5e5, 1e7]), mscale=rng.choice([1.0, 1.2]))
    h_k = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randint(0, 1 << 30)
    if op == "store":
        seqs = _log(rng, 1, 256)
        tokens = seqs * rng.choice([1, 1, rng.randint(2, 6), _log(rng, 2, max(3, 16384 // seqs))])
        return store(seqs=seqs, tokens=tokens, ragged=rng.random() < 0.5, old=rng.choice([0, 60, 1000]), h_k=h_k, d=d, page=page,
                     dtype=dtype, lens=lens)
    while True:
        new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
        ctx = _log(rng, max(new, 16), 32768 if new < 9 else 8192)
        c = attend(seqs=(seqs := _log(rng, 1, 64)), tokens=seqs * new, ragged=new > 1 and rng.random() < 0.5,
                   ctx_min=max(1, ctx // rng.choice([1, 4, 16])), ctx_max=ctx, h_q=h_k * rng.choice([1, 2, 4, 6, 8]), h_k=h_k, d=d,
                   page=page, causal=rng.random() < 0.9, window=rng.choice([0, 0, 0, rng.randint(1, 2 * ctx)]),
                   gate=rng.random() < 0.4, lse=rng.random() < 0.4, dtype=dtype, lens=lens)
        longest, keys = max(new_lengths(c)), max(context_lengths(c))
        # the plain form holds every score of the padded pack, and the pack's keys and values in 32 bits
        if seqs * c["h_q"] * longest * keys < 1 << 30 and seqs * h_k * keys * d < 1 << 30 and work(c)["flops"] < 3e11:
            return c


# ---- the lengths of a pack: a matter of the case, not of the seed --------------------------------------------------


def new_lengths(c):
    """New tokens of each sequence."""
    n, t = c["seqs"], c["tokens"]
    if not c["ragged"]:
        return [t // n] * n
    cuts = sorted(random.Random(c["lens"]).randint(0, t) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


def old_lengths(c):
    """Tokens that each sequence has in the cache already (store)."""
    r = random.Random(c["lens"] + 1)
    return [r.randint(0, c["old"]) for _ in range(c["seqs"])]


def context_lengths(c):
    """Tokens of each sequence, the new ones among them (attend)."""
    r = random.Random(c["lens"] + 2)
    lo, hi = math.log(c["ctx_min"]), math.log(c["ctx_max"])
    return [max(new, int(round(math.exp(r.uniform(lo, hi))))) for new in new_lengths(c)]


def visible(c):
    """(pairs of a query and a key that it sees, cached tokens that some query sees)."""
    pairs = read = 0
    for new, ctx in zip(new_lengths(c), context_lengths(c)):
        if not new:
            continue
        first = ctx - new
        w = c["window"] or ctx + 1
        read += ctx - max(0, first - w + 1)
        for at in range(first, ctx):
            pairs += (at + 1 if c["causal"] else ctx) - max(0, at - w + 1)
    return pairs, read


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        n = c["tokens"] * c["heads"] * c["width"]
        arrays = 2 + (c["gate"] != "")
        if c["backward"]:
            arrays += 1 + (c["gate"] != "") + (2 if c["residual"] and c["order"] == "pre" else 0)
        elif c["residual"]:
            arrays += 2 if c["order"] == "pre" else 1
        return {"bytes": n * es * arrays + c["width"] * (es + (4 if c["backward"] else 0)), "flops": n * (20 if c["backward"] else 8)}
    if c["op"] == "rope":
        n = c["tokens"] * (c["h_q"] + c["h_k"]) * c["d"]
        return {"bytes": 2 * n * es + 8 * c["tokens"] + 4 * c["rot"], "flops": n * 3}
    if c["op"] == "store":
        n = 2 * c["tokens"] * c["h_k"] * c["d"]
        return {"bytes": n * es + n + 8 * n // (c["page"] * c["d"]), "flops": 3 * n}
    pairs, read = visible(c)
    q = c["tokens"] * c["h_q"] * c["d"] * es
    return {"bytes": 2 * read * c["h_k"] * c["d"] + 8 * read // c["page"] * c["h_k"] + q * (3 if c["gate"] else 2),
            "flops": 4 * pairs * c["h_q"] * c["d"]}


# ---- inputs --------------------------------------------------------------------------------------------------------


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, of=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(of)

    s = {"case": c}
    if c["op"] == "norm":
        shape = (c["tokens"], c["heads"], c["width"])
        cols = c["heads"] * c["width"]

        def rows():  # columns of a wider projection's output, where the case says so
            return normal(c["tokens"], cols + c["pad"], of=dt)[:, :cols].unflatten(1, shape[1:])

        s["x"] = rows()
        s["weight"] = (1 + 0.1 * normal(c["width"])).to(dt)
        s["gate"] = rows() if c["gate"] else None
        s["residual"] = (4 * normal(*shape)).to(dt) if c["residual"] and not c["backward"] else None
        s["dy"] = normal(*shape, of=dt) if c["backward"] else None
        s["d_sum"] = normal(*shape, of=dt) if c["backward"] and c["residual"] and c["order"] == "pre" else None
        return s
    if c["op"] == "rope":
        s["q"] = normal(c["tokens"], c["h_q"], c["d"], of=dt)
        s["k"] = normal(c["tokens"], c["h_k"], c["d"], of=dt)
        s["inv_freq"] = c["base"] ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device="cuda")
        return s
    new = new_lengths(c)
    s["max_new"] = max(new)
    s["cu"] = torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32, device="cuda") if c["ragged"] else None
    h, d, page = c["h_k"], c["d"], c["page"]
    if c["op"] == "store":
        old = old_lengths(c)
        total = [a + b for a, b in zip(old, new)]
        s["lens"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        # channels of unequal size, as keys have them
        size = torch.exp(0.5 * normal(2, 1, h, d))
        s["k"], s["v"] = ((normal(c["tokens"], h, d) * size[i]).to(dt) for i in (0, 1))
    else:
        total = context_lengths(c)
        s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        s["q"] = normal(c["tokens"], c["h_q"], d, of=dt)
        s["gate"] = normal(c["tokens"], c["h_q"], d, of=dt) if c["gate"] else None
        s["scale"] = d ** -0.5
    per = [-(-t // page) for t in total]
    pages, width = sum(per) + 1, max(1, max(per))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(per[:i]) for i in range(len(per))], device="cuda")
    col = torch.arange(width, device="cuda")
    used = col < torch.tensor(per, device="cuda")[:, None]
    s["table"] = torch.where(used, order[(at[:, None] + col).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    for side, shape in (("k", (pages, h, page, d)), ("v", (pages, h, d, page))):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        step = 1024
        for p in range(0, pages, step):
            codes[p:p + step] = (normal(*codes[p:p + step].shape) * 80).clamp(-FP8_MAX, FP8_MAX).to(codes.dtype)
        s[side + "_cache"] = codes
        # a store leaves powers of two; a cache written by others has any scale
        scale = torch.rand((pages, h), generator=g, device="cuda") + 0.5
        s[side + "_scale"] = torch.exp2(torch.round(torch.log2(scale)) - 7) if c["op"] == "store" else scale / 80
    s["cache"] = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    if c["op"] == "norm":
        return _norm_backward(s, c) if c["backward"] else _norm(s, c)
    return {"rope": _rope, "store": _store, "attend": _attend}[c["op"]](s, c)


def _own(s, c):
    import linear_attention_token_conv1d_amd as gdn

    if c["op"] == "norm":
        how = dict(order=c["order"], activation=c["gate"] or "silu", scale=c["scale"], eps=EPS)
        if c["backward"]:
            return gdn.rms_norm_backward(s["x"], s["dy"], s["weight"], gate=s["gate"], d_sum=s["d_sum"], **how)
        return gdn.rms_norm(s["x"], s["weight"], gate=s["gate"], residual=s["residual"], **how)
    if c["op"] == "rope":
        f = gdn.rope_backward if c["backward"] else gdn.rope
        return f(s["q"], s["positions"], s["inv_freq"], k=s["k"], layout=c["layout"], mscale=c["mscale"])
    if c["op"] == "store":
        gdn.cache_store(s["k"], s["v"], s["cache"], s["table"], s["lens"], cu_seqlens=s["cu"])
        return s["cache"]
    return gdn.cache_attention(s["q"], s["cache"], s["table"], s["lens"], cu_seqlens=s["cu"], scale=s["scale"], causal=c["causal"],
                               window=c["window"], gate=s["gate"], return_lse=c["lse"])


def _act(c, z):
    return z * torch.sigmoid(z) if c["gate"] == "silu" else torch.sigmoid(z)


def _norm(s, c):
    """h = residual + scale x, y = norm(h) weight act(gate); or y = residual + scale norm(x) weight act(gate)."""
    dt = s["x"].dtype
    h = s["x"].float()
    pre = c["order"] == "pre"
    if pre and s["residual"] is not None:
        h = s["residual"].float() + c["scale"] * h
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["gate"] is not None:
        y = y * _act(c, s["gate"].float())
    if pre:
        return y.to(dt) if s["residual"] is None else (y.to(dt), h.to(dt))
    return (s["residual"].float() + c["scale"] * y).to(dt)


def _norm_backward(s, c):
    """Gradients of x (of the sum, where there is one), the weight and the gate."""
    dt = s["x"].dtype
    x, w, dy = s["x"].float(), s["weight"].float(), s["dy"].float()
    if c["order"] == "post":
        dy = dy * c["scale"]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    z = None if s["gate"] is None else s["gate"].float()
    a = None if z is None else _act(c, z)
    u = dy * w if z is None else dy * w * a
    dh = r * (u - n * (u * n).mean(-1, keepdim=True))
    dw = dy * n if z is None else dy * n * a
    grads = []
    if s["d_sum"] is not None:
        dh = dh + s["d_sum"].float()
        grads = [(c["scale"] * dh).to(dt), dh.to(dt)]
    else:
        grads = [dh.to(dt), None]
    dz = None
    if z is not None:
        p = torch.sigmoid(z)
        slope = p * (1 + z * (1 - p)) if c["gate"] == "silu" else p * (1 - p)
        dz = (dy * n * w * slope).to(dt)
    return (*grads, dw.sum((0, 1)), dz)


def _turn(x, cos, sin, layout, rot, dt):
    x = x.float()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((p, q), -1) if layout == "half" else torch.stack((p, q), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1).to(dt)


def _rope(s, c):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = ((c["mscale"] * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    sin = -sin if c["backward"] else sin
    return tuple(_turn(s[n], cos, sin, c["layout"], c["rot"], s[n].dtype) for n in ("q", "k"))


def _where(s, tokens):
    """Each new token's sequence and its place among that sequence's new ones; the sequences' numbers of new tokens."""
    n = s["table"].shape[0]
    t = torch.arange(tokens, device=s["table"].device)
    if s["cu"] is None:
        return t // (tokens // n), t % (tokens // n), torch.full((n,), tokens // n, device=t.device)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, t - cu[seq], cu[1:] - cu[:-1]


def _store(s, c):
    """A page's scale is the least power of two that takes its largest value to 448, never less than it was for the
    tokens that the page has already, whose codes are rounded anew where it grows."""
    page, lens, table = c["page"], s["lens"].long(), s["table"].long()
    seq, off, _ = _where(s, c["tokens"])
    at = lens[seq] + off
    to, slot = table[seq, at // page], at % page
    rows = ((lens % page > 0) & (lens // page < table.shape[1])).nonzero()[:, 0]  # sequences whose last page has room
    last, kept = table[rows, lens[rows] // page], lens[rows] % page
    for x, codes, scales, token in ((s["k"].float(), s["k_cache"], s["k_scale"], 2), (s["v"].float(), s["v_cache"], s["v_scale"], 3)):
        most = torch.full_like(scales, -1.0).scatter_reduce_(0, to[:, None].expand(-1, c["h_k"]), x.abs().amax(-1), "amax")
        m, e = torch.frexp(most)
        e = torch.where(most > 0, torch.where(m > 0.875, e - 8, e - 9), -126).clamp(min=-126)
        held = torch.zeros_like(scales)
        held[last] = scales[last]
        fresh = torch.where(most < 0, scales, torch.maximum(torch.ldexp(torch.ones_like(most), e), held))
        raw = codes.view(torch.uint8)
        was = raw[last]
        again = (was.view(codes.dtype).float() * (scales[last] / fresh[last])[..., None, None]).to(codes.dtype).view(torch.uint8)
        old = torch.arange(page, device=x.device) < kept[:, None]
        raw[last] = torch.where(old[:, None, :, None] if token == 2 else old[:, None, None, :], again, was)
        new = (x / fresh[to][..., None]).clamp(-FP8_MAX, FP8_MAX).to(codes.dtype).view(torch.uint8)
        if token == 2:
            raw[to, :, slot] = new
        else:
            raw[to, :, :, slot] = new
        scales.copy_(fresh)
    return s["cache"]


def _attend(s, c):
    n, width = s["table"].shape
    h, d, page, per = c["h_k"], c["d"], c["page"], c["h_q"] // c["h_k"]
    seq, off, new = _where(s, c["tokens"])
    at = s["table"].long().clamp(min=0)
    key = torch.arange(width * page, device=at.device)
    lens = s["lens"].long()

    def values(codes, scales):
        return codes.view(torch.uint8)[at].view(codes.dtype).float() * scales[at][..., None, None]

    k = values(s["k_cache"], s["k_scale"]).permute(0, 2, 1, 3, 4).reshape(n, h, width * page, d)
    v = values(s["v_cache"], s["v_scale"]).permute(0, 2, 1, 4, 3).reshape(n, h, width * page, d)
    v = v * (key < lens[:, None])[:, None, :, None]
    q = torch.zeros((n, s["max_new"], h, per, d), device=at.device)
    q[seq, off] = s["q"].float().unflatten(1, (h, per))
    q = q.permute(0, 2, 1, 3, 4).reshape(n, h, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    pos = (lens - new)[:, None] + torch.arange(s["max_new"], device=at.device)
    sees = (key < lens[:, None])[:, None].expand(n, s["max_new"], -1)
    if c["causal"]:
        sees = sees & (key <= pos[..., None])
    if c["window"]:
        sees = sees & (key > pos[..., None] - c["window"])
    sees = sees[:, None, :, None].expand(n, h, -1, per, -1).reshape(score.shape)
    score = score.masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(top.clamp(min=-1e30)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).reshape(n, h, s["max_new"], per).permute(0, 2, 1, 3).reshape(n, -1, c["h_q"])
    o = o.reshape(n, h, s["max_new"], per, d).permute(0, 2, 1, 3, 4).reshape(n, -1, c["h_q"], d)[seq, off]
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    o = o.to(s["q"].dtype)
    return (o, lse[seq, off]) if c["lse"] else o


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    f = {"norm": _exact_norm, "rope": _exact_rope, "store": _exact_store, "attend": _exact_attend}[c["op"]]
    return f(s, c)


def _exact_norm(s, c):
    d = torch.float64
    x, w = s["x"].to(d).requires_grad_(c["backward"]), s["weight"].to(d).requires_grad_(c["backward"])
    z = None if s["gate"] is None else s["gate"].to(d).requires_grad_(c["backward"])
    h = x if s["residual"] is None or c["order"] == "post" else x * c["scale"] + s["residual"].to(d)
    size = torch.linalg.vector_norm(h, dim=-1, keepdim=True) / math.sqrt(c["width"])
    y = h / torch.hypot(size, torch.full_like(size, math.sqrt(EPS))) * w
    if z is not None:
        y = y * {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[c["gate"]](z)
    if not c["backward"]:
        if c["order"] == "post":
            return s["residual"].to(d) + c["scale"] * y
        return y if s["residual"] is None else (y, h)
    if c["order"] == "post":
        y = y * c["scale"]
    loss = (y * s["dy"].to(d)).sum()
    if s["d_sum"] is not None:
        loss = loss + (h * s["d_sum"].to(d)).sum()
    loss.backward()
    both = (c["scale"] * x.grad, x.grad) if s["d_sum"] is not None else (x.grad, None)
    return (*both, w.grad, None if z is None else z.grad)


def _exact_rope(s, c):
    angle = torch.outer(s["positions"].double(), s["inv_freq"]) * (-1 if c["backward"] else 1)
    spin = torch.polar(torch.full_like(angle, c["mscale"]), angle)[:, None]
    got = []
    for x in (s["q"].double(), s["k"].double()):
        part = x[..., :c["rot"]]
        pairs = part.unflatten(-1, (2, -1)).transpose(-1, -2) if c["layout"] == "half" else part.unflatten(-1, (-1, 2))
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * spin)
        part = (pairs.transpose(-1, -2) if c["layout"] == "half" else pairs).flatten(-2)
        got.append(torch.cat((part, x[..., c["rot"]:]), -1))
    return tuple(got)


def _exact_store(s, c):
    """Codes before their rounding to 8 bits, and the scales."""
    out = [s["k_cache"].double(), s["v_cache"].double(), s["k_scale"].double(), s["v_scale"].double()]
    begin = 0
    table = s["table"].tolist()
    for n, (old, new) in enumerate(zip(old_lengths(c), new_lengths(c))):
        for j in range(old // c["page"], -(-(old + new) // c["page"]) if new else 0):
            lo, hi = max(old, j * c["page"]), min(old + new, (j + 1) * c["page"])
            p, a, b = table[n][j], lo - j * c["page"], hi - j * c["page"]
            rows = slice(begin + lo - old, begin + hi - old)
            for x, codes, scales in ((s["k"][rows].double(), out[0][p], out[2][p]), (s["v"][rows].double(), out[1][p].transpose(1, 2), out[3][p])):
                least = torch.exp2(torch.ceil(torch.log2(x.abs().amax((0, 2)) / FP8_MAX)).clamp(min=-126))
                scale = torch.maximum(least, scales) if a else least
                codes[:, :a] *= (scales / scale)[:, None, None]
                codes[:, a:b] = x.transpose(0, 1) / scale[:, None, None]
                scales.copy_(scale)
        begin += new
    return tuple(out)


def _exact_attend(s, c):
    per, page, d = c["h_q"] // c["h_k"], c["page"], torch.float64
    o = torch.zeros(s["q"].shape, dtype=d, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=d, device="cuda")
    begin = 0
    for n, (new, ctx) in enumerate(zip(new_lengths(c), context_lengths(c))):
        if new:
            at = s["table"][n, :-(-ctx // page)].long()
            k, v = ((x.view(torch.uint8)[at].view(x.dtype).to(d) * y[at].to(d)[..., None, None]) for x, y in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            pos = torch.arange(ctx - new, ctx, device="cuda")[:, None]
            key = torch.arange(ctx, device="cuda")[None]
            hide = (key > pos) if c["causal"] else torch.zeros_like(key > pos)
            hide = hide | (key <= pos - c["window"]) if c["window"] else hide
            for h in range(c["h_q"]):
                kh = k[:, h // per].reshape(-1, c["d"])[:ctx]
                vh = v[:, h // per].transpose(1, 2).reshape(-1, c["d"])[:ctx]
                score = (s["q"][begin:begin + new, h].to(d) @ kh.T * s["scale"]).masked_fill(hide, -math.inf)
                lse[begin:begin + new, h] = torch.logsumexp(score, -1)
                o[begin:begin + new, h] = torch.nan_to_num(torch.softmax(score, -1)) @ vh
        begin += new
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].to(d))
    return (o, lse) if c["lse"] else o
