"""CPU checks of the entry points around the mixer: argument structs match the
header, and bad arguments are refused before any launch."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import linear_attention_token_conv1d_amd as gdn
from linear_attention_token_conv1d_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"gdn_rms_norm_args": block.NormArgs, "gdn_rms_norm_backward_args": block.NormBwdArgs, "gdn_rope_args": block.RopeArgs,
           "gdn_cache_store_args": block.CacheStoreArgs, "gdn_cache_attention_args": block.CacheAttentionArgs}


def test_structs_match_the_header():
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void) {' + "\n".join(lines) + "return 0; }"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        key, value = line.split()
        name, _, field = key.partition(".")
        cls = STRUCTS[name]
        assert int(value) == (getattr(cls, field).offset if field else ctypes.sizeof(cls)), key


def _call(entry, cls, base, kw):
    base = dict(base, struct_size=ctypes.sizeof(cls))
    base.update(kw)
    a = cls(**base)
    st = getattr(gdn.lib(), entry)(a, None)
    return st, gdn.lib().gdn_last_error().decode()


NORM = dict(dtype=1, weight_dtype=1, heads=2, width=64, eps=1e-6, scale=1.0, tokens=4, x=0x10000, weight=0x20000, y=0x30000,
            x_stride=128, gate_stride=128, residual_stride=128, y_stride=128, sum_stride=128)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), 1), (dict(dtype=2), 1), (dict(weight_dtype=5), 1), (dict(order=2), 1), (dict(gate=0x40000), 1),
    (dict(heads=0), 1), (dict(tokens=-1), 1), (dict(tokens=1 << 31), 1), (dict(width=0), 1), (dict(width=16385), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=0), 1), (dict(y=0), 1), (dict(sum=0x40000), 1),
    (dict(residual=0x40000), 1), (dict(scale=2.0), 1), (dict(x_stride=127), 1), (dict(x=0x10001), 3), (dict(weight=0x20001), 3),
    (dict(y=0x10080), 1), (dict(y=0x10000, y_stride=256), 1), (dict(y=0x20000), 1),
    (dict(residual=0x40000, sum=0x30000), 1), (dict(residual=0x40000, sum=0x40002), 1),
])
def test_norm_refusals(kw, code):
    st, msg = _call("gdn_rms_norm", block.NormArgs, NORM, kw)
    assert st == code and msg.startswith("gdn_rms_norm"), msg


NORM_BWD = dict(dtype=1, weight_dtype=1, heads=2, width=64, eps=1e-6, scale=1.0, tokens=4, x=0x10000, weight=0x20000,
                dy=0x30000, dx=0x40000, dweight=0x50000, x_stride=128, gate_stride=128, dy_stride=128, d_sum_stride=128,
                dx_stride=128, d_residual_stride=128, dgate_stride=128, workspace=0x1000000, workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), 1), (dict(dy=0), 1), (dict(gate=0x60000, activation=1), 1), (dict(dgate=0x60000), 1),
    (dict(order=1, d_sum=0x60000), 1), (dict(order=1, d_residual=0x60000), 1), (dict(weight=0), 1), (dict(workspace=0), 4),
    (dict(workspace_bytes=100), 4), (dict(workspace=0x1000001), 3), (dict(dweight=0x50002), 3), (dict(dx=0x10002), 1),
    (dict(d_residual=0x40000), 1), (dict(dweight=0x40000), 1), (dict(workspace=0x10000), 1), (dict(dweight=0x20000), 1),
    (dict(dy_stride=5), 1),
])
def test_norm_backward_refusals(kw, code):
    st, msg = _call("gdn_rms_norm_backward", block.NormBwdArgs, NORM_BWD, kw)
    assert st == code and msg.startswith("gdn_rms_norm_backward"), msg


def test_norm_backward_workspace():
    a = block.NormBwdArgs(**dict(NORM_BWD, struct_size=ctypes.sizeof(block.NormBwdArgs)))
    assert gdn.lib().gdn_rms_norm_backward_workspace_size(a) >= 4 * 64
    a.width = 0
    assert gdn.lib().gdn_rms_norm_backward_workspace_size(a) == 0


def test_wrappers_need_gpu_tensors():
    import torch

    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(gdn.GdnError, match="GPU"):
        gdn.rms_norm(x)
    with pytest.raises(gdn.GdnError, match="GPU"):
        gdn.rms_norm_backward(x, x)


ROPE = dict(dtype=1, position_bits=64, h_q=2, h_k=1, d=64, rot=32, mscale=1.0, tokens=4, q=0x10000, k=0x20000, positions=0x30000,
            inv_freq=0x40000, q_out=0x50000, k_out=0x60000, q_stride=128, k_stride=64, q_out_stride=128, k_out_stride=64)


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), 1), (dict(dtype=3), 1), (dict(layout=2), 1), (dict(inverse=2), 1), (dict(position_bits=16), 1), (dict(h_q=0), 1),
    (dict(h_k=-1), 1), (dict(d=1), 1), (dict(rot=0), 1), (dict(rot=33), 1), (dict(rot=66), 1), (dict(mscale=float("nan")), 1),
    (dict(tokens=-1), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(k_out=0), 1), (dict(h_k=0), 1), (dict(positions=0x30004), 3),
    (dict(inv_freq=0x40004), 3), (dict(q_stride=127), 1), (dict(q=0x10001), 3), (dict(q_out=0x10080), 1), (dict(q_out=0x20000), 1),
    (dict(k_out=0x50000), 1), (dict(q_out=0x30000), 1), (dict(q_out=0x10000, q_out_stride=256), 1),
])
def test_rope_refusals(kw, code):
    st, msg = _call("gdn_rope", block.RopeArgs, ROPE, kw)
    assert st == code and msg.startswith("gdn_rope"), msg


POOL = dict(io_dtype=1, n_seqs=2, h_kv=2, d=64, page_size=16, pages=8, max_pages=4, tokens=4, k_cache=0x1000000, v_cache=0x2000000,
            k_scale=0x3000000, v_scale=0x4000000, page_table=0x50000, lens=0x60000)
STORE = dict(POOL, k=0x10000, v=0x20000, k_stride=128, v_stride=128)
ATTEND = dict(POOL, h_q=4, causal=1, scale=0.125, q=0x10000, o=0x20000, q_stride=256, gate_stride=256, o_stride=256)
POOL_BAD = [
    (dict(struct_size=8), 1), (dict(io_dtype=2), 1), (dict(n_seqs=0), 1), (dict(tokens=-2), 1), (dict(tokens=5), 1), (dict(h_kv=0), 1),
    (dict(h_kv=65536), 1), (dict(d=96), 2), (dict(page_size=48), 2), (dict(page_size=8), 2), (dict(page_size=512), 2), (dict(pages=0), 1),
    (dict(max_pages=0), 1), (dict(k_cache=0), 1), (dict(v_scale=0), 1), (dict(page_table=0), 1), (dict(lens=0), 1),
    (dict(v_cache=0x2000008), 3), (dict(k_scale=0x3000002), 3), (dict(cu_seqlens=0x70001), 3), (dict(tokens=1 << 31), 1),
]


@pytest.mark.parametrize("kw,code", POOL_BAD + [
    (dict(k=0), 1), (dict(k_stride=127), 1), (dict(v_stride=132), 3), (dict(v=0x20008), 3), (dict(v_cache=0x1000100), 1),
    (dict(k=0x1000000), 1), (dict(k_scale=0x4000000), 1), (dict(lens=0x1000000), 1),
])
def test_cache_store_refusals(kw, code):
    st, msg = _call("gdn_cache_store", block.CacheStoreArgs, STORE, kw)
    assert st == code and msg.startswith("gdn_cache_store"), msg


@pytest.mark.parametrize("kw,code", POOL_BAD + [
    (dict(h_q=3), 1), (dict(h_q=0), 1), (dict(causal=2), 1), (dict(window=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("inf")), 1), (dict(q=0), 1), (dict(o=0), 1), (dict(q_stride=255), 1), (dict(o_stride=260), 3), (dict(gate=0x30008), 3),
    (dict(o=0x10010), 1), (dict(lse=0x80002), 3), (dict(lse=0x20000), 1), (dict(gate=0x20000), 1), (dict(o=0x1000000), 1),
    (dict(max_pages=4096), 4), (dict(max_pages=4096, workspace=0x7000001, workspace_bytes=1 << 30), 3),
    (dict(max_pages=4096, workspace=0x1000000, workspace_bytes=1 << 30), 1),
])
def test_cache_attention_refusals(kw, code):
    st, msg = _call("gdn_cache_attention", block.CacheAttentionArgs, ATTEND, kw)
    assert st == code and msg.startswith("gdn_cache_attention"), msg


def test_cache_attention_workspace():
    size = gdn.cache_attention_workspace_size
    assert size(1, 1, 1, 24, 4, 256) == 0  # one piece: nothing to join
    assert size(64, 64, 512, 24, 4, 256) > 0
    assert size(0, 1, 512, 24, 4, 256) == 0
    assert size(1, 1, 512, 23, 4, 256) == 0  # invalid


def test_rope_frequencies():
    import math

    import torch

    f, m = gdn.rope_frequencies(64, 1e4)
    assert f.dtype == torch.float64 and m == 1.0 and f[0] == 1.0 and math.isclose(f[31].item(), 1e4 ** (-62 / 64))
    g, _ = gdn.rope_frequencies(64, 1e4, "linear", 4.0)
    assert torch.allclose(g, f / 4)
    g, _ = gdn.rope_frequencies(64, 1e4, "ntk", 4.0)
    assert g[0] == 1.0 and math.isclose(g[31].item(), f[31].item() / 4)
    g, m = gdn.rope_frequencies(64, 1e4, "by_parts", 4.0, original=4096)
    assert g[0] == f[0] and math.isclose(g[31].item(), f[31].item() / 4) and math.isclose(m, 0.1 * math.log(4) + 1)
    assert ((g <= f) & (g >= f / 4)).all()
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="other"), dict(rot=8, scaling="by_parts"), dict(rot=8, factor=0.5)):
        with pytest.raises(gdn.GdnError):
            gdn.rope_frequencies(**bad)
