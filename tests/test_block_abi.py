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
STRUCTS = {"gdn_rms_norm_args": block.NormArgs, "gdn_rms_norm_backward_args": block.NormBwdArgs}


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
