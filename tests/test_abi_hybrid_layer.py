"""The hybrid layers' part of the C ABI, without a GPU: its structs lie in memory as the binding
packs them, and bad arguments are refused before any CUDA call."""

import ctypes
import re
import shutil
import subprocess
from pathlib import Path

import pytest

HEADER = Path(__file__).resolve().parent.parent / "include" / "bfp8.h"
STRUCTS = {"bfp8_causal_conv_args": "_CAUSAL_CONV", "bfp8_delta_rule_args": "_DELTA_RULE",
           "bfp8_gated_norm_args": "_GATED_NORM", "bfp8_rotary_args": "_ROTARY"}
INVAL, SCALE_DTYPE, UNSUPPORTED = 1, 8, 13
P = 256   # a placeholder address


def _fields(name):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    body = re.search(r"typedef struct \{([^{}]*)\} " + name + ";", text).group(1)
    return [re.search(r"(\w+)(\[\d+\])?\s*$", f).group(1) for line in body.split(";") for f in line.split(",") if f.strip()]


@pytest.mark.parametrize("name", STRUCTS)
def test_structs_lie_as_the_header_lays_them_out(bfp8, name, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields, cls, packed = _fields(name), getattr(bfp8, name), getattr(bfp8, STRUCTS[name])
    offsets = "".join(f'printf("%zu ", offsetof({name}, {f}));' for f in fields)
    (tmp_path / "t.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "bfp8.h"\n'
                                  f'int main(void) {{ printf("%zu ", sizeof({name})); {offsets} return 0; }}\n')
    subprocess.run([cc, "-I", str(HEADER.parent), str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    size, *at = map(int, subprocess.run([tmp_path / "t"], capture_output=True, check=True, text=True).stdout.split())
    assert [f for f, _ in cls._fields_] == fields
    assert [getattr(cls, f).offset for f in fields] == at and ctypes.sizeof(cls) == size == packed.size
    codes = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([PqifN])", packed.format))
    values = [float(i + 1) if c == "f" else i + 1 for i, c in enumerate(codes)]
    got = cls.from_buffer_copy(packed.pack(*values))
    flat = []
    for f in fields:
        v = getattr(got, f)
        flat += list(v) if isinstance(v, ctypes.Array) else [v]
    assert flat == values


def _conv(bfp8, **kw):
    a = dict(x_bf16=P, x_stride_token=64, out_bf16=2 * P, out_stride_token=64, weight=P, bias=P, w_dtype=3, width=4, silu=1,
             state_bf16=P, state_stride_slot=192, state_stride_row=64, n_slots=2, slots_in=P, slots_out=P, q_offsets=P, batch=1,
             tokens=4, channels=64)
    return bfp8._lib.bfp8_causal_conv(ctypes.byref(bfp8.bfp8_causal_conv_args(**(a | kw))), None)


def _delta(bfp8, **kw):
    a = dict(q_bf16=P, q_stride_token=512, q_stride_head=128, k_bf16=P, k_stride_token=512, k_stride_head=128, v_bf16=P,
             v_stride_token=512, v_stride_head=128, a_bf16=P, a_stride_token=2, b_bf16=P, b_stride_token=2, a_log=P, dt_bias=P,
             state=P, state_stride_slot=32768, state_stride_head=16384, n_slots=2, slots_in=P, slots_out=P, q_offsets=P,
             out_bf16=P, out_stride_token=256, out_stride_head=128, batch=1, tokens=4, max_q_len=4, qk_heads=1, v_heads=2,
             head_dim=128, scale=1.0, eps=1e-6, workspace=P, ws_bytes=1 << 40)
    return bfp8._lib.bfp8_delta_rule(ctypes.byref(bfp8.bfp8_delta_rule_args(**(a | kw))), None)


def _gated(bfp8, **kw):
    a = dict(x_bf16=P, x_stride_token=256, x_stride_head=128, gate_bf16=P, gate_stride_token=256, gate_stride_head=128, weight=P,
             w_dtype=5, gate_act=0, eps=1e-6, weight_offset=0.0, out_bf16=P, out_stride_token=256, out_stride_head=128, q_e4m3=P,
             ldq=256, scales=P, s_stride_m=2, s_stride_kb=1, tokens=4, heads=2, head_dim=128)
    return bfp8._lib.bfp8_gated_norm(ctypes.byref(bfp8.bfp8_gated_norm_args(**(a | kw))), None)


def _rotary(bfp8, sections=(16, 0, 0, 0), **kw):
    a = dict(q_bf16=P, q_stride_token=256, q_stride_head=128, q_out_bf16=P, q_out_stride_token=256, q_out_stride_head=128,
             k_bf16=P, k_stride_token=128, k_stride_head=128, k_out_bf16=P, k_out_stride_token=128, k_out_stride_head=128,
             positions=P, ld_positions=4, inv_freq=P, q_weight=P, k_weight=P, w_dtype=3, eps=1e-6, weight_offset=0.0, factor=1.0,
             tokens=4, q_heads=2, k_heads=1, head_dim=128, rotary_dim=32, axes=1, interleaved=0, adjacent=0)
    s = bfp8.bfp8_rotary_args(**(a | kw))
    s.sections[:] = sections
    return bfp8._lib.bfp8_rotary(ctypes.byref(s), None)


CASES = [
    (_conv, dict(tokens=-1), INVAL), (_conv, dict(batch=-1), INVAL), (_conv, dict(n_slots=-1), INVAL), (_conv, dict(tokens=0), 0),
    (_conv, dict(batch=0), 0), (_conv, dict(channels=0), 0), (_conv, dict(width=5), UNSUPPORTED), (_conv, dict(width=1), UNSUPPORTED),
    (_conv, dict(w_dtype=4), SCALE_DTYPE), (_conv, dict(x_bf16=None), INVAL), (_conv, dict(out_bf16=None), INVAL),
    (_conv, dict(out_bf16=P), INVAL), (_conv, dict(weight=None), INVAL), (_conv, dict(q_offsets=None), INVAL),
    (_conv, dict(x_stride_token=56), INVAL), (_conv, dict(out_stride_token=56), INVAL), (_conv, dict(state_bf16=None), INVAL),
    (_conv, dict(state_stride_row=56), INVAL), (_conv, dict(state_stride_slot=184), INVAL), (_conv, dict(x_bf16=P + 8), UNSUPPORTED),
    (_conv, dict(weight=P + 4), UNSUPPORTED), (_conv, dict(x_stride_token=68), UNSUPPORTED),
    (_conv, dict(channels=60), UNSUPPORTED), (_conv, dict(batch=70000), UNSUPPORTED),
    (_delta, dict(tokens=-1), INVAL), (_delta, dict(batch=-1), INVAL), (_delta, dict(max_q_len=-1), INVAL),
    (_delta, dict(tokens=0), 0), (_delta, dict(batch=0), 0), (_delta, dict(max_q_len=0), 0), (_delta, dict(qk_heads=0), INVAL),
    (_delta, dict(v_heads=0), INVAL), (_delta, dict(qk_heads=3, v_heads=4), INVAL), (_delta, dict(head_dim=64), UNSUPPORTED),
    (_delta, dict(q_bf16=None), INVAL), (_delta, dict(a_log=None), INVAL), (_delta, dict(out_bf16=None), INVAL),
    (_delta, dict(q_offsets=None), INVAL), (_delta, dict(a_stride_token=1), INVAL), (_delta, dict(v_stride_head=64), INVAL),
    (_delta, dict(k_stride_token=516), UNSUPPORTED), (_delta, dict(v_bf16=P + 2), UNSUPPORTED), (_delta, dict(state=None), INVAL),
    (_delta, dict(state_stride_head=16380), INVAL), (_delta, dict(state_stride_slot=32770), UNSUPPORTED),
    (_delta, dict(eps=-1.0), INVAL), (_delta, dict(eps=float("nan")), INVAL), (_delta, dict(scale=float("inf")), INVAL),
    (_gated, dict(tokens=-1), INVAL), (_gated, dict(heads=-1), INVAL), (_gated, dict(tokens=0), 0), (_gated, dict(heads=0), 0),
    (_gated, dict(head_dim=96), UNSUPPORTED), (_gated, dict(x_bf16=None), INVAL), (_gated, dict(gate_bf16=None), INVAL),
    (_gated, dict(out_bf16=None, q_e4m3=None), INVAL), (_gated, dict(scales=None), INVAL), (_gated, dict(ldq=255), INVAL),
    (_gated, dict(s_stride_m=0), INVAL), (_gated, dict(s_stride_kb=0), INVAL), (_gated, dict(gate_act=2), INVAL),
    (_gated, dict(eps=-1.0), INVAL), (_gated, dict(w_dtype=4), SCALE_DTYPE), (_gated, dict(x_stride_head=64), INVAL),
    (_gated, dict(x_stride_token=260), UNSUPPORTED), (_gated, dict(gate_bf16=P + 8), UNSUPPORTED), (_gated, dict(ldq=260), UNSUPPORTED),
    (_rotary, dict(tokens=-1), INVAL), (_rotary, dict(q_heads=-1), INVAL), (_rotary, dict(tokens=0), 0),
    (_rotary, dict(q_heads=0, k_heads=0), 0), (_rotary, dict(head_dim=80), UNSUPPORTED), (_rotary, dict(rotary_dim=24), UNSUPPORTED),
    (_rotary, dict(rotary_dim=144), INVAL), (_rotary, dict(axes=0), INVAL), (_rotary, dict(axes=5), INVAL),
    (_rotary, dict(sections=(15, 0, 0, 0)), INVAL), (_rotary, dict(axes=2, sections=(17, -1, 0, 0)), INVAL),
    (_rotary, dict(axes=2, sections=(8, 8, 0, 0), ld_positions=3), INVAL), (_rotary, dict(positions=None), INVAL),
    (_rotary, dict(inv_freq=None), INVAL), (_rotary, dict(q_bf16=None), INVAL), (_rotary, dict(k_out_bf16=None), INVAL),
    (_rotary, dict(eps=float("nan")), INVAL), (_rotary, dict(factor=float("inf")), INVAL), (_rotary, dict(w_dtype=4), SCALE_DTYPE),
    (_rotary, dict(q_stride_head=64), INVAL), (_rotary, dict(k_stride_token=132), UNSUPPORTED), (_rotary, dict(q_out_bf16=P + 8), UNSUPPORTED),
]


@pytest.mark.parametrize("call,change,want", CASES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_refusals_without_a_gpu(bfp8, call, change, want):
    assert call(bfp8, **change) == want


def test_null_structs_and_workspaces(bfp8):
    lib = bfp8._lib
    for f in (lib.bfp8_causal_conv, lib.bfp8_delta_rule, lib.bfp8_gated_norm, lib.bfp8_rotary):
        assert f(None, None) == INVAL
    for bad in [(0, 1, 1, 1, 1), (1, 0, 1, 1, 1), (1, 1, 0, 1, 1), (1, 1, 1, 0, 1), (1, 1, 1, 1, 0), (1, 1, 1, 2, 3)]:
        assert lib.bfp8_delta_rule_workspace(*bad) == 0
