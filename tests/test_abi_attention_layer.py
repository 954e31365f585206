"""The attention layer's part of the C ABI, without a GPU: its structs lie in memory as the binding
packs them, and bad arguments are refused before any CUDA call."""

import ctypes
import re
import shutil
import subprocess
from pathlib import Path

import pytest

HEADER = Path(__file__).resolve().parent.parent / "include" / "bfp8.h"
STRUCTS = {"bfp8_kv_cache": "_KV_CACHE", "bfp8_kv_attention_args": "_KV_ATTENTION", "bfp8_norm_args": "_NORM"}


def _fields(name):
    """The struct's member names in the header, in order."""
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    body = re.search(r"typedef struct \{([^{}]*)\} " + name + ";", text).group(1)
    return [re.search(r"(\w+)\s*$", f).group(1) for line in body.split(";") for f in line.split(",") if f.strip()]


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
    assert [getattr(cls, f).offset for f in fields] == at and ctypes.sizeof(cls) == size
    assert packed.size == size
    # each packed value is where its member is: one distinct value a member, read back through the struct
    codes = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([PqifN])", packed.format))
    values = [float(i + 1) if c == "f" else i + 1 for i, c in enumerate(codes)]
    got = cls.from_buffer_copy(packed.pack(*values))
    assert [getattr(got, f) for f in fields] == values


def test_refusals_without_a_gpu(bfp8):
    lib, p = bfp8._lib, 256
    INVAL, SCALE_DTYPE, UNSUPPORTED = 1, 8, 13

    def cache(**kw):
        a = dict(k_e4m3=p, v_e4m3=p, k_exp=p, v_exp=p, n_pages=4, page_size=16, n_kv_heads=2, head_dim=128,
                 k_stride_page=4096, k_stride_head=2048, k_stride_token=128, v_stride_page=4096, v_stride_head=2048,
                 v_stride_token=128, exp_stride_page=2, exp_stride_head=1)
        return ctypes.byref(bfp8.bfp8_kv_cache(**(a | kw)))

    def plan(*, B=1, n_free=4, table=p, ld=4, width=4, page=16, T=4, slots=p, counts=p):
        return lib.bfp8_kv_plan(p, p, B, p, n_free, table, ld, width, page, p, p, slots, p, T, counts, None)

    def append(k=p, ldt=256, ldh=128, slots=p, T=4, **kw):
        return lib.bfp8_kv_append(k, ldt, ldh, p, 256, 128, slots, T, cache(**kw), None)

    def attention(cache_kw={}, **kw):
        a = dict(q_bf16=p, q_stride_token=512, q_stride_head=128, out_bf16=p, out_stride_token=512, out_stride_head=128,
                 lse=None, lse_stride_token=4, block_table=p, ld_table=4, max_blocks=4, q_offsets=p, kv_len=p, batch=1,
                 tokens=1, max_q_len=1, n_heads=4, softmax_scale=1.0, window=-1, workspace=p, ws_bytes=1 << 30)
        return lib.bfp8_kv_attention(ctypes.byref(bfp8.bfp8_kv_attention_args(**(a | kw))), cache(**cache_kw), None)

    def norm(T=2, H=256, **kw):
        a = dict(y=p, ldy=256, residual=p, ld_residual=256, w_post=p, w_pre=p, w_dtype=3, residual_scale=1.0, eps=1e-6,
                 residual_out=p, ld_residual_out=256, norm_out=p, ld_norm_out=256, q_e4m3=p, ldq=256, scales=p,
                 s_stride_m=2, s_stride_kb=1)
        return lib.bfp8_residual_norm(ctypes.byref(bfp8.bfp8_norm_args(**(a | kw))), T, H, None)

    cases = [
        (plan(B=-1), INVAL), (plan(T=-1), INVAL), (plan(n_free=-1), INVAL), (plan(ld=3), INVAL), (plan(table=None), INVAL),
        (plan(slots=None), INVAL), (plan(counts=None), INVAL), (plan(page=24), UNSUPPORTED), (plan(B=16385), UNSUPPORTED),
        (append(T=-1), INVAL), (append(T=0), 0), (append(k=None), INVAL), (append(slots=None), INVAL),
        (append(ldt=-8), INVAL), (append(ldt=252), UNSUPPORTED), (append(k=p + 8), UNSUPPORTED),
        (append(page_size=8), UNSUPPORTED), (append(head_dim=64), UNSUPPORTED), (append(n_pages=0), INVAL),
        (append(k_stride_token=64), INVAL), (append(v_stride_head=2056), UNSUPPORTED), (append(v_e4m3=p + 8), UNSUPPORTED),
        (append(exp_stride_head=0), INVAL), (lib.bfp8_kv_append(p, 256, 128, p, 256, 128, p, 4, None, None), INVAL),
        (attention(batch=-1), INVAL), (attention(tokens=-1), INVAL), (attention(max_q_len=-1), INVAL),
        (attention(batch=0), 0), (attention(tokens=0), 0), (attention(max_q_len=0), 0), (attention(n_heads=3), INVAL),
        (attention(n_heads=0), INVAL), (attention(ld_table=3), INVAL), (attention(q_bf16=None), INVAL),
        (attention(block_table=None), INVAL), (attention(out_stride_head=64), INVAL), (attention(q_stride_head=132), UNSUPPORTED),
        (attention(out_bf16=p + 8), UNSUPPORTED), (attention(lse=p, lse_stride_token=3), INVAL),
        (attention(softmax_scale=float("inf")), INVAL), (attention(softmax_scale=float("nan")), INVAL),
        (attention(tokens=1 << 30, max_q_len=1), UNSUPPORTED), (attention({"page_size": 48}), UNSUPPORTED),
        (attention({"k_exp": None}), INVAL), (lib.bfp8_kv_attention(None, cache(), None), INVAL),
        (norm(T=-1), INVAL), (norm(T=0), 0), (norm(H=0), 0), (norm(residual=None), INVAL), (norm(ld_residual=255), INVAL),
        (norm(y=None), INVAL), (norm(ldy=255), INVAL), (norm(gate=p, ld_gate=255), INVAL), (norm(w_pre=None), INVAL),
        (norm(scales=None), INVAL), (norm(ldq=255), INVAL), (norm(s_stride_m=0), INVAL), (norm(s_stride_kb=0), INVAL),
        (norm(eps=-1.0), INVAL), (norm(eps=float("nan")), INVAL), (norm(w_dtype=4), SCALE_DTYPE),
        (norm(residual_out=None, norm_out=None, q_e4m3=None), INVAL),
        (norm(H=16392, ldy=16392, ld_residual=16392, ld_residual_out=16392, ld_norm_out=16392, ldq=16392, s_stride_m=129),
         UNSUPPORTED),
        (lib.bfp8_residual_norm(None, 1, 1, None), INVAL),
    ]
    for i, (got, want) in enumerate(cases):
        assert got == want, (i, got, want)
    for bad in [(0, 1, 1, 4, 2), (1, 0, 1, 4, 2), (1, 1, 0, 4, 2), (1, 1, 1, 0, 1), (1, 1, 1, 4, 0), (1, 1, 1, 4, 3)]:
        assert lib.bfp8_kv_attention_workspace(*bad) == 0
