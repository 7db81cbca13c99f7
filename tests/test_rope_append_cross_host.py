"""Argument checks of the rotary, append and cross-attention calls that need no
GPU: statuses before anything is launched, the mirrors of their argument
structs."""
import ctypes
import os
import subprocess

import pytest

from tests.conftest import ROOT
from vector_quantized_bit_gb300 import _build, _lib


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.lib()


def _with(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def _table(**kw):
    return _with(_lib.RopeTableArgs(n_pos=16, rot_dim=64, scaling=0, original_len=4096, base=1e4, factor=4.0, low_turns=1.0,
                                    high_turns=4.0, amplitude=1.0, table=0x1000), kw)


def _rope(**kw):
    return _with(_lib.RopeArgs(dtype=0, n_tokens=4, n_heads=3, head_dim=128, rot_dim=64, n_pos=16, x_token_stride=384,
                               x_head_stride=128, out_token_stride=384, out_head_stride=128, x=0x10000, positions=0x1000,
                               table=0x2000, out=0x20000, error_flags=0x3000), kw)


def _append(**kw):
    return _with(_lib.AppendArgs(mode=0, dtype=0, B=2, Hkv=2, head_dim=128, n_tokens=4, cap_len=64, rot_dim=64, n_pos=16,
                                 k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128, k=0x10000,
                                 v=0x20000, row_start=0x1000, pos=0x2000, rope_pos=0x3000, rope_table=0x4000, s=0x5000,
                                 k_codebook=0x6000, v_codebook=0x7000, k_codes=0x8000, v_codes=0x9000, near_tie_count=0xa000,
                                 error_flags=0xb000), kw)


def _cross(**kw):
    d = _lib.DecodeArgs(mode=0, B=2, Hq=4, Hkv=2, head_dim=128, cap_len=128, max_seq_len=128, q=0x10000, k_codes=0x1000,
                        v_codes=0x2000, seq_lens=0x3000, k_codebook=0x4000, v_codebook=0x5000, s=0x6000, num_splits=0,
                        workspace=0x100, workspace_bytes=1 << 30, out=0x40000)
    a = _lib.CrossArgs(decode=d, dtype=0, n_rows=5, max_queries=3, q_row_stride=512, row_start=0x7000)
    for k, v in kw.items():
        setattr(a.decode if hasattr(_lib.DecodeArgs, k) else a, k, v)
    return ctypes.byref(a)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=4), 2), (dict(rot_dim=12), 2), (dict(rot_dim=136), 2), (dict(rot_dim=0), 2), (dict(scaling=5), 2),
    (dict(scaling=-1), 2), (dict(n_pos=-1), 1), (dict(base=1.0), 1), (dict(base=NAN), 1), (dict(base=INF), 1),
    (dict(amplitude=NAN), 1), (dict(amplitude=INF), 1), (dict(table=None), 1), (dict(table=0x1008), 1),
    (dict(scaling=1, factor=0.0), 1), (dict(scaling=1, factor=NAN), 1), (dict(scaling=2, factor=-1.0), 1),
    (dict(scaling=2, factor=1e-300), 1), (dict(scaling=3, low_turns=0.0), 1), (dict(scaling=3, low_turns=4.0), 1),
    (dict(scaling=4, high_turns=INF), 1), (dict(scaling=4, original_len=0), 1), (dict(scaling=3, high_turns=NAN), 1),
])
def test_rope_table_validation(lib, kw, status):
    assert lib.vqkv_rope_table(_table(**kw), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(head_dim=64), 2), (dict(rot_dim=20), 2), (dict(n_heads=65536), 2),
    (dict(n_tokens=-1), 1), (dict(n_heads=0), 1), (dict(n_pos=0), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(positions=None), 1), (dict(table=None), 1), (dict(x=0x10004), 1), (dict(dtype=1, x=0x10008), 1),
    (dict(out=0x20002), 1), (dict(positions=0x1002), 1), (dict(table=0x2004), 1), (dict(error_flags=0x3001), 1),
    (dict(x_token_stride=386), 1), (dict(x_head_stride=-128), 1), (dict(out_token_stride=-384), 1),
    (dict(x_token_stride=1 << 41), 1),
    (dict(out_head_stride=0), 1), (dict(out_token_stride=0), 1), (dict(out_head_stride=64), 1),   # rows of out that meet
    (dict(out=0x10000 + 8), 1), (dict(out=0x10000, out_token_stride=512), 1),                     # out across x
    (dict(out=0x10000 + 2 * 3 * 384), 1),
])
def test_rope_validation(lib, kw, status):
    assert lib.vqkv_rope(_rope(**kw), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(mode=5), 2), (dict(mode=-1), 2), (dict(dtype=7), 2), (dict(head_dim=64), 2), (dict(Hkv=32768), 2), (dict(rot_dim=6), 2),
    (dict(n_tokens=2**30 + 1), 2), (dict(cap_len=2**30 + 1), 2), (dict(B=2**30), 2),
    (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(n_tokens=-1), 1), (dict(cap_len=0), 1), (dict(n_pos=0), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(row_start=None), 1), (dict(pos=None), 1), (dict(s=None), 1), (dict(k_codebook=None), 1),
    (dict(v_codebook=None), 1), (dict(k_codes=None), 1), (dict(v_codes=None), 1), (dict(k=0x10004), 1),
    (dict(dtype=1, v=0x20008), 1), (dict(k_token_stride=258), 1), (dict(v_head_stride=-4), 1), (dict(row_start=0x1001), 1),
    (dict(pos=0x2002), 1), (dict(rope_pos=0x3002), 1), (dict(rope_table=0x4004), 1), (dict(s=0x5004), 1),
    (dict(k_codebook=0x6008), 1), (dict(v_codebook=0x7008), 1), (dict(near_tie_count=0xa004), 1), (dict(error_flags=0xb002), 1),
])
def test_append_validation(lib, kw, status):
    assert lib.vqkv_append(_append(**kw), None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(mode=5), 2), (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(head_dim=64), 2), (dict(Hq=18), 2), (dict(Hq=5), 1),
    (dict(n_rows=-1), 1), (dict(max_queries=0), 1), (dict(n_rows=2**27 + 1), 2), (dict(max_queries=2**27 + 1), 2),
    (dict(B=1000, cap_len=2**26, max_seq_len=2**26, max_queries=2**14), 2), (dict(row_start=None), 1), (dict(row_start=0x7002), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=0x10004), 1), (dict(q_row_stride=508), 1), (dict(q_row_stride=514), 1),
    (dict(q_row_stride=1 << 41), 1), (dict(seq_lens=None), 1), (dict(max_seq_len=129), 1), (dict(num_splits=-1), 1),
    (dict(softmax_scale=NAN), 1), (dict(out=0x10000 + 1024), 1), (dict(out=0x10000, q_row_stride=1024), 1),
])
def test_cross_validation(lib, kw, status):
    assert lib.vqkv_cross_attn(_cross(**kw), None, None) == status


def test_empty_calls_are_no_ops(lib):
    assert lib.vqkv_rope_table(_table(n_pos=0, table=None), None) == 0
    assert lib.vqkv_rope(_rope(n_tokens=0, x=None, out=None, positions=None, table=None), None) == 0
    assert lib.vqkv_append(_append(B=0, k=None, row_start=None), None, None) == 0
    assert lib.vqkv_append(_append(n_tokens=0, k=None, v=None, s=None), None, None) == 0
    assert lib.vqkv_cross_attn(_cross(B=0), None, None) == 0
    assert lib.vqkv_cross_attn(_cross(n_rows=0, q=None, out=None), None, None) == 0
    for call, more in ((lib.vqkv_rope_table, ()), (lib.vqkv_rope, ()), (lib.vqkv_append, (None,)), (lib.vqkv_cross_attn, (None,))):
        assert call(None, *more, None) == 1
    assert lib.vqkv_cross_attn_workspace_bytes(None) == 0
    assert lib.vqkv_cross_attn_workspace_bytes(_cross(Hq=5)) == 0


@pytest.mark.parametrize("kw", [dict(block_tokens=100), dict(block_tokens=32), dict(max_blocks=0), dict(num_blocks=0),
                                dict(max_blocks=1), dict(block_table=None), dict(block_table=0x9002)])
def test_paging_validation(lib, kw):
    pg = _lib.Paging(block_table=0x9000, max_blocks=2, block_tokens=64, num_blocks=4)
    for k, v in kw.items():
        setattr(pg, k, v)
    assert lib.vqkv_append(_append(cap_len=128), ctypes.byref(pg), None) == 1
    assert lib.vqkv_cross_attn(_cross(), ctypes.byref(pg), None) == 1


def test_struct_layout_matches_header(tmp_path):
    fields = {"vqkv_rope_table_args": _lib.RopeTableArgs, "vqkv_rope_args": _lib.RopeArgs, "vqkv_append_args": _lib.AppendArgs,
              "vqkv_cross_args": _lib.CrossArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "vqkv.h"', "int main(void){"]
    for cname, cls in fields.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));')
    for name in ("VQKV_DTYPE_F16", "VQKV_DTYPE_F32", "VQKV_DTYPE_BF16", "VQKV_ROPE_NONE", "VQKV_ROPE_LINEAR", "VQKV_ROPE_BASE",
                 "VQKV_ROPE_WAVELENGTH", "VQKV_ROPE_RAMP"):
        lines.append(f'printf("{name} %d\\n", (int){name});')
    lines.append("return 0;}")
    c = tmp_path / "layout.c"
    c.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    out = dict(line.rsplit(" ", 1) for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                              check=True).stdout.split("\n") if line)
    for cname, cls in fields.items():
        assert int(out[cname]) == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(out[f"{cname}.{f}"]) == getattr(cls, f).offset, (cname, f)
    for name in [n for n in out if n.startswith("VQKV_")]:
        assert int(out[name]) == getattr(_lib, name)
