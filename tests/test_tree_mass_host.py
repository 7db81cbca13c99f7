"""Argument checks of the draft-tree and attention-weight calls that need no GPU."""
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


def _dec(**kw):
    a = _lib.DecodeArgs(mode=0, B=1, Hq=4, Hkv=1, head_dim=128, cap_len=64, max_seq_len=64,
                        q=0x1000, k_codes=0x2000, v_codes=0x3000, seq_lens=0x4000, k_codebook=0x5000,
                        v_codebook=0x6000, s=0x7000, softmax_scale=0.0, num_splits=0, workspace=0x8000,
                        workspace_bytes=1 << 20, out=0x9000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _tree(n_queries=8, tree_mask=0xa000, **kw):
    return _lib.DecodeTreeArgs(decode=_dec(**kw), n_queries=n_queries, tree_mask=tree_mask)


@pytest.mark.parametrize("kw,status", [
    (dict(n_queries=0), 1), (dict(n_queries=65), 2), (dict(tree_mask=None), 1), (dict(tree_mask=0xa004), 1),
    (dict(mode=5), 2), (dict(head_dim=64), 2), (dict(Hq=9), 2), (dict(Hq=6, Hkv=4), 1), (dict(max_seq_len=65), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(k_codes=0x2008), 1), (dict(softmax_scale=float("inf")), 1),
    (dict(num_splits=-1), 1), (dict(B=128, cap_len=2**30, max_seq_len=2**30), 2), (dict(Hkv=65536, Hq=65536), 2), (dict(cap_len=2**30 + 1), 2),
])
def test_tree_validation(lib, kw, status):
    assert lib.vqkv_decode_attn_tree(ctypes.byref(_tree(**kw)), None, None) == status
    if not set(kw) & {"tree_mask", "q", "out", "k_codes", "softmax_scale"}:
        assert lib.vqkv_decode_tree_workspace_bytes(ctypes.byref(_tree(**kw))) == 0


def test_tree_empty_and_null(lib):
    assert lib.vqkv_decode_attn_tree(ctypes.byref(_tree(B=0, q=None, tree_mask=None)), None, None) == 0
    assert lib.vqkv_decode_attn_tree(None, None, None) == 1
    assert lib.vqkv_decode_tree_workspace_bytes(None) == 0


def _mass(n_queries=2, mass=0xa000, **kw):
    return _lib.DecodeMassArgs(decode=_dec(**kw), n_queries=n_queries, mass=mass)


@pytest.mark.parametrize("kw,status", [
    (dict(n_queries=0), 1), (dict(n_queries=17), 2), (dict(n_queries=2**31 - 1), 2), (dict(mass=None), 1),
    (dict(mass=0xa002), 1), (dict(mode=7), 2), (dict(head_dim=64), 2), (dict(max_seq_len=65), 1), (dict(q=None), 1),
    (dict(v_codes=0x3008), 1), (dict(B=65536), 2), (dict(cap_len=2**30 + 1), 2),
    (dict(n_queries=16, B=128, cap_len=2**30, max_seq_len=2**30), 2),
])
def test_mass_validation(lib, kw, status):
    assert lib.vqkv_decode_attn_mass(ctypes.byref(_mass(**kw)), None, None) == status
    if not set(kw) & {"mass", "q", "v_codes"}:
        assert lib.vqkv_decode_mass_workspace_bytes(ctypes.byref(_mass(**kw))) == 0


def test_mass_empty_and_null(lib):
    assert lib.vqkv_decode_attn_mass(ctypes.byref(_mass(B=0, q=None, mass=None)), None, None) == 0
    assert lib.vqkv_decode_attn_mass(None, None, None) == 1
    assert lib.vqkv_decode_mass_workspace_bytes(None) == 0


@pytest.mark.parametrize("kw", [dict(block_tokens=100), dict(max_blocks=0), dict(num_blocks=0), dict(max_blocks=1),
                                dict(block_table=None), dict(block_table=0x9002)])
def test_paging_validation(lib, kw):
    pg = _lib.Paging(block_table=0x9000, max_blocks=2, block_tokens=64, num_blocks=4)
    for k, v in kw.items():
        setattr(pg, k, v)
    assert lib.vqkv_decode_attn_tree(ctypes.byref(_tree(cap_len=128, max_seq_len=128)), ctypes.byref(pg), None) == 1
    assert lib.vqkv_decode_attn_mass(ctypes.byref(_mass(cap_len=128, max_seq_len=128)), ctypes.byref(pg), None) == 1


def test_struct_layout_matches_header(tmp_path):
    fields = {"vqkv_decode_tree_args": _lib.DecodeTreeArgs, "vqkv_decode_mass_args": _lib.DecodeMassArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "vqkv.h"', "int main(void){"]
    for cname, cls in fields.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));')
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
