"""Argument checks of the cache-editing calls that need no GPU: the C entries'
statuses before anything is launched, the mirrors of their argument structs."""
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


def _sel(**kw):
    a = _lib.EvictSelectArgs(B=2, Hkv=4, cap_len=128, max_seq_len=128, n_keep=32, n_sink=4, n_recent=8, mass=0x1000,
                             seq_lens=0x2000, keep=0x3000, keep_lens=0x4000, error_flags=0x5000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _cmp(**kw):
    a = _lib.CacheCompactArgs(mode=0, B=2, Hkv=4, cap_len=128, n_src=16, src_heads=4, k_codes=0x1000, v_codes=0x2000,
                              seq_lens=0x3000, src=0x4000, counts=0x5000, start=0x6000, mass=0x7000, error_flags=0x8000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(cap_len=0, max_seq_len=0), 1), (dict(max_seq_len=129), 1),
    (dict(max_seq_len=-1), 1), (dict(n_keep=0, n_sink=0, n_recent=0), 1), (dict(n_sink=-1), 1), (dict(n_recent=-1), 1),
    (dict(n_sink=20, n_recent=13), 1), (dict(n_sink=2**31 - 1, n_recent=2**31 - 1), 1), (dict(mass=None), 1),
    (dict(seq_lens=None), 1), (dict(keep=None), 1), (dict(keep_lens=None), 1), (dict(mass=0x1002), 1),
    (dict(keep=0x3001), 1), (dict(error_flags=0x5002), 1), (dict(B=65536), 2), (dict(Hkv=65536), 2),
    (dict(cap_len=2**30 + 1), 2),
])
def test_select_validation(lib, kw, status):
    assert lib.vqkv_evict_select(ctypes.byref(_sel(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(mode=5), 2), (dict(mode=-1), 2), (dict(B=-1), 1), (dict(Hkv=0, src_heads=1), 1), (dict(cap_len=0), 1),
    (dict(n_src=-1), 1), (dict(src_heads=2), 1), (dict(src_heads=0), 1), (dict(k_codes=None), 1),
    (dict(v_codes=None), 1), (dict(seq_lens=None), 1), (dict(src=None), 1), (dict(counts=None), 1),
    (dict(k_codes=0x1008), 1), (dict(v_codes=0x2004), 1), (dict(src=0x4002), 1), (dict(start=0x6001), 1),
    (dict(mass=0x7002), 1), (dict(B=65536), 2), (dict(Hkv=21846, src_heads=1), 2), (dict(cap_len=2**30 + 1), 2),
])
def test_compact_validation(lib, kw, status):
    assert lib.vqkv_cache_compact(ctypes.byref(_cmp(**kw)), None, None) == status


def test_empty_calls_are_no_ops(lib):
    assert lib.vqkv_evict_select(ctypes.byref(_sel(B=0, mass=None, keep=None)), None) == 0
    assert lib.vqkv_cache_compact(ctypes.byref(_cmp(B=0, k_codes=None, src=None)), None, None) == 0
    assert lib.vqkv_cache_compact(ctypes.byref(_cmp(n_src=0, src=None, mass=None)), None, None) == 0
    assert lib.vqkv_evict_select(None, None) == 1
    assert lib.vqkv_cache_compact(None, None, None) == 1


@pytest.mark.parametrize("kw", [dict(block_tokens=100), dict(block_tokens=32), dict(max_blocks=0), dict(num_blocks=0),
                                dict(max_blocks=1), dict(block_table=None), dict(block_table=0x9002)])
def test_compact_paging_validation(lib, kw):
    pg = _lib.Paging(block_table=0x9000, max_blocks=2, block_tokens=64, num_blocks=4)
    for k, v in kw.items():
        setattr(pg, k, v)
    assert lib.vqkv_cache_compact(ctypes.byref(_cmp()), ctypes.byref(pg), None) == 1


def test_struct_layout_matches_header(tmp_path):
    fields = {"vqkv_evict_select_args": _lib.EvictSelectArgs, "vqkv_cache_compact_args": _lib.CacheCompactArgs}
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
