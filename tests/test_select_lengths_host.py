"""vqkv_evict_select refuses to write the kept lengths over the lengths it reads; no GPU needed."""
import ctypes

import pytest

from tests.test_cache_edit_host import _sel
from tests.test_prepare_host import run  # noqa: F401  (fixture: the CUDA runtime's stand-in)
from vector_quantized_bit_gb300 import _build, _lib


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.lib()


@pytest.mark.parametrize("B,seq_lens,keep_lens", [(2, 0x2000, 0x2000), (2, 0x2000, 0x2004), (2, 0x2004, 0x2000),
                                                  (65535, 0x100000, 0x100000 + 4 * 65534)])
def test_overlapping_lengths_are_refused(lib, B, seq_lens, keep_lens):
    assert lib.vqkv_evict_select(ctypes.byref(_sel(B=B, seq_lens=seq_lens, keep_lens=keep_lens)), None) == 1


def test_neighbouring_lengths_are_not(run):
    run("""
a = select()
for a.seq_lens, a.keep_lens in ((0x2000, 0x2008), (0x2008, 0x2000)):
    assert L.vqkv_evict_select(ctypes.byref(a), None) == 0
assert len([x for x in log() if x.startswith("launch")]) == 2
""")
