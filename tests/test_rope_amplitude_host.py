"""Amplitudes of the rotary table that fp32 does not hold are refused.  No GPU needed: the
arguments are checked before any device is looked for."""
import numpy as np
import pytest

from tests.test_rope_append_cross_host import _table
from vector_quantized_bit_gb300 import _build, _lib

FMAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.lib()


@pytest.mark.parametrize("amplitude", [1e300, -1e300, 1e39, 2.0 ** 128, -FMAX * (1 + 1e-7), np.nextafter(FMAX, np.inf)])
@pytest.mark.parametrize("n_pos", [0, 16])
def test_beyond_fp32(lib, amplitude, n_pos):
    """inf * 0 would be NaN in the rows of angles that are multiples of a quarter turn, position 0 among them."""
    assert lib.vqkv_rope_table(_table(amplitude=amplitude, n_pos=n_pos), None) == 1


@pytest.mark.parametrize("amplitude", [FMAX, -FMAX, 0.0, 1e-300, -1.0])
def test_within_fp32(lib, amplitude):
    assert lib.vqkv_rope_table(_table(amplitude=amplitude, n_pos=0), None) == 0
