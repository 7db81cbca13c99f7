"""Argument checks of the tile kernels' timeout hooks; no GPU needed."""
import ctypes

import pytest

from tests.test_tree_mass_host import _mass, _tree
from vector_quantized_bit_gb300 import _build, _lib


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.lib()


@pytest.mark.parametrize("stage,polls", [(-1, 64), (2, 64), (0, 0), (1, 4097)])
def test_hook_limits(lib, stage, polls):
    assert lib.vqkv_test_decode_tree_timeout(ctypes.byref(_tree()), stage, polls, None) == 1
    assert lib.vqkv_test_decode_mass_timeout(ctypes.byref(_mass(n_queries=10)), 0, stage, polls, None) == 1
    assert lib.vqkv_test_decode_mass_timeout(ctypes.byref(_mass(n_queries=10)), 1, stage, polls, None) == 1


def test_hooks_check_their_arguments(lib):
    assert lib.vqkv_test_decode_tree_timeout(None, 0, 64, None) == 1
    assert lib.vqkv_test_decode_mass_timeout(None, 0, 0, 64, None) == 1
    assert lib.vqkv_test_decode_tree_timeout(ctypes.byref(_tree(n_queries=65)), 0, 64, None) == 2
    assert lib.vqkv_test_decode_mass_timeout(ctypes.byref(_mass(n_queries=17)), 0, 0, 64, None) == 2
