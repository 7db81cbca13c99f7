"""Rows and lengths that leave nothing to see: NaN and infinities there reach no result."""
import numpy as np
import pytest

from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_mass import causal, gpu_mass
from tests.test_gpu_tree import case, gpu_tree, tree_masks, visible_of
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("M", [3, 13, 16])           # few columns, many
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_weights_of_queries_before_position_zero(mode, M, value):
    """A sequence shorter than the window: its first queries see nothing, whatever their rows hold."""
    lens, cap = [2, 500, 0, 1], 512
    r, q, kc, vc, s, kcb, vcb = case(mode, 4, 4, 1, M, cap, seed=mode)
    clean = q.copy()
    for b, L in enumerate(lens):
        q[b, :max(M - L, 0)] = value
    before = r.random((4, 1, cap), dtype=np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, lens, cap, before)
    ref, w, tol = R.attend(clean, kc, vc, kcb, vcb, s, lens, causal(M))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, lens, R.attend.score_size)
    assert err == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("Hq,M", [(4, 12), (8, 30)])     # one and two query tiles
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_drafts_that_see_nothing(mode, Hq, M, value):
    """No prefix and an empty mask: a zero row; the other drafts as if the row held numbers."""
    lens, cap = [M, 3], 64
    r, q, kc, vc, s, kcb, vcb = case(mode, 2, Hq, 1, M, cap, seed=mode)
    masks = tree_masks(r, 2, M, "tree")
    masks[0, [1, M // 2]] = 0
    masks[1, :M - 3] = 0                                  # their tokens lie before position 0 anyway
    clean = q.copy()
    q[0, [1, M // 2]] = value
    q[1, :M - 3] = value
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, lens, cap)
    ref, _, tol = R.attend(clean, kc, vc, kcb, vcb, s, lens, visible_of(masks, M))
    R.check_output(o, ref, tol)
    assert err == 0 and np.all(o[0, [1, M // 2]] == 0) and np.all(o[1, :M - 3] == 0)


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_max_seq_len_of_zero(mode):
    """Every length clamped to nothing: zero rows, untouched weights, nothing kept."""
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(mode, 2, 4, 1, 5, 64, seed=mode)
    masks = tree_masks(r, 2, 5, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, [0, 0], 64, max_seq_len=0)
    assert np.all(o == 0) and err == 0
    before = r.random((2, 1, 64), dtype=np.float32)
    for M in (1, 5):
        o, mass, err = gpu_mass(mode, q[:, :M].copy(), kc, vc, s, kcb, vcb, [0, 9], 64, before, max_seq_len=0)
        assert np.all(o == 0) and np.array_equal(mass, before) and err == _lib.VQKV_DEVERR_SEQ_LEN
    keep, kl = t.full((2, 1, 8), -7, dtype=t.int32, device="cuda"), t.full((2,), -7, dtype=t.int32, device="cuda")
    _lib.vqkv_evict_select(H.dev(before), H.dev(np.array([0, 9], dtype=np.int32)), keep, kl, max_seq_len=0)
    assert kl.tolist() == [0, 0] and (keep == -7).all()
