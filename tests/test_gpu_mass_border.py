"""16 columns at 1.25 bit on both sides of the border between the two ways to
compute attention weights."""
import numpy as np
import pytest

from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_mass import causal, gpu_mass
from tests.test_gpu_tree import case
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("L", [24575, 24577])     # 8 KV heads: 196,600 and 196,616 (token, KV head) pairs
def test_weights_beside_the_border(L):
    r, q, kc, vc, s, kcb, vcb = case(4, 1, 32, 8, 4, L, seed=5)
    before = np.zeros((1, 8, L), dtype=np.float32)
    o, mass, err = gpu_mass(4, q, kc, vc, s, kcb, vcb, [L], L, before)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, [L], causal(4))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, [L], R.attend.score_size)
    assert err == 0
