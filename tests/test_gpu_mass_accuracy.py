"""How far accumulated attention weights may be off: bounds from the two fp16
parts of q', also where the low part is subnormal."""
import math

import numpy as np
import pytest

from oracle import vqkv_oracle as vo
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


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("M", [1, 12])          # few columns, many
@pytest.mark.parametrize("shift", [0, 5, 9])    # q' smaller and K' larger by 2^shift: the same scores
def test_weights_within_the_bound_of_two_fp16_parts(mode, M, shift):
    """Score t is off, in the log2 domain, by at most sum_c max(2^-22 |q'_c|, 2^-25) |K'_tc|, and by the
    roundings of fp32 sums: q' has 10 of 2^-24 in its transform and scaling, the product of 128 terms up to 40
    steps of 2^-23 (tensor cores add groups of terms at the group's exponent), together under 2^-17 of
    sum |q' K'|.  A normalised weight moves by a factor within 2^(+-2 e) of a score error e (its own and the
    sum's); exp2, the sum, its reciprocal and the sum over columns add under 2^-17."""
    B, Hq, Hkv, cap, L = 1, 4, 1, 700, 700
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=40 + mode)
    kcb = (kcb.astype(np.float32) * 2.0 ** shift).astype(np.float16)
    scale = 2.0 ** -shift / math.sqrt(128)
    before = np.zeros((B, Hkv, cap), dtype=np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [L], cap, before, scale=scale)
    assert err == 0
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, [L], causal(M), scale=scale)
    qt = np.abs(vo.transform_query(q[0].reshape(-1, 128).astype(np.float64), s[0])) * scale * math.log2(math.e)
    kt = np.abs(vo.dequantize(kc[0][0][:L], kcb[0]).astype(np.float64))
    parts = np.maximum(2.0 ** -22 * qt, 2.0 ** -25) @ kt.T                   # [columns][L]
    e = (parts + 2.0 ** -17 * (qt @ kt.T)).max()
    bound = 2.0 ** (2 * e) - 1 + 2.0 ** -17
    assert (np.abs(mass[0, 0] - w[0][0]) <= bound * w[0][0]).all()
    R.check_output(o, ref, tol)
