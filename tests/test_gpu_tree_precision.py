"""Short draft trees take their scores from two fp16 parts of q': large scores
keep the precision of fp32 arithmetic with fp16 weights and output."""
import math

import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_tree import case, gpu_tree, tree_masks, visible_of
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("B,Hq,Hkv,M,lens,page", [
    (1, 32, 8, 8, [519], 0), (1, 8, 2, 16, [2000], 0), (1, 4, 4, 64, [300], 0), (3, 4, 1, 5, [64, 0, 130], 64),
    (2, 10, 2, 11, [200, 7], 128), (1, 1, 1, 1, [1], 0),
])
def test_short_trees_keep_fp32_scores(mode, B, Hq, Hkv, M, lens, page):
    """q times 12: scores near 40.  A score is off by e = ln 2 (sum max(2^-22 |q'|, 2^-25) |K'| + 2^-17 sum |q' K'|)
    (two fp16 parts; fp32 transform and sums), a normalised weight by a factor within exp(+-2e) and by the 2^-11 of
    its rounding to fp16, O by another 2^-11.  One part of q' alone would be off by 2^-11 sum |q' K'|, 2e-2."""
    cap = max(64, (max(lens) + 127) // 128 * 128)
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=300 + mode)
    q = (q.astype(np.float32) * 12).astype(np.float16)
    masks = tree_masks(r, B, M, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, lens, cap, page=page)
    assert err == 0
    visible = visible_of(masks, M)
    ref, _, _ = R.attend(q, kc, vc, kcb, vcb, s, lens, visible)
    g, scale = Hq // Hkv, 1 / math.sqrt(128)
    bound = np.zeros_like(ref)
    for b in range(B):
        for h in range(Hkv):
            kt = np.abs(vo.dequantize(kc[b][h][:lens[b]], kcb[h]).astype(np.float64))
            k = R.rows(kc[b][h][:lens[b]], kcb[h], s[h])
            v = R.rows(vc[b][h][:lens[b]], vcb[h])
            for m in range(M):
                see = visible(b, m, lens[b])
                if not see.any():
                    continue
                qh = q[b, m, h * g:(h + 1) * g].astype(np.float64)
                qt = np.abs(vo.transform_query(qh, s[h])) * scale * math.log2(math.e)
                e = math.log(2) * (np.maximum(2.0 ** -22 * qt, 2.0 ** -25) @ kt[see].T + 2.0 ** -17 * (qt @ kt[see].T)).max(axis=1)
                sc = scale * (qh @ k[see].T)
                p = np.exp(sc - sc.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                x = ref[b, m, h * g:(h + 1) * g]
                rel = (np.exp(2 * e) - 1 + 2.0 ** -11 + 2.0 ** -16)[:, None]
                bound[b, m, h * g:(h + 1) * g] = rel * (p @ np.abs(v[see]) + np.abs(x)) + 2.0 ** -11 * np.abs(x) * (1 + rel) + 2.0 ** -24
    d = np.abs(o.astype(np.float64) - ref)
    assert (d <= bound).all(), float((d - bound).max())
    # in the 2-norm: the roundings of the weights and of O are 2^-11 / sqrt(3) rms at most each, e averages out: 4e-4
    # together, and half as much again for a few dominant weights
    assert np.linalg.norm(d) <= 6e-4 * np.linalg.norm(ref), np.linalg.norm(d) / np.linalg.norm(ref)
