"""Scores that climb by more than the lazy-rescale slack (2^8) from tile to
tile: the running max moves, and the accumulator in tensor memory, the running
sum and the merge of the two softmax warpgroups have to follow.

A column looks along one channel r of K'.  There the 64 tokens of tile j < r
stand at d (j - r) in the log2 domain, one token of tile r at 0 and the rest
of it at -40, later tiles at -20.  With d = 8.5 (a warpgroup that takes every
tile) or 4.25 (every other tile) the max moves by 8.5 in each of a warpgroup's
tiles up to the last, and the tile before the last move still holds 64 x 2^-8.5
= 0.18 of the last one's weight, so an accumulator that is not scaled, scaled
twice or dropped shows in O.  Columns of one warp look along different
channels: some rise while others have passed their top.  q' and K' are exact
in fp16."""
import math

import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_mass import causal, gpu_mass
from tests.test_gpu_tree import gpu_tree, tree_masks, visible_of
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu

TILES, TOK = 16, 64
L = TILES * TOK
SCALE = math.sqrt(128) / math.log2(math.e) * 2.0 ** -7     # q' = 2^-7 x the unnormalised transform of q


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def climbing(mode, Hq, M, step, seed):
    """One sequence of one KV head: q, codes, s, codebooks; column c looks along channel 1 + c % 15."""
    r = np.random.default_rng(seed)
    E, d = vo.GEOMETRY[mode]
    s, kcb, vcb = H.random_codebooks(mode, 1, seed)
    s[:] = 1.0
    top = r.integers(0, TOK, size=TILES)                   # the token of tile r that stands at 0
    level = np.empty((TILES, 2, 16))                       # [tile][is its top][channel]
    for j in range(TILES):
        for c in range(16):
            level[j, :, c] = step * (j - c) if j < c else (-40.0, 0.0) if j == c else -20.0
    kc = r.integers(0, E, size=(L, 128 // d))
    for u in range(16 // d):                               # entries 32 u .. 32 u + 31 are subvector u's
        for j in range(TILES):
            for f in range(2):
                kcb[0, 32 * u + 2 * j + f] = level[j, f, d * u:d * u + d].astype(np.float16)
        is_top = np.arange(L) % TOK == np.repeat(top, TOK)
        kc[:, u] = 32 * u + 2 * (np.arange(L) // TOK) + is_top
    vc = r.integers(0, E, size=(L, 128 // d))
    had = np.round(vo.normalized_hadamard() * math.sqrt(128))
    q = np.empty((1, M, Hq, 128), dtype=np.float16)
    for m in range(M):
        for h in range(Hq):
            q[0, m, h] = had[1 + (m * Hq + h) % 15]
    return r, q, [[kc]], [[vc]], s, kcb, vcb


def check_the_climb(q, kc, kcb, s, every):
    """The lazy rule on the CPU: how often a warpgroup's columns move their max, and what the moved-over tiles weigh."""
    qt = np.round(vo.transform_query(q[0].reshape(-1, 128).astype(np.float64), s[0]) * SCALE * math.log2(math.e), 6)
    sc = qt @ vo.dequantize(kc[0][0], kcb[0]).astype(np.float64).T          # log2 domain [columns][L]
    moves, kept = [], []
    for col in sc:
        p = np.exp2(col - col.max())
        for first in range(every):
            m, n, at = -1e30, 0, 0
            for j in range(first, TILES, every):
                x = col[TOK * j:TOK * (j + 1)].max()
                if x > m + 8:
                    n, m, at = n + (m > -1e29), x, j
            moves.append(n)
            mine = np.concatenate([p[TOK * j:TOK * (j + 1)] for j in range(first, TILES, every)])
            old = sum(p[TOK * j:TOK * (j + 1)].sum() for j in range(first, at, every))
            kept.append(old / mine.sum())
    assert max(moves) >= TILES // every - 2 and np.mean(moves) >= TILES / every / 4
    assert np.mean(np.array(kept) > 0.05) > 0.4          # in many columns the rescaled part counts


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("Hq,M,step,every", [(4, 9, 4.25, 2), (8, 16, 4.25, 2), (8, 20, 8.5, 1), (8, 32, 8.5, 1)])
def test_tree_rescales_the_accumulator(mode, Hq, M, step, every):
    """Up to 128 columns the warpgroups take the tiles in turn; above, each takes every tile."""
    r, q, kc, vc, s, kcb, vcb = climbing(mode, Hq, M, step, seed=mode)
    check_the_climb(q, kc, kcb, s, every)
    masks = tree_masks(r, 1, M, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, [L], L, num_splits=1, scale=SCALE)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, [L], visible_of(masks, M), scale=SCALE)
    R.check_output(o, ref, tol)
    assert err == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("M", [3, 9, 16])        # few columns (the decode's kernels), many
def test_mass_rescales_the_accumulator(mode, M):
    r, q, kc, vc, s, kcb, vcb = climbing(mode, 4, M, 4.25, seed=10 + mode)
    check_the_climb(q, kc, kcb, s, 2)
    before = np.zeros((1, 1, L), dtype=np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [L], L, before, num_splits=1, scale=SCALE)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, [L], causal(M), scale=SCALE)
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, [L], R.attend.score_size)
    assert err == 0
