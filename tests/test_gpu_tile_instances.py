"""Every instance of the tile kernels: mode x contiguous or paged x one or two
query tiles (draft trees), up to 32 or up to 64 columns (key pass)."""
import numpy as np
import pytest

from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_mass import causal, gpu_mass
from tests.test_gpu_tree import case, gpu_tree, tree_masks, visible_of
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu

LENS, CAP = [333, 64, 0, 513], 640


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("page", [0, 64, 128])
@pytest.mark.parametrize("Hq,M", [(8, 11), (12, 23)])      # 44 and 138 columns per KV head
def test_tree_instances(mode, page, Hq, M):
    B = len(LENS)
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, 2, M, CAP, seed=200 + mode)
    masks = tree_masks(r, B, M, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, LENS, CAP, num_splits=3, page=page)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, LENS, visible_of(masks, M))
    R.check_output(o, ref, tol)
    assert err == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("page", [0, 64, 128])
@pytest.mark.parametrize("Hq,M", [(8, 7), (10, 11)])       # 28 and 55 columns per KV head
def test_mass_instances(mode, page, Hq, M):
    B = len(LENS)
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, 2, M, CAP, seed=210 + mode)
    before = (r.random((B, 2, CAP)) * M / 100).astype(np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, LENS, CAP, before, num_splits=3, page=page)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, LENS, causal(M))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, LENS, R.attend.score_size)
    assert err == 0
