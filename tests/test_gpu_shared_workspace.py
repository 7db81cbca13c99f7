"""One workspace that serves a draft step and plain decode steps in turn."""
import numpy as np
import pytest

from tests import helpers as H
from tests.test_gpu_tree import case, tree_masks
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode,B,Hq,Hkv,M,queries,num_splits", [
    (0, 1, 4, 1, 8, 1, 5), (0, 3, 8, 2, 9, 1, 0), (0, 2, 16, 2, 40, 8, 3),     # 8 column groups of the plain queries
    (1, 2, 8, 2, 8, 3, 3), (2, 1, 8, 1, 33, 4, 4), (3, 2, 8, 2, 5, 1, 4), (4, 2, 4, 1, 16, 2, 0),
])
def test_draft_steps_and_plain_steps_share_a_workspace(mode, B, Hq, Hkv, M, queries, num_splits):
    """Tree, plain, tree, plain on one workspace: each result has the bits that a workspace of its own gives."""
    t = H.torch()
    cap = 1024
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=60 + mode)
    k, v = (H.dev(H.pack_cache_role(mode, role, c, cap)) for role, c in ((0, kc), (1, vc)))
    lens = r.integers(500, cap + 1, size=B).astype(np.int32)
    q1 = r.standard_normal((B, queries, Hq, 128)).astype(np.float16)
    dq, dm, dl, dk, dv, ds, dq1 = (H.dev(x) for x in (q, tree_masks(r, B, M, "tree").view(np.int64), lens, kcb, vcb, s, q1))
    a, c = t.zeros_like(dq), t.zeros_like(dq1)
    tree_ws = _lib.decode_tree_workspace(mode, B, Hq, Hkv, M, cap, cap, num_splits)
    plain_ws = _lib.decode_workspace(mode, B, Hq, Hkv, cap, cap, num_splits, n_queries=queries)

    def tree(ws):
        a.fill_(float("nan"))
        _lib.vqkv_decode_attn_tree(mode, dq, dm, k, v, dl, dk, dv, ds, a, ws, cap, cap, num_splits=num_splits)
        return a.clone()

    def plain(ws):
        c.fill_(float("nan"))
        _lib.vqkv_decode_attn_multi(mode, dq1, k, v, dl, dk, dv, ds, c, ws, cap, cap, num_splits=num_splits)
        return c.clone()

    want = [tree(tree_ws), plain(plain_ws)]
    ws = t.zeros(max(tree_ws.numel(), plain_ws.numel()), dtype=t.uint8, device="cuda")
    for _ in range(2):
        got = [tree(ws), plain(ws)]
        assert t.isfinite(want[0]).all() and t.isfinite(want[1]).all()
        assert t.equal(got[0], want[0]) and t.equal(got[1], want[1])
    assert int(ws[:4].view(t.int32).item()) == 0
