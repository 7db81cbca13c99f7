"""The bounded waits of the draft-tree and attention-weight kernels on the
tensor cores, made to run out on purpose.

The test hooks give one ring stage's barrier an arrival that nothing makes and
limit each wait to a few polls.  The call must finish, set VQKV_DEVERR_TIMEOUT
in the workspace's error word and leave the context usable: the next ordinary
call on the same workspace is correct.  No fault, trap or hang is involved:
nothing waits for more than max_polls polls, and the products already issued
end by themselves."""
import ctypes

import numpy as np
import pytest

from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_tree import case, tree_masks, visible_of
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu

LENS = [1, 0, 700, 64, 65, 0, 333, 128, 449, 17]   # pieces of one tile and of many, shares that hold several
CAP = 768


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def flags(ws):
    return int(ws[:4].view(H.torch().int32).item())


@pytest.mark.parametrize("stage", [0, 1])   # every CTA has several tiles, so both stages are used
@pytest.mark.parametrize("mode,Hq,Hkv,M,num_splits", [
    (0, 8, 2, 9, 3), (0, 8, 1, 33, 2), (1, 4, 1, 9, 3), (2, 8, 1, 20, 2), (3, 4, 2, 9, 2), (4, 8, 1, 50, 4),
])
def test_tree_waits_run_out_and_are_reported(mode, Hq, Hkv, M, num_splits, stage):
    t = H.torch()
    B = len(LENS)
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, CAP, seed=70 + mode)
    masks = tree_masks(r, B, M, "tree")
    k, v = (H.dev(H.pack_cache_role(mode, role, c, CAP)) for role, c in ((0, kc), (1, vc)))
    dq, dm, dl, dk, dv, ds = (H.dev(x) for x in (q, masks.astype(np.uint64).view(np.int64), np.array(LENS, dtype=np.int32),
                                                 kcb, vcb, s))
    out = t.zeros((B, M, Hq, 128), dtype=t.float16, device="cuda")
    ws = _lib.decode_tree_workspace(mode, B, Hq, Hkv, M, CAP, CAP, num_splits)
    a = _lib.DecodeTreeArgs(decode=_lib.decode_args(mode, dq.view(B, M * Hq, 128), k, v, dl, dk, dv, ds, out, ws, CAP, CAP,
                                                    num_splits=num_splits), n_queries=M, tree_mask=dm.data_ptr())
    a.decode.Hq = Hq
    for _ in range(3):
        ws[:4] = 0
        assert _lib.lib().vqkv_test_decode_tree_timeout(ctypes.byref(a), stage, 64, None) == 0
        t.cuda.synchronize()
        assert flags(ws) == _lib.VQKV_DEVERR_TIMEOUT
    ws[:4] = 0
    _lib.vqkv_decode_attn_tree(mode, dq, dm, k, v, dl, dk, dv, ds, out, ws, CAP, CAP, num_splits=num_splits)
    t.cuda.synchronize()
    assert flags(ws) == 0
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, LENS, visible_of(masks, M))
    R.check_output(out.cpu().numpy(), ref, tol)
