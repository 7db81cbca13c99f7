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
from tests.test_gpu_mass import causal
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


def mass_call(mode, Hq, Hkv, M, num_splits, key_pass, stage, polls, seed):
    """The hooked call, then an ordinary one before and one after the error word is cleared: the weights before all,
    after each of the three, the reference's, and the last call's O with its reference and bound."""
    t = H.torch()
    B = len(LENS)
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, CAP, seed=seed)
    before = r.random((B, Hkv, CAP), dtype=np.float32)
    k, v = (H.dev(H.pack_cache_role(mode, role, c, CAP)) for role, c in ((0, kc), (1, vc)))
    dq, dl, dk, dv, ds = (H.dev(x) for x in (q, np.array(LENS, dtype=np.int32), kcb, vcb, s))
    out = t.zeros((B, M, Hq, 128), dtype=t.float16, device="cuda")
    mass = H.dev(before)
    ws = _lib.decode_mass_workspace(mode, B, Hq, Hkv, M, CAP, CAP, num_splits)
    a = _lib.DecodeMassArgs(decode=_lib.decode_args(mode, dq.view(B, M * Hq, 128), k, v, dl, dk, dv, ds, out, ws, CAP, CAP,
                                                    num_splits=num_splits), n_queries=M, mass=mass.data_ptr())
    a.decode.Hq = Hq
    seen = []
    for hooked in (True, False, False):
        if hooked:
            assert _lib.lib().vqkv_test_decode_mass_timeout(ctypes.byref(a), key_pass, stage, polls, None) == 0
        else:
            _lib.vqkv_decode_attn_mass(mode, dq, k, v, dl, dk, dv, ds, out, mass, ws, CAP, CAP, num_splits=num_splits)
        t.cuda.synchronize()
        assert flags(ws) == (_lib.VQKV_DEVERR_TIMEOUT if len(seen) < 2 else 0)
        if len(seen) == 1:
            ws[:4] = 0
        seen.append(mass.cpu().numpy())
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, LENS, causal(M))
    R.check_output(out.cpu().numpy(), ref, tol)
    return before, seen, w


@pytest.mark.parametrize("mode,Hq,Hkv,M,num_splits,stage", [
    (0, 8, 2, 9, 3, 0), (0, 8, 2, 9, 3, 1), (1, 8, 2, 4, 2, 1), (2, 8, 2, 9, 2, 0), (3, 4, 1, 16, 3, 1), (4, 8, 1, 3, 2, 0),
    (0, 4, 1, 1, 0, 0), (0, 8, 2, 3, 3, 0),       # few columns: the ring's waits
])
def test_mass_is_left_alone_when_the_attention_times_out(mode, Hq, Hkv, M, num_splits, stage):
    """Not by the call itself and not by the next one while the error word is set; once it is cleared, as ever."""
    before, seen, w = mass_call(mode, Hq, Hkv, M, num_splits, 0, stage, 512, seed=80 + mode)
    assert np.array_equal(seen[0], before) and np.array_equal(seen[1], before)
    R.check_mass(seen[2], before, w, LENS, R.attend.score_size)


@pytest.mark.parametrize("mode,Hq,Hkv,M,num_splits", [
    (0, 8, 2, 9, 3), (1, 8, 2, 4, 2), (2, 8, 2, 9, 2), (3, 4, 1, 16, 3), (4, 8, 1, 3, 2),
])
@pytest.mark.parametrize("stage", [0, 1])
def test_mass_of_a_timed_out_key_pass_is_whole_or_untouched(mode, Hq, Hkv, M, num_splits, stage):
    """Stage 0: nothing is added.  Stage 1: at most each share's first tile of 128 tokens is."""
    before, seen, w = mass_call(mode, Hq, Hkv, M, num_splits, 1, stage, 4096, seed=90 + mode)
    assert np.array_equal(seen[1], seen[0])
    added = seen[0] != before
    if stage == 0:
        assert not added.any()
    assert added.sum() <= Hkv * num_splits * 128
    whole = seen[2].astype(np.float64) - seen[0]        # the last call added every token's weight once
    for b, L in enumerate(LENS):
        for h in range(Hkv):
            got = np.where(added[b, h, :L], seen[0][b, h, :L].astype(np.float64) - before[b, h, :L], w[b][h])
            # two fp32 additions to values below 1 + M g round by 2^-24 of them each; the weights as in check_mass
            tol = (2 * 2.0 ** -17 * R.attend.score_size + 2.0 ** -17) * w[b][h] + 2.0 ** -23 * (1 + w[b][h])
            assert (np.abs(got - w[b][h]) <= tol).all()
            assert (np.abs(whole[b, h, :L] - w[b][h]) <= 2 * tol).all()
