"""Cross attention where the running max moves in nearly every tile (the scores of
tests/test_gpu_rescale.py), and where scores are large: every way its columns are laid
out on the tensor cores."""
import numpy as np
import pytest

from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_cross import Cross
from tests.test_gpu_rescale import L, SCALE, TILES, check_the_climb, climbing
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("Hq,M,dt", [(4, 9, "fp16"), (8, 9, "fp16"), (8, 33, "fp16"), (8, 16, "bf16"), (8, 33, "bf16")])
@pytest.mark.parametrize("num_splits", [1, 3])
def test_the_accumulator_is_rescaled(t, mode, Hq, M, dt, num_splits):
    """Columns on paired rows; one query tile of both parts of q', two items of it; one and two query tiles of one part."""
    _, q, kc, vc, s, kcb, vcb = climbing(mode, Hq, M, 8.5, seed=20 + mode)
    check_the_climb(q, kc, kcb, s, 1)
    assert L == 64 * TILES
    dtype = t.float16 if dt == "fp16" else t.bfloat16
    rows = H.dev(q[0]).to(dtype)                          # entries of a Hadamard matrix: exact in both types
    out = t.full_like(rows, 3.0)
    k, v = (H.dev(H.pack_cache_role(mode, role, c, L)) for role, c in ((0, kc), (1, vc)))
    ws = _lib.cross_attn_workspace(mode, 1, Hq, 1, M, M, L, L, num_splits, dtype=0 if dt == "fp16" else 2)
    _lib.vqkv_cross_attn(mode, rows, H.dev(np.array([0, M], dtype=np.int32)), k, v, H.dev(np.array([L], dtype=np.int32)),
                         H.dev(kcb), H.dev(vcb), H.dev(s), out, ws, L, L, M, softmax_scale=SCALE, num_splits=num_splits)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, [L], lambda *_: np.ones(L, dtype=bool), scale=SCALE)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol[0]).all()
    assert int(ws.view(t.int32)[0]) == 0


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("queries", [[8, 5], [65, 33], [200, 1]])
def test_both_parts_of_the_query_count(t, mode, queries):
    """Scores of some 11 nats (rms): a q' rounded to 2^-12 (rms about 1.4e-4 of a score) would move every weight by
    about 1e-3.  With both parts only the weights' and the result's roundings to fp16 are left, uniform within 2^-11
    relative each: 2^-11 / sqrt(3) rms at most, together below 4.0e-4, and 2 % for the sample."""
    x = Cross(t, mode, 8, 4, queries, [500, 300], seed=30 + mode, qscale=12.0)
    got = x.run().double().cpu().numpy()
    ref, _ = x.reference()
    assert np.linalg.norm(got - ref) <= 4.1e-4 * np.linalg.norm(ref)
    assert x.flags() == 0


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("dt,block_tokens", [("fp16", 0), ("bf16", 64), ("fp16", 256)])
@pytest.mark.parametrize("queries,lens", [
    ([1, 1, 0, 1, 1], [6000, 17, 400, 0, 2500]),       # shares of all sequences' tokens, but at 1.5 bit
    ([1] * 40, [300 + 7 * i for i in range(40)]),      # a CTA per sequence
    ([1], [7000]),                                     # splits of one
])
def test_single_queries_long_and_short(t, mode, dt, block_tokens, queries, lens):
    x = Cross(t, mode, 4, 2, queries, lens, dt=dt, block_tokens=block_tokens, seed=mode)
    got = x.run()
    x.check(got, *x.reference())
    assert x.flags() == 0
    assert t.equal(got, x.run(out=t.full_like(x.out, 3.0), ws=x.ws))
