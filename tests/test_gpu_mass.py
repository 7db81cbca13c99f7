"""Decode attention with accumulated attention weights (vqkv_decode_attn_mass)
through the C ABI against a plain fp64 attention."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import attn_reference as R
from tests import helpers as H
from tests.test_gpu_tree import case, paged_args
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def causal(M):
    return lambda b, m, L: np.arange(L) <= L - M + m


def gpu_mass(mode, q, kc, vc, s, kcb, vcb, lens, cap, before, num_splits=0, page=0, calls=1, scale=0.0, max_seq_len=None):
    t = H.torch()
    B, M, Hq, _ = q.shape
    Hkv = kcb.shape[0]
    bufs = [H.pack_cache_role(mode, 0, kc, cap), H.pack_cache_role(mode, 1, vc, cap)]
    kw = {}
    if page:
        bufs, kw = paged_args(np.random.default_rng(7), page, bufs, B, Hkv, mode, cap)
    else:
        bufs = [H.dev(x) for x in bufs]
    hi = cap if max_seq_len is None else max_seq_len
    out = t.full((B, M, Hq, 128), float("nan"), dtype=t.float16, device="cuda")
    mass = H.dev(before)
    ws = _lib.decode_mass_workspace(mode, B, Hq, Hkv, M, cap, hi, num_splits)
    args = [H.dev(x) for x in (q, np.asarray(lens, dtype=np.int32), kcb, vcb, s)]
    for _ in range(calls):
        _lib.vqkv_decode_attn_mass(mode, args[0], bufs[0], bufs[1], args[1], args[2], args[3], args[4], out, mass, ws, cap,
                                   hi, softmax_scale=scale, num_splits=num_splits, **kw)
    t.cuda.synchronize()
    return out.cpu().numpy(), mass.cpu().numpy(), int(ws[:4].view(t.int32).item())


CASES = [
    # mode, B, Hq, Hkv, M, lens, cap, num_splits, page
    (0, 1, 1, 1, 1, [1], 16, 0, 0),
    (0, 1, 4, 1, 1, [1000], 1024, 0, 0),
    (0, 1, 4, 1, 1, [1000], 1024, 1, 0),
    (0, 1, 8, 1, 1, [1000], 1024, 5, 0),            # 8 heads per KV head: two column groups
    (0, 1, 5, 1, 1, [333], 400, 0, 0),              # groups of 4 and 1
    (0, 3, 8, 2, 1, [0, 517, 49], 640, 0, 0),       # the flat plan; an empty sequence
    (0, 2, 8, 2, 7, [517, 3], 640, 0, 64),          # an observation window; fewer tokens than queries
    (0, 1, 8, 8, 64, [200], 208, 3, 0),             # 64 queries of one head
    (1, 1, 4, 1, 1, [1000], 1024, 3, 0),
    (1, 3, 10, 2, 1, [700, 64, 1], 768, 0, 256),    # several sequences per CTA, deferred merge
    (1, 2, 4, 2, 5, [300, 4], 320, 0, 0),
    (2, 1, 4, 1, 1, [1000], 1024, 0, 0),
    (2, 3, 6, 2, 3, [513, 100, 0], 576, 0, 64),
    (3, 1, 4, 1, 1, [1000], 1024, 0, 0),
    (3, 3, 8, 2, 2, [600, 17, 300], 640, 0, 128),
    (4, 1, 4, 1, 1, [1000], 1024, 0, 0),
    (4, 3, 3, 1, 4, [600, 20, 2], 640, 0, 64),
]


@pytest.mark.parametrize("mode,B,Hq,Hkv,M,lens,cap,num_splits,page", CASES)
def test_mass_against_reference(mode, B, Hq, Hkv, M, lens, cap, num_splits, page):
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=50 * mode + M + B)
    before = (r.random((B, Hkv, cap)) * M / max(max(lens), 1)).astype(np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, lens, cap, before, num_splits, page)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, causal(M))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, lens, R.attend.score_size)
    assert err == 0


@pytest.mark.parametrize("mode,Hq,Hkv,M,num_splits,page", [
    (0, 8, 2, 3, 0, 0), (0, 8, 2, 4, 0, 0), (0, 8, 2, 5, 0, 0), (0, 8, 2, 8, 3, 64), (0, 8, 2, 9, 0, 0), (0, 4, 1, 16, 5, 0), (1, 10, 2, 6, 0, 128),
    (2, 8, 1, 8, 0, 64), (3, 8, 2, 16, 2, 0), (4, 3, 1, 21, 0, 64),
])
def test_mass_many_columns_ragged_batch(mode, Hq, Hkv, M, num_splits, page):
    """More columns than the decode path takes: shares that begin and end inside sequences, hold several, or none."""
    lens = [1, 0, 700, 128, 129, 0, 333, 127, 449, 17]
    B, cap = len(lens), 768
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=3 * mode + M)
    before = (r.random((B, Hkv, cap)) * M / 100).astype(np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, lens, cap, before, num_splits, page)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, causal(M))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, lens, R.attend.score_size)
    assert err == 0


@pytest.mark.parametrize("M", [1, 9])   # few columns; many, in launches of at most 1024 sequences
def test_mass_more_sequences_than_one_launch_takes(M):
    B = 1027
    r = np.random.default_rng(3)
    lens = r.integers(0, 40, size=B)
    s, kcb, vcb = H.random_codebooks(0, 1, 4)
    kc = [[r.integers(0, 256, size=(48, 32))] for _ in range(B)]
    vc = [[r.integers(0, 256, size=(48, 32))] for _ in range(B)]
    q = r.standard_normal((B, M, 2, 128)).astype(np.float16)
    before = np.zeros((B, 1, 48), dtype=np.float32)
    o, mass, err = gpu_mass(0, q, kc, vc, s, kcb, vcb, lens, 48, before)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, causal(M))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, lens, R.attend.score_size)


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_mass_many_columns_long_and_repeatable(mode):
    r, q, kc, vc, s, kcb, vcb = case(mode, 1, 8, 2, 12, 4100, seed=mode)
    before = np.zeros((1, 2, 4100), dtype=np.float32)
    o, mass, err = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [4099], 4100, before, num_splits=2)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, [4099], causal(12))
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, [4099], R.attend.score_size)
    o2, again, _ = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [4099], 4100, before, num_splits=2)
    assert np.array_equal(mass, again) and np.array_equal(o, o2)


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_mass_sums_to_the_number_of_columns_and_repeats(mode):
    """From zero: each (sequence, KV head) row gains g per call; a second run gives the same bits."""
    r, q, kc, vc, s, kcb, vcb = case(mode, 2, 8, 2, 1, 3000, seed=mode)
    before = np.zeros((2, 2, 3000), dtype=np.float32)
    o, a, _ = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [2999, 1234], 3000, before)
    _, c, _ = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [2999, 1234], 3000, before)
    assert np.array_equal(a, c)
    assert np.abs(a.astype(np.float64).sum(axis=2) - 4).max() <= 4e-5
    _, d, _ = gpu_mass(mode, q, kc, vc, s, kcb, vcb, [2999, 1234], 3000, before, calls=3)
    assert np.abs(d - 3 * a.astype(np.float64)).max() <= 3 * 2.0 ** -23 * a.max() * 2


def test_mass_scale_and_clamped_lengths():
    r, q, kc, vc, s, kcb, vcb = case(0, 3, 4, 2, 2, 300, seed=9)
    before = np.ones((3, 2, 300), dtype=np.float32)
    o, mass, err = gpu_mass(0, q, kc, vc, s, kcb, vcb, [400, -2, 77], 300, before, scale=0.05, max_seq_len=250)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, [250, 0, 77], causal(2), scale=0.05)
    R.check_output(o, ref, tol)
    R.check_mass(mass, before, w, [250, 0, 77], R.attend.score_size)
    assert err == _lib.VQKV_DEVERR_SEQ_LEN


@pytest.mark.parametrize("M", [1, 9])
def test_mass_large_scores_keep_fp32_weights(M):
    """Scores near 40: a single fp16 part of q' would put 1e-2 into the weights (few and many columns)."""
    r, q, kc, vc, s, kcb, vcb = case(0, 1, 4, 1, M, 512, seed=4)
    q = (q.astype(np.float32) * 12).astype(np.float16)
    before = np.zeros((1, 1, 512), dtype=np.float32)
    o, mass, _ = gpu_mass(0, q, kc, vc, s, kcb, vcb, [512], 512, before)
    ref, w, tol = R.attend(q, kc, vc, kcb, vcb, s, [512], causal(M))
    rel = np.linalg.norm(mass[0, 0] - w[0][0]) / np.linalg.norm(w[0][0])
    assert rel <= 2 * 2.0 ** -17 * R.attend.score_size + 2.0 ** -17


def test_mass_matches_plain_decode_and_graphs():
    """O equals vqkv_decode_attn's up to rounding; a captured step on another stream accumulates at each replay."""
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(2, 2, 8, 2, 1, 900, seed=12)
    lens = [900, 321]
    bufs = [H.pack_cache_role(2, 0, kc, 900), H.pack_cache_role(2, 1, vc, 900)]
    want = H.gpu_decode(2, q[:, 0], bufs[0], bufs[1], lens, kcb, vcb, s, 900, 900).astype(np.float64)
    dq, dl, dk, dv, ds = (H.dev(x) for x in (q, np.array(lens, dtype=np.int32), kcb, vcb, s))
    k, v = H.dev(bufs[0]), H.dev(bufs[1])
    out = t.zeros((2, 1, 8, 128), dtype=t.float16, device="cuda")
    mass = t.zeros((2, 2, 900), device="cuda")
    ws = _lib.decode_mass_workspace(2, 2, 8, 2, 1, 900, 900)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        _lib.vqkv_decode_attn_mass(2, dq, k, v, dl, dk, dv, ds, out, mass, ws, 900, 900)
    side.synchronize()
    once = mass.clone()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side):
        _lib.vqkv_decode_attn_mass(2, dq, k, v, dl, dk, dv, ds, out, mass, ws, 900, 900)
    mass.zero_()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        g.replay()
        g.replay()
    t.cuda.synchronize()
    assert t.equal(mass, once + once)
    o = out.cpu().numpy()[:, 0].astype(np.float64)
    assert np.linalg.norm(o - want) <= 4e-3 * np.linalg.norm(want)


def test_mass_bad_block_ids_are_reported():
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(0, 1, 4, 1, 1, 128, seed=2)
    bufs = [H.pack_cache_role(0, 0, kc, 128), H.pack_cache_role(0, 1, vc, 128)]
    pools, kw = paged_args(r, 64, bufs, 1, 1, 0, 128)
    kw["block_table"] = H.dev(np.array([[kw["num_blocks"], -5]], dtype=np.int32))
    ws = _lib.decode_mass_workspace(0, 1, 4, 1, 1, 128, 128)
    out, mass = t.zeros((1, 1, 4, 128), dtype=t.float16, device="cuda"), t.zeros((1, 1, 128), device="cuda")
    _lib.vqkv_decode_attn_mass(0, H.dev(q), pools[0], pools[1], H.dev(np.array([128], dtype=np.int32)), H.dev(kcb),
                               H.dev(vcb), H.dev(s), out, mass, ws, 128, 128, **kw)
    assert int(ws[:4].view(t.int32).item()) == _lib.VQKV_DEVERR_BLOCK
    assert t.isfinite(out).all() and t.isfinite(mass).all()


def test_binding_refuses_wrong_tensors():
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(0, 1, 4, 1, 1, 64, seed=2)
    k, v = H.dev(H.pack_cache_role(0, 0, kc, 64)), H.dev(H.pack_cache_role(0, 1, vc, 64))
    dq, dl, dk, dv, ds = (H.dev(x) for x in (q, np.array([64], dtype=np.int32), kcb, vcb, s))
    out, mass = t.zeros((1, 1, 4, 128), dtype=t.float16, device="cuda"), t.zeros((1, 1, 64), device="cuda")
    ws = _lib.decode_mass_workspace(0, 1, 4, 1, 1, 64, 64)
    tree = t.ones((1, 1), dtype=t.int64, device="cuda")
    with pytest.raises(ValueError):
        _lib.vqkv_decode_attn_mass(0, dq, k, v, dl, dk, dv, ds, out, mass[:, :, :32].contiguous(), ws, 64, 64)
    with pytest.raises(ValueError):
        _lib.vqkv_decode_attn_mass(1, dq, k, v, dl, dk, dv, ds, out, mass, ws, 64, 64)    # codebooks of another mode
    with pytest.raises(TypeError):
        _lib.vqkv_decode_attn_mass(0, dq, k, v, dl, dk, dv, ds, out, mass.double(), ws, 64, 64)
    with pytest.raises(_lib.VqkvError):
        _lib.vqkv_decode_attn_mass(0, dq, k, v, dl, dk, dv, ds, out, mass, ws[:256], 64, 64)
    with pytest.raises(TypeError):
        _lib.vqkv_decode_attn_tree(0, dq, tree.int(), k, v, dl, dk, dv, ds, out, ws, 64, 64)
    with pytest.raises(ValueError):
        _lib.vqkv_decode_attn_tree(0, dq, tree.expand(1, 2), k, v, dl, dk, dv, ds, out, ws, 64, 64)
    with pytest.raises(ValueError):
        _lib.vqkv_decode_attn_tree(0, dq, tree, k.expand(2, -1, -1)[1:], v[:, :, :256], dl, dk, dv, ds, out, ws, 64, 64)
