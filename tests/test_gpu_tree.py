"""Draft-tree attention (vqkv_decode_attn_tree) through the C ABI against a
plain fp64 attention with the same visibility."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import attn_reference as R
from tests import helpers as H
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def tree_masks(r, B, M, kind):
    """uint64 [B][M]."""
    full = (1 << M) - 1
    out = np.zeros((B, M), dtype=np.uint64)
    for b in range(B):
        for m in range(M):
            if kind == "chain":
                v = (1 << (m + 1)) - 1
            elif kind == "tree":
                v = (1 << m) | (int(out[b, r.integers(0, m)]) if m else 0)
            elif kind == "random":
                v = int(r.integers(0, 1 << 62)) & full
            elif kind == "none":
                v = 0
            elif kind == "high":      # bits past M and bits of later drafts
                v = (1 << m) | (~full & (2**64 - 1)) | (full & 0x5555555555555555)
            else:
                v = full
            out[b, m] = v
    return out


def case(mode, B, Hq, Hkv, M, cap, seed):
    r = np.random.default_rng(seed)
    E, d = vo.GEOMETRY[mode]
    s, kcb, vcb = H.random_codebooks(mode, Hkv, seed + 1)
    kc = [[r.integers(0, E, size=(cap, 128 // d)) for _ in range(Hkv)] for _ in range(B)]
    vc = [[r.integers(0, E, size=(cap, 128 // d)) for _ in range(Hkv)] for _ in range(B)]
    q = r.standard_normal((B, M, Hq, 128)).astype(np.float16)
    return r, q, kc, vc, s, kcb, vcb


def visible_of(masks, M):
    def visible(b, m, L):
        t = np.arange(L)
        j = t - (L - M)
        bit = (int(masks[b, m]) >> np.clip(j, 0, 63).astype(object)) & 1
        return (j < 0) | (bit.astype(np.int64) == 1)
    return visible


def paged_args(r, page, bufs, B, Hkv, mode, cap):
    """Pools, shuffled, from contiguous streams of a whole number of pages."""
    per, bb = cap // page, vo.code_bytes(mode, page)
    nblk = B * per + 2
    table = r.permutation(nblk)[:B * per].reshape(B, per).astype(np.int32)
    pools = []
    for x in bufs:
        pool = r.integers(0, 256, size=(nblk, Hkv, bb), dtype=np.uint8)
        for b in range(B):
            for i in range(per):
                pool[table[b, i]] = x[b, :, i * bb:(i + 1) * bb]
        pools.append(H.dev(pool))
    return pools, {"block_table": H.dev(table), "block_tokens": page, "num_blocks": nblk}


def gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, lens, cap, num_splits=0, page=0, seed=0, scale=0.0, max_seq_len=None):
    t = H.torch()
    B, M, Hq, _ = q.shape
    Hkv = kcb.shape[0]
    bufs = [H.pack_cache_role(mode, 0, kc, cap), H.pack_cache_role(mode, 1, vc, cap)]
    kw = {}
    if page:
        bufs, kw = paged_args(np.random.default_rng(seed), page, bufs, B, Hkv, mode, cap)
    else:
        bufs = [H.dev(x) for x in bufs]
    hi = cap if max_seq_len is None else max_seq_len
    out = t.full((B, M, Hq, 128), float("nan"), dtype=t.float16, device="cuda")
    ws = _lib.decode_tree_workspace(mode, B, Hq, Hkv, M, cap, hi, num_splits)
    _lib.vqkv_decode_attn_tree(mode, H.dev(q), H.dev(masks.astype(np.uint64).view(np.int64)), bufs[0], bufs[1],
                               H.dev(np.asarray(lens, dtype=np.int32)), H.dev(kcb), H.dev(vcb), H.dev(s), out, ws, cap, hi,
                               softmax_scale=scale, num_splits=num_splits, **kw)
    t.cuda.synchronize()
    return out.cpu().numpy(), int(ws[:4].view(t.int32).item())


CASES = [
    # mode, B, Hq, Hkv, M, lens, cap, num_splits, page, masks
    (0, 1, 4, 1, 1, [1], 16, 0, 0, "chain"),
    (0, 1, 4, 1, 1, [64], 64, 0, 0, "chain"),
    (0, 1, 4, 1, 2, [65], 128, 0, 0, "none"),
    (0, 1, 8, 2, 8, [1000], 1024, 0, 0, "tree"),
    (0, 1, 8, 2, 8, [1000], 1024, 1, 0, "tree"),
    (0, 2, 8, 2, 9, [130, 5], 257, 3, 0, "tree"),            # a sequence shorter than its drafts
    (0, 2, 4, 4, 16, [16, 0], 64, 0, 0, "random"),           # no prefix; an empty sequence
    (0, 1, 4, 4, 16, [16], 64, 0, 0, "none"),                # no prefix and no mask: zero rows
    (0, 1, 40, 5, 64, [700], 704, 0, 0, "random"),           # 512 columns in four groups
    (0, 1, 5, 1, 33, [193], 200, 2, 0, "high"),              # 165 columns
    (0, 1, 2, 2, 64, [64], 64, 0, 0, "full"),
    (0, 3, 4, 1, 31, [900, 33, 448], 960, 0, 64, "tree"),
    (1, 1, 8, 2, 8, [1000], 1024, 0, 0, "tree"),
    (1, 2, 10, 2, 27, [700, 64], 768, 4, 256, "tree"),
    (2, 1, 8, 2, 8, [1000], 1024, 0, 0, "tree"),
    (2, 2, 6, 2, 40, [513, 100], 576, 2, 64, "random"),
    (3, 1, 8, 2, 8, [1000], 1024, 0, 0, "tree"),
    (3, 2, 8, 1, 17, [600, 17], 640, 3, 128, "tree"),
    (4, 1, 8, 2, 8, [1000], 1024, 0, 0, "tree"),
    (4, 2, 3, 3, 21, [600, 20], 640, 3, 64, "random"),
]


@pytest.mark.parametrize("mode,B,Hq,Hkv,M,lens,cap,num_splits,page,kind", CASES)
def test_tree_against_reference(mode, B, Hq, Hkv, M, lens, cap, num_splits, page, kind):
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=100 * mode + M)
    masks = tree_masks(r, B, M, kind)
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, lens, cap, num_splits, page)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, visible_of(masks, M))
    R.check_output(o, ref, tol)
    assert err == 0
    vis = visible_of(masks, M)
    for b in range(B):
        for m in range(M):
            if not vis(b, m, int(lens[b])).any():
                assert np.all(o[b, m] == 0)


@pytest.mark.parametrize("mode,Hq,Hkv,M,num_splits,page", [
    (0, 8, 2, 9, 0, 0), (0, 8, 2, 9, 5, 64), (0, 8, 1, 33, 7, 0), (0, 8, 1, 33, 0, 0), (1, 5, 1, 30, 3, 128),
    (2, 4, 1, 64, 5, 0), (3, 8, 1, 20, 4, 0), (4, 8, 1, 50, 6, 64), (4, 3, 1, 7, 1, 0),
])
def test_tree_ragged_batches(mode, Hq, Hkv, M, num_splits, page):
    """Shares that begin and end inside sequences, hold several of them, an odd number of tiles, or none; one and two
    query tiles per CTA, a second one with few columns."""
    lens = [1, 0, 700, 64, 65, 0, 333, 128, 449, 17]
    B, cap = len(lens), 768
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=7 * mode + M)
    masks = tree_masks(r, B, M, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, lens, cap, num_splits, page)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, visible_of(masks, M))
    R.check_output(o, ref, tol)
    assert err == 0
    assert np.all(o[1] == 0) and np.all(o[5] == 0)


@pytest.mark.parametrize("mode,Hq,M", [(0, 4, 9), (1, 4, 9), (2, 8, 20), (3, 4, 33), (4, 8, 30)])   # one and two query tiles
def test_tree_many_short_sequences_in_two_shares_repeat(mode, Hq, M):
    """Twenty calls back to back over 24 short sequences in two CTAs, whose roles run ahead of each other from one
    sequence to the next: every call the reference's result, and all the same bits."""
    t = H.torch()
    B, cap = 24, 208
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, 1, M, cap, seed=31 + mode)
    lens = r.integers(0, cap + 1, size=B).astype(np.int32)
    masks = tree_masks(r, B, M, "tree")
    k, v = (H.dev(H.pack_cache_role(mode, role, c, cap)) for role, c in ((0, kc), (1, vc)))
    args = [H.dev(x) for x in (q, masks.astype(np.uint64).view(np.int64), lens, kcb, vcb, s)]
    outs = [t.full((B, M, Hq, 128), float("nan"), dtype=t.float16, device="cuda") for _ in range(20)]
    ws = _lib.decode_tree_workspace(mode, B, Hq, 1, M, cap, cap, 2)
    for o in outs:
        _lib.vqkv_decode_attn_tree(mode, args[0], args[1], k, v, args[2], args[3], args[4], args[5], o, ws, cap, cap,
                                   num_splits=2)
    t.cuda.synchronize()
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, visible_of(masks, M))
    R.check_output(outs[0].cpu().numpy(), ref, tol)
    assert all(t.equal(o, outs[0]) for o in outs[1:])
    assert int(ws[:4].view(t.int32).item()) == 0


def test_tree_more_sequences_than_one_launch_takes():
    B, M = 1030, 2
    r = np.random.default_rng(3)
    lens = r.integers(0, 40, size=B)
    s, kcb, vcb = H.random_codebooks(0, 1, 4)
    kc = [[r.integers(0, 256, size=(48, 32))] for _ in range(B)]
    vc = [[r.integers(0, 256, size=(48, 32))] for _ in range(B)]
    q = r.standard_normal((B, M, 2, 128)).astype(np.float16)
    masks = tree_masks(r, B, M, "random")
    o, err = gpu_tree(0, q, masks, kc, vc, s, kcb, vcb, lens, 48)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, lens, visible_of(masks, M))
    R.check_output(o, ref, tol)


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_tree_long_prefix_two_query_tiles(mode):
    r, q, kc, vc, s, kcb, vcb = case(mode, 1, 8, 1, 20, 3000, seed=mode)
    masks = tree_masks(r, 1, 20, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, [2999], 3000, num_splits=2)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, [2999], visible_of(masks, 20))
    R.check_output(o, ref, tol)
    assert err == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_tree_long_prefix_many_tiles(mode):
    # enough tiles per CTA to wrap both rings and the code prefetch many times
    r, q, kc, vc, s, kcb, vcb = case(mode, 1, 4, 1, 6, 5000, seed=mode)
    masks = tree_masks(r, 1, 6, "tree")
    o, err = gpu_tree(mode, q, masks, kc, vc, s, kcb, vcb, [4999], 5000, num_splits=2)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, [4999], visible_of(masks, 6))
    R.check_output(o, ref, tol)
    assert err == 0


@pytest.mark.parametrize("M", [8, 40])
def test_tree_rising_scores_rescale_the_accumulator(M):
    """Keys whose scores climb tile after tile: the running max moves in every tile (one and two query tiles)."""
    r, q, kc, vc, s, kcb, vcb = case(0, 1, 4, 1, M, 1024, seed=5)
    s[:] = 1.0
    # codebook entry e is e/256 of a fixed direction, token t takes entry t / 4
    d = vo.transform_query(q[0, 0, 0][None], s[0])[0]
    step = (np.arange(256) / 256.0)[:, None] * np.sign(d[:4])[None, :] * 4.0
    kcb[0] = step.astype(np.float16)
    kc[0][0] = np.repeat((np.arange(1024) // 4)[:, None], 32, axis=1)
    q[:] = np.sign(vo.normalized_hadamard() @ np.tile(np.sign(d[:4]), 32)).astype(np.float16)[None, None, None]
    masks = tree_masks(r, 1, M, "chain")
    o, err = gpu_tree(0, q, masks, kc, vc, s, kcb, vcb, [1024], 1024, num_splits=1)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, [1024], visible_of(masks, M))
    R.check_output(o, ref, tol)


def test_tree_scale_and_clamped_lengths():
    r, q, kc, vc, s, kcb, vcb = case(0, 3, 4, 2, 5, 300, seed=9)
    masks = tree_masks(r, 3, 5, "tree")
    o, err = gpu_tree(0, q, masks, kc, vc, s, kcb, vcb, [400, -2, 77], 300, scale=0.05, max_seq_len=250)
    ref, _, tol = R.attend(q, kc, vc, kcb, vcb, s, [250, 0, 77], visible_of(masks, 5), scale=0.05)
    R.check_output(o, ref, tol)
    assert err == _lib.VQKV_DEVERR_SEQ_LEN


def test_tree_bad_block_ids_are_reported():
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(0, 1, 4, 1, 4, 128, seed=2)
    bufs = [H.pack_cache_role(0, 0, kc, 128), H.pack_cache_role(0, 1, vc, 128)]
    pools, kw = paged_args(r, 64, bufs, 1, 1, 0, 128)
    kw["block_table"] = H.dev(np.array([[kw["num_blocks"], -5]], dtype=np.int32))
    ws = _lib.decode_tree_workspace(0, 1, 4, 1, 4, 128, 128)
    out = t.zeros((1, 4, 4, 128), dtype=t.float16, device="cuda")
    _lib.vqkv_decode_attn_tree(0, H.dev(q), H.dev(tree_masks(r, 1, 4, "chain").view(np.int64)), pools[0], pools[1],
                               H.dev(np.array([128], dtype=np.int32)), H.dev(kcb), H.dev(vcb), H.dev(s), out, ws, 128, 128,
                               **kw)
    assert int(ws[:4].view(t.int32).item()) == _lib.VQKV_DEVERR_BLOCK
    assert t.isfinite(out).all()


def test_tree_chain_equals_causal_queries():
    """A chain's masks give the visibility of vqkv_decode_attn_multi."""
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(0, 2, 8, 2, 6, 512, seed=21)
    lens = [511, 3]
    o, _ = gpu_tree(0, q, tree_masks(r, 2, 6, "chain"), kc, vc, s, kcb, vcb, lens, 512)
    out = t.zeros((2, 6, 8, 128), dtype=t.float16, device="cuda")
    ws = _lib.decode_workspace(0, 2, 8, 2, 512, 512, n_queries=6)
    _lib.vqkv_decode_attn_multi(0, H.dev(q), H.dev(H.pack_cache_role(0, 0, kc, 512)), H.dev(H.pack_cache_role(0, 1, vc, 512)),
                                H.dev(np.array(lens, dtype=np.int32)), H.dev(kcb), H.dev(vcb), H.dev(s), out, ws, 512, 512)
    a, c = o.astype(np.float64), out.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(a - c) <= 4e-3 * np.linalg.norm(c)     # each within 2e-3 of the definition
    assert np.array_equal(a[1, :3], c[1, :3])                    # zero rows: queries before position 0


def test_tree_graphs_streams_and_unaligned_output():
    """Two captured graphs with a workspace each, replayed on two streams; an output that is only 2-byte aligned."""
    t = H.torch()
    r, q, kc, vc, s, kcb, vcb = case(0, 2, 8, 2, 7, 700, seed=33)
    masks = tree_masks(r, 2, 7, "tree")
    lens = [700, 444]
    want, _ = gpu_tree(0, q, masks, kc, vc, s, kcb, vcb, lens, 700)
    dq, dm = H.dev(q), H.dev(masks.view(np.int64))
    bufs = [H.dev(H.pack_cache_role(0, role, c, 700)) for role, c in ((0, kc), (1, vc))]
    dl, dk, dv, ds = H.dev(np.array(lens, dtype=np.int32)), H.dev(kcb), H.dev(vcb), H.dev(s)
    jobs = []
    for i in range(2):
        raw = t.zeros(2 * 7 * 8 * 128 + 1, dtype=t.float16, device="cuda")
        out = raw[i:i + 2 * 7 * 8 * 128].view(2, 7, 8, 128)
        ws = _lib.decode_tree_workspace(0, 2, 8, 2, 7, 700, 700, num_splits=i + 1)
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        args = (0, dq, dm, bufs[0], bufs[1], dl, dk, dv, ds, out, ws, 700, 700)
        with t.cuda.stream(side):
            _lib.vqkv_decode_attn_tree(*args, num_splits=i + 1)
        side.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            _lib.vqkv_decode_attn_tree(*args, num_splits=i + 1)
        jobs.append((g, side, out))
    for _, _, out in jobs:
        out.zero_()
    t.cuda.synchronize()
    for _ in range(3):
        for g, side, _ in jobs:
            with t.cuda.stream(side):
                g.replay()
    t.cuda.synchronize()
    for _, _, out in jobs:
        d = out.cpu().numpy().astype(np.float64) - want
        assert np.linalg.norm(d) <= 1e-3 * np.linalg.norm(want)   # other splits: the fp16 roundings of P differ
