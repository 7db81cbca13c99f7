"""Cache editing through the C ABI: vqkv_evict_select against a sorted
selection and vqkv_cache_compact against a token-by-token copy, byte for byte
over the whole cache."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import helpers as H
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# ---------------------------------------------------------------- selection

def ref_select(mass, lens, n_keep, n_sink, n_recent):
    """keep rows (lists) by a stable sort: protected, then larger mass (NaN last), then lower position."""
    B, Hkv, _ = mass.shape
    out = [[None] * Hkv for _ in range(B)]
    for b in range(B):
        L = int(lens[b])
        for h in range(Hkv):
            def rank(t):
                x = float(mass[b, h, t])
                if t < n_sink or t >= L - n_recent:
                    return (0, 0.0, t)
                return (2, 0.0, t) if np.isnan(x) else (1, -x + 0.0, t)
            out[b][h] = sorted(sorted(range(L), key=rank)[:min(L, n_keep)])
    return out


def run_select(mass, lens, n_keep, n_sink, n_recent, max_seq_len=None):
    t = H.torch()
    B, Hkv, cap = mass.shape
    keep = t.full((B, Hkv, n_keep), -7, dtype=t.int32, device="cuda")
    kl = t.full((B,), -7, dtype=t.int32, device="cuda")
    err = t.zeros(1, dtype=t.int32, device="cuda")
    _lib.vqkv_evict_select(H.dev(mass), H.dev(np.asarray(lens, dtype=np.int32)), keep, kl, n_sink, n_recent,
                           max_seq_len, err)
    t.cuda.synchronize()
    return keep.cpu().numpy(), kl.cpu().numpy(), int(err.item())


def check_select(mass, lens, n_keep, n_sink, n_recent):
    keep, kl, err = run_select(mass, lens, n_keep, n_sink, n_recent)
    ref = ref_select(mass, lens, n_keep, n_sink, n_recent)
    for b in range(mass.shape[0]):
        K = min(int(lens[b]), n_keep)
        assert kl[b] == K
        for h in range(mass.shape[1]):
            assert keep[b, h, :K].tolist() == ref[b][h], (b, h)
            assert (keep[b, h, K:] == -7).all()      # entries past the kept ones are not written
    assert err == 0


@pytest.mark.parametrize("B,Hkv,cap,lens,n_keep,n_sink,n_recent", [
    (1, 1, 1, [1], 1, 0, 0),
    (1, 2, 40, [33], 32, 0, 0),
    (2, 3, 100, [0, 77], 10, 2, 3),            # an empty sequence
    (3, 2, 515, [515, 10, 11], 10, 4, 6),      # only protected tokens fit
    (2, 1, 5000, [4097, 31], 1000, 0, 100),    # two CTAs per row
    (1, 3, 20001, [20001], 19999, 64, 1),      # four CTAs, almost everything kept
    (1, 1, 70001, [70001], 5, 0, 0),           # eight CTAs, odd row pitch
    (1, 2, 400003, [400001], 123457, 7, 4096),   # parts beyond the shared-memory keys: read again each pass
])
def test_select_against_sort(B, Hkv, cap, lens, n_keep, n_sink, n_recent):
    r = np.random.default_rng(cap + n_keep)
    mass = np.exp(2 * r.standard_normal((B, Hkv, cap))).astype(np.float32)
    mass[r.random(mass.shape) < 0.2] = 0.0
    check_select(mass, lens, n_keep, n_sink, n_recent)


@pytest.mark.parametrize("B,Hkv,cap,n_keep", [(1, 1, 21000, 7777), (40, 4, 9000, 100), (78, 1, 9001, 8990)])
def test_select_long_rows_of_few_values(B, Hkv, cap, n_keep):
    """More keys in the deciding bin than a warp lists; few rows (a cluster each) and many (one CTA each)."""
    r = np.random.default_rng(cap)
    mass = np.where(r.random((B, Hkv, cap)) < 0.97, 0.25, r.random((B, Hkv, cap))).astype(np.float32)
    check_select(mass, [cap - (b % 7) for b in range(B)], n_keep, 3, 5)


def test_select_many_rows_of_random_weights():
    r = np.random.default_rng(8)
    mass = np.exp(2 * r.standard_normal((60, 3, 6001))).astype(np.float32)
    check_select(mass, r.integers(0, 6002, size=60), 1500, 4, 64)


@pytest.mark.parametrize("n_keep", [1, 31, 32, 500, 1023])
def test_select_ties_take_the_lowest_position(n_keep):
    r = np.random.default_rng(n_keep)
    mass = r.integers(0, 3, size=(2, 2, 1024)).astype(np.float32)
    check_select(mass, [1024, 1000], n_keep, 0, 0)
    mass[:] = 1.0                                # all equal
    check_select(mass, [1024, 1000], n_keep, 0, 0)


@pytest.mark.parametrize("cap", [600, 9000])
def test_select_special_values(cap):
    r = np.random.default_rng(cap)
    mass = r.standard_normal((1, 2, cap)).astype(np.float32)     # negative weights too
    special = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, np.finfo(np.float32).max,
                        np.finfo(np.float32).min, -np.nan], dtype=np.float32)
    at = r.permutation(cap)[:cap // 3]
    mass[:, :, at] = special[r.integers(0, len(special), size=(1, 2, len(at)))]
    for n_keep in (1, cap // 10, cap // 2, cap - 5):
        check_select(mass, [cap], n_keep, 0, 0)


def test_select_clamps_lengths_and_reports():
    mass = np.random.default_rng(1).random((3, 1, 300), dtype=np.float32)
    keep, kl, err = run_select(mass, [-4, 500, 100], 50, 0, 0, max_seq_len=200)
    ref = ref_select(mass, [0, 200, 100], 50, 0, 0)
    assert kl.tolist() == [0, 50, 50] and err == _lib.VQKV_DEVERR_SEQ_LEN
    for b in (1, 2):
        assert keep[b, 0].tolist() == ref[b][0]


def test_select_is_repeatable_in_a_graph_on_another_stream():
    t = H.torch()
    r = np.random.default_rng(5)
    mass = H.dev(r.random((2, 4, 30000), dtype=np.float32))
    lens = H.dev(np.array([30000, 12345], dtype=np.int32))
    keep = t.zeros((2, 4, 4000), dtype=t.int32, device="cuda")
    kl = t.zeros(2, dtype=t.int32, device="cuda")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        _lib.vqkv_evict_select(mass, lens, keep, kl, 4, 100)
    side.synchronize()
    first = keep.clone()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        _lib.vqkv_evict_select(mass, lens, keep, kl, 4, 100)
    keep.zero_()
    g.replay()
    t.cuda.synchronize()
    assert t.equal(keep, first)


# ---------------------------------------------------------------- compaction

def ref_move(codes, L, start, count, src):
    """Token codes [T][J] after the move, the sources copied out first; bad sources leave their token."""
    out = codes.copy()
    for i in range(count):
        d, s = start + i, int(src[i])
        if d <= s < L:
            out[d] = codes[s]
    return out


def tile_cap(mode, cap):
    T = vo.TILE_TOKENS[mode]
    return (cap + T - 1) // T * T


def run_compact(mode, B, Hkv, cap, lens, src, counts, start, seed, page=0, with_mass=True):
    """Runs the call on random caches and checks every byte of the cache, the mass and the error word."""
    t = H.torch()
    r = np.random.default_rng(seed)
    E, d = vo.GEOMETRY[mode]
    full = tile_cap(mode, cap) if not page else (cap + page - 1) // page * page
    toks = [r.integers(0, E, size=(B, Hkv, full, 128 // d)) for _ in range(2)]
    streams = [np.stack([np.stack([vo.pack_stream_fast(toks[role][b, h], mode, role, full) for h in range(Hkv)])
                         for b in range(B)]) for role in (0, 1)]
    mass = r.random((B, Hkv, cap), dtype=np.float32)
    lens32 = np.asarray(lens, dtype=np.int32)
    kw = {}
    if page:
        per = full // page
        nblk = B * per + 2
        table = r.permutation(nblk)[:B * per].reshape(B, per).astype(np.int32)
        bb = vo.code_bytes(mode, page)
        pools = []
        for x in streams:
            pool = r.integers(0, 256, size=(nblk, Hkv, bb), dtype=np.uint8)
            for b in range(B):
                for i in range(per):
                    pool[table[b, i]] = x[b, :, i * bb:(i + 1) * bb]
            pools.append(pool)
        bufs, before = [H.dev(p) for p in pools], pools
        kw = {"block_table": H.dev(table), "block_tokens": page, "num_blocks": nblk}
    else:
        bufs = [H.dev(x) for x in streams]
    dmass = H.dev(mass) if with_mass else None
    err = t.zeros(1, dtype=t.int32, device="cuda")
    dstart = H.dev(np.asarray(start, dtype=np.int32)) if start is not None else None
    _lib.vqkv_cache_compact(mode, bufs[0], bufs[1], H.dev(lens32), H.dev(np.asarray(src, dtype=np.int32)),
                            H.dev(np.asarray(counts, dtype=np.int32)), cap, start=dstart, mass=dmass, error_flags=err,
                            **kw)
    t.cuda.synchronize()
    st = start if start is not None else [0] * B
    n_src = src.shape[2]
    for role in (0, 1):
        got = bufs[role].cpu().numpy()
        want = before[role].copy() if page else np.empty_like(streams[role])
        for b in range(B):
            n = min(max(int(counts[b]), 0), n_src, cap - st[b]) if 0 <= st[b] <= cap else 0
            for h in range(Hkv):
                row = src[b, h if src.shape[1] > 1 else 0]
                new = ref_move(toks[role][b, h], min(max(int(lens[b]), 0), cap), st[b], n, row)
                packed = vo.pack_stream_fast(new, mode, role, full)
                if page:
                    for i in range(full // page):
                        want[table[b, i], h] = packed[i * bb:(i + 1) * bb]
                else:
                    want[b, h] = packed
        assert np.array_equal(got, want), role
    if with_mass:
        want = mass.copy()
        for b in range(B):
            if not 0 <= st[b] <= cap:
                continue
            L = min(max(int(lens[b]), 0), cap)
            n = min(max(int(counts[b]), 0), n_src, cap - st[b])
            for h in range(Hkv):
                row = src[b, h if src.shape[1] > 1 else 0]
                want[b, h] = ref_move(mass[b, h][:, None], L, st[b], n, row)[:, 0]
                want[b, h, st[b] + n:L] = 0.0
        assert np.array_equal(dmass.cpu().numpy(), want)
    return int(err.item())


def kept(r, B, heads, lens, n):
    """Random ascending kept positions, the rest 0."""
    src = np.zeros((B, heads, n), dtype=np.int32)
    counts = np.array([min(n, int(L)) for L in lens], dtype=np.int32)
    for b in range(B):
        for h in range(heads):
            src[b, h, :counts[b]] = np.sort(r.permutation(int(lens[b]))[:counts[b]])
    return src, counts


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("page", [0, 64, 256])
def test_compact_random_kept_tokens(mode, page):
    r = np.random.default_rng(10 * mode + page)
    lens = [700, 1, 333]
    src, counts = kept(r, 3, 2, lens, 250)
    assert run_compact(mode, 3, 2, 701, lens, src, counts, None, seed=mode, page=page) == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_compact_many_rounds(mode):
    # one stream of a cluster, several rounds of 8 x 16 groups of 16 tokens; sources near their places
    r = np.random.default_rng(mode)
    L = 9001
    keep = np.sort(r.permutation(L)[:7500])
    src = keep[None, None].astype(np.int32)
    assert run_compact(mode, 1, 1, L, [L], src, [7500], None, seed=40 + mode) == 0


@pytest.mark.parametrize("mode,page", [(0, 0), (0, 256), (1, 0), (2, 0), (3, 64), (4, 0)])
def test_compact_rounds_of_the_largest_cluster(mode, page):
    # more kept tokens than the largest cluster moves in one round (16 x 16 warps x 4 groups of 16 tokens)
    r = np.random.default_rng(70 + mode)
    L, n = 70001, 60000
    src = np.sort(r.permutation(L)[:n])[None, None].astype(np.int32)
    assert run_compact(mode, 1, 1, L, [L], src, [n], None, seed=80 + mode, page=page) == 0


@pytest.mark.parametrize("mode", [0, 3])
def test_compact_unordered_sources_over_rounds(mode):
    # every source at or after its place, in any order, many read by several tokens
    r = np.random.default_rng(6)
    L, n = 52000, 50000
    src = np.minimum(np.arange(n) + r.integers(0, 2000, size=(1, 1, n)), L - 1).astype(np.int32)
    assert run_compact(mode, 1, 1, L, [L], src, [n], None, seed=9) == 0


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("page", [0, 128])
def test_compact_accepted_path_shared_by_heads(mode, page):
    # drafts at L - 9 .. L - 1; the accepted ones move to L - 9; starts inside 16-token groups
    lens = [200, 25, 9, 130]
    start = [L - 9 for L in lens]
    paths = [[0, 2, 5, 8], [1], [], [0, 1, 2, 3, 4, 5, 6, 7, 8]]
    src = np.zeros((4, 1, 9), dtype=np.int32)
    for b in range(4):
        src[b, 0, :len(paths[b])] = [start[b] + j for j in paths[b]]
    assert run_compact(mode, 4, 3, 211, lens, src, [len(x) for x in paths], start, seed=mode, page=page) == 0


@pytest.mark.parametrize("mode", [0, 4])
def test_compact_repeated_and_unordered_sources(mode):
    r = np.random.default_rng(3)
    L, n = 3000, 1200
    src = r.integers(np.arange(n), L, size=(1, 2, n)).astype(np.int32)   # any source at or after its place
    assert run_compact(mode, 1, 2, L, [L], src, [n], None, seed=7) == 0


def test_compact_twice_in_a_graph_and_on_another_stream():
    """Two calls back to back, the second on what the first left, directly on a side stream and replayed twice."""
    t = H.torch()
    r = np.random.default_rng(11)
    B, Hkv, cap, n1, n2 = 2, 2, 5008, 3500, 1700
    lens = [5001, 3777]
    toks = [r.integers(0, 256, size=(B, Hkv, cap, 32)) for _ in range(2)]
    packed = [np.stack([np.stack([vo.pack_stream_fast(toks[role][b, h], 0, role, cap) for h in range(Hkv)])
                        for b in range(B)]) for role in (0, 1)]
    mass = r.random((B, Hkv, cap), dtype=np.float32)
    src1, c1 = kept(r, B, Hkv, lens, n1)
    src2, c2 = kept(r, B, Hkv, c1, n2)
    full = [H.dev(x) for x in packed] + [H.dev(mass)]
    k, v, dm = [x.clone() for x in full]
    ints = [H.dev(np.asarray(x, dtype=np.int32)) for x in (lens, src1, c1, src2, c2)]
    err = t.zeros(1, dtype=t.int32, device="cuda")

    def restore():
        for x, y in zip((k, v, dm), full):
            x.copy_(y)

    def both():
        _lib.vqkv_cache_compact(0, k, v, ints[0], ints[1], ints[2], cap, mass=dm, error_flags=err)
        _lib.vqkv_cache_compact(0, k, v, ints[2], ints[3], ints[4], cap, mass=dm, error_flags=err)

    want, wmass = [x.copy() for x in packed], mass.copy()
    for b in range(B):
        for h in range(Hkv):
            for role in (0, 1):
                new = ref_move(toks[role][b, h], lens[b], 0, c1[b], src1[b, h])
                want[role][b, h] = vo.pack_stream_fast(ref_move(new, c1[b], 0, c2[b], src2[b, h]), 0, role, cap)
            m1 = ref_move(mass[b, h][:, None], lens[b], 0, c1[b], src1[b, h])[:, 0]
            m1[c1[b]:lens[b]] = 0.0
            m2 = ref_move(m1[:, None], c1[b], 0, c2[b], src2[b, h])[:, 0]
            m2[c2[b]:c1[b]] = 0.0
            wmass[b, h] = m2

    def check():
        assert np.array_equal(k.cpu().numpy(), want[0]) and np.array_equal(v.cpu().numpy(), want[1])
        assert np.array_equal(dm.cpu().numpy(), wmass) and int(err.item()) == 0

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        both()
    side.synchronize()
    check()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        both()
    for _ in range(2):
        restore()
        g.replay()
        t.cuda.synchronize()
        check()


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_compact_identity_and_no_mass(mode):
    src = np.tile(np.arange(100, dtype=np.int32), (2, 2, 1))
    assert run_compact(mode, 2, 2, 128, [100, 60], src, [100, 60], None, seed=1, with_mass=False) == 0


def test_compact_reports_bad_sources_and_leaves_their_tokens():
    src = np.tile(np.arange(20, 60, dtype=np.int32), (2, 2, 1))
    src[0, 0, 5] = 3          # before its place
    src[0, 1, 6] = 90         # at the length
    src[1, 0, 7] = -1
    src[1, 1, 8] = 2**31 - 1
    assert run_compact(0, 2, 2, 100, [90, 90], src, [40, 40], None, seed=2) == _lib.VQKV_DEVERR_POSITION


def test_compact_clamps_lengths_counts_and_starts():
    P, S = _lib.VQKV_DEVERR_POSITION, _lib.VQKV_DEVERR_SEQ_LEN
    src = np.tile(np.arange(30, 70, dtype=np.int32), (1, 1, 1))
    assert run_compact(0, 1, 1, 100, [130], src, [99], None, seed=3) == S     # length past the capacity, count past n_src
    assert run_compact(0, 1, 1, 100, [90], src, [-3], None, seed=4) == 0      # nothing moves, the mass is cleared
    assert run_compact(0, 1, 1, 100, [90], src, [40], [-1], seed=5) == P      # nothing changes
    assert run_compact(0, 1, 1, 100, [90], src, [40], [101], seed=6) == P
    tail = np.full((1, 1, 8), 99, dtype=np.int32)
    assert run_compact(0, 1, 1, 100, [100], tail, [8], [96], seed=7) == P     # destinations past the capacity
    assert run_compact(0, 1, 1, 100, [0], src, [5], None, seed=8) == P        # an empty sequence has no sources


def test_compact_without_sources_clears_the_mass():
    t = H.torch()
    k = t.zeros((1, 1, 512), dtype=t.uint8, device="cuda")
    mass = t.ones((1, 1, 16), device="cuda")
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    _lib.vqkv_cache_compact(0, k, k.clone(), i32(12), t.zeros((1, 1, 0), dtype=t.int32, device="cuda"), i32(0), 16,
                            start=i32(5), mass=mass)
    assert mass.flatten().tolist() == [1.0] * 5 + [0.0] * 7 + [1.0] * 4


def test_compact_bad_block_ids_are_reported_and_skipped():
    t = H.torch()
    mode, page = 0, 64
    r = np.random.default_rng(11)
    bb = vo.code_bytes(mode, page)
    pool = r.integers(0, 256, size=(5, 1, bb), dtype=np.uint8)
    k, v = H.dev(pool), H.dev(pool)
    table = np.array([[2, 9, 3, -1]], dtype=np.int32)      # blocks 1 and 3 of the sequence are not in the pool
    src = np.concatenate([np.arange(64, 80), np.arange(128, 144)]).astype(np.int32)[None, None]
    err = t.zeros(1, dtype=t.int32, device="cuda")
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    _lib.vqkv_cache_compact(mode, k, v, i32(256), H.dev(src), i32(32), 256, error_flags=err, block_table=H.dev(table),
                            block_tokens=page, num_blocks=5)
    assert int(err.item()) == _lib.VQKV_DEVERR_BLOCK
    for role, buf in ((0, k), (1, v)):
        got = buf.cpu().numpy()
        want = pool.copy()
        tok = vo.unpack_stream_fast(pool[2, 0], mode, role, page)
        new = tok.copy()
        new[16:32] = vo.unpack_stream_fast(pool[3, 0], mode, role, page)[:16]   # 128.. sit in pool block 3
        want[2, 0] = vo.pack_stream_fast(new, mode, role, page)
        assert np.array_equal(got, want)


def test_binding_refuses_wrong_tensors():
    t = H.torch()
    k = t.zeros((1, 2, 512), dtype=t.uint8, device="cuda")
    i32 = lambda *shape: t.zeros(shape, dtype=t.int32, device="cuda")   # noqa: E731
    mass = t.zeros((1, 2, 16), device="cuda")
    with pytest.raises(TypeError):
        _lib.vqkv_cache_compact(0, k, k, i32(1), i32(1, 2, 4).long(), i32(1), 16)
    with pytest.raises(ValueError):
        _lib.vqkv_cache_compact(0, k, k, i32(1), i32(1, 2, 8)[:, :, ::2], i32(1), 16)
    with pytest.raises(ValueError):
        _lib.vqkv_cache_compact(0, k, k, i32(1), i32(1, 2, 4), i32(1), 64)        # capacity and codes disagree
    with pytest.raises(ValueError):
        _lib.vqkv_evict_select(mass, i32(1).cpu(), i32(1, 2, 4), i32(1))
    with pytest.raises(TypeError):
        _lib.vqkv_evict_select(mass.half(), i32(1), i32(1, 2, 4), i32(1))
    with pytest.raises(_lib.VqkvError):
        _lib.vqkv_evict_select(mass, i32(1), i32(1, 2, 4), i32(1), n_sink=3, n_recent=2)
