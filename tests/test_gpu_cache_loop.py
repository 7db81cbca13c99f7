"""The cache-editing calls together, as a serving loop uses them: draft trees
verified, their accepted paths kept, and caches cut by accumulated weight,
with the library's encode and decode calls around them."""
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


class Cache:
    """A packed cache on the GPU, contiguous or paged, and what its calls need."""

    def __init__(self, mode, B, Hkv, cap, page, seed):
        t = H.torch()
        self.mode, self.B, self.Hkv, self.cap, self.page = mode, B, Hkv, cap, page
        self.r = np.random.default_rng(seed)
        self.s, self.kcb, self.vcb = H.random_codebooks(mode, Hkv, seed + 1)
        self.ds, self.dk, self.dv = H.dev(self.s), H.dev(self.kcb), H.dev(self.vcb)
        self.kw = {}
        shape = (B, Hkv, vo.code_bytes(mode, cap))
        if page:
            per = cap // page
            n = B * per + 1
            self.table = self.r.permutation(n)[:B * per].reshape(B, per).astype(np.int32)
            shape = (n, Hkv, vo.code_bytes(mode, page))
            self.kw = {"block_table": H.dev(self.table), "block_tokens": page, "num_blocks": n}
        self.k, self.v = (t.zeros(shape, dtype=t.uint8, device="cuda") for _ in range(2))

    def encode(self, k, v, pos):
        """fp16 rows [B][Hkv][n][128] at positions pos[b] .."""
        p = H.dev(np.asarray(pos, dtype=np.int32))
        for role, x, s, cb, buf in ((0, k, self.ds, self.dk, self.k), (1, v, None, self.dv, self.v)):
            if self.page:
                _lib.vqkv_encode_paged(self.mode, role, H.dev(x), p, s, cb, buf, self.cap, self.kw["block_table"],
                                       self.page, self.kw["num_blocks"])
            else:
                _lib.vqkv_encode(self.mode, role, H.dev(x), p, s, cb, buf, self.cap)

    def codes(self, b, h, n):
        """The codes of the first n tokens of a stream pair, read back."""
        out = []
        for role, buf in ((0, self.k), (1, self.v)):
            x = buf.cpu().numpy()
            stream = np.concatenate([x[i, h] for i in self.table[b]]) if self.page else x[b, h]
            out.append(vo.unpack_stream_fast(stream, self.mode, role, n))
        return out

    def all_codes(self, lens):
        both = [[self.codes(b, h, int(lens[b])) for h in range(self.Hkv)] for b in range(self.B)]
        return [[[both[b][h][i] for h in range(self.Hkv)] for b in range(self.B)] for i in (0, 1)]


def rows(r, B, Hkv, n):
    return r.standard_normal((B, Hkv, n, 128)).astype(np.float16)


@pytest.mark.parametrize("mode,page", [(0, 0), (0, 64), (1, 0), (2, 64), (3, 0), (4, 64)])
def test_speculative_steps_leave_the_cache_of_the_accepted_tokens(mode, page):
    t = H.torch()
    B, Hkv, g, M, cap = 2, 2, 4, 7, 256
    c = Cache(mode, B, Hkv, cap, page, seed=3 + mode)
    plain = Cache(mode, B, Hkv, cap, 0, seed=3 + mode)        # the same codebooks: accepted tokens only
    lens = np.array([61, 90])
    k0, v0 = rows(c.r, B, Hkv, 90), rows(c.r, B, Hkv, 90)
    for x in (c, plain):
        x.encode(k0, v0, [0, 0])
    ws = _lib.decode_tree_workspace(mode, B, Hkv * g, Hkv, M, cap, cap)
    out = t.zeros((B, M, Hkv * g, 128), dtype=t.float16, device="cuda")
    for step in range(4):
        kd, vd, q = rows(c.r, B, Hkv, M), rows(c.r, B, Hkv, M), c.r.standard_normal((B, M, Hkv * g, 128)).astype(np.float16)
        parent = np.array([[-1] + [int(c.r.integers(0, m)) for m in range(1, M)] for _ in range(B)])
        mask = np.zeros((B, M), dtype=np.int64)
        for b in range(B):
            for m in range(M):
                mask[b, m] = (1 << m) | (mask[b, parent[b, m]] if m else 0)
        c.encode(kd, vd, lens)
        dl = H.dev((lens + M).astype(np.int32))
        _lib.vqkv_decode_attn_tree(mode, H.dev(q), H.dev(mask), c.k, c.v, dl, c.dk, c.dv, c.ds, out, ws, cap, cap, **c.kw)
        kc, vc = c.all_codes(lens + M)

        def visible(b, m, L):
            j = np.arange(L) - (L - M)
            return (j < 0) | (((int(mask[b, m]) >> np.clip(j, 0, 63)) & 1) == 1)
        ref, _, tol = R.attend(q, kc, vc, c.kcb, c.vcb, c.s, lens + M, visible)
        R.check_output(out.cpu().numpy(), ref, tol)
        # accept the ancestors of a random leaf
        src, counts, paths = np.zeros((B, 1, M), dtype=np.int32), np.zeros(B, dtype=np.int32), []
        for b in range(B):
            m, path = int(c.r.integers(0, M)), []
            while m >= 0:
                path.append(m)
                m = parent[b, m]
            path = path[::-1]
            paths.append(path)
            src[b, 0, :len(path)] = lens[b] + np.array(path)
            counts[b] = len(path)
        _lib.vqkv_cache_compact(mode, c.k, c.v, dl, H.dev(src), H.dev(counts), cap, start=H.dev(lens.astype(np.int32)), **c.kw)
        for b in range(B):   # the plain cache takes the accepted tokens one after another
            for i, m in enumerate(paths[b]):
                pos = np.full(B, cap, dtype=np.int32)          # other sequences: past the capacity, not written
                pos[b] = lens[b] + i
                plain.encode(kd[:, :, m:m + 1], vd[:, :, m:m + 1], pos)
        lens = lens + counts
        for b in range(B):
            for h in range(Hkv):
                for a, z in zip(c.codes(b, h, int(lens[b])), plain.codes(b, h, int(lens[b]))):
                    assert np.array_equal(a, z), (step, b, h)


@pytest.mark.parametrize("mode,page", [(0, 0), (0, 64), (1, 64), (2, 0), (3, 64), (4, 0)])
def test_eviction_by_accumulated_weight(mode, page):
    t = H.torch()
    B, Hkv, g, cap, keep, sink, recent = 2, 2, 4, 320, 96, 4, 16
    c = Cache(mode, B, Hkv, cap, page, seed=13 + mode)
    lens = np.array([240, 60])
    c.encode(rows(c.r, B, Hkv, 240), rows(c.r, B, Hkv, 240), [0, 0])
    mass = t.zeros((B, Hkv, cap), device="cuda")
    want = np.zeros((B, Hkv, cap))
    ws = {m: _lib.decode_mass_workspace(mode, B, Hkv * g, Hkv, m, cap, cap) for m in (1, 6)}
    # the prompt's last queries as an observation window, then single steps
    for M in (6, 1, 1, 1):
        if M == 1:
            c.encode(rows(c.r, B, Hkv, 1), rows(c.r, B, Hkv, 1), lens)
            lens = lens + 1
        q = c.r.standard_normal((B, M, Hkv * g, 128)).astype(np.float16)
        out = t.zeros((B, M, Hkv * g, 128), dtype=t.float16, device="cuda")
        dl = H.dev(lens.astype(np.int32))
        before = mass.cpu().numpy()
        _lib.vqkv_decode_attn_mass(mode, H.dev(q), c.k, c.v, dl, c.dk, c.dv, c.ds, out, mass, ws[M], cap, cap, **c.kw)
        kc, vc = c.all_codes(lens)
        ref, w, tol = R.attend(q, kc, vc, c.kcb, c.vcb, c.s, lens, lambda b, m, L: np.arange(L) <= L - M + m)
        R.check_output(out.cpu().numpy(), ref, tol)
        R.check_mass(mass.cpu().numpy(), before, w, lens, R.attend.score_size)
    got = mass.cpu().numpy()
    kept = t.full((B, Hkv, keep), -1, dtype=t.int32, device="cuda")
    kl = t.zeros(B, dtype=t.int32, device="cuda")
    _lib.vqkv_evict_select(mass, dl, kept, kl, n_sink=sink, n_recent=recent, max_seq_len=cap)
    _lib.vqkv_cache_compact(mode, c.k, c.v, dl, kept, kl, cap, mass=mass, **c.kw)
    new = kl.cpu().numpy()
    assert new.tolist() == [keep, 63]
    k, after = kept.cpu().numpy(), mass.cpu().numpy()
    new_k, new_v = c.all_codes(new)
    for b in range(B):
        for h in range(Hkv):
            i = k[b, h, :new[b]]
            L = int(lens[b])
            assert (np.diff(i) > 0).all() and set(range(min(sink, L))) <= set(i) and set(range(L - recent, L)) <= set(i)
            dropped = np.setdiff1d(np.arange(L), i)
            free = np.setdiff1d(i, np.r_[0:sink, L - recent:L])
            if len(dropped) and len(free):
                assert got[b, h, dropped].max() <= got[b, h, free].min()
            assert np.array_equal(new_k[b][h], kc[b][h][i]) and np.array_equal(new_v[b][h], vc[b][h][i])
            assert np.array_equal(after[b, h, :new[b]], got[b, h, i]) and not after[b, h, new[b]:L].any()
    # the next step appends behind the kept tokens and attends over them
    c.encode(rows(c.r, B, Hkv, 1), rows(c.r, B, Hkv, 1), new)
    q = c.r.standard_normal((B, 1, Hkv * g, 128)).astype(np.float16)
    before = mass.cpu().numpy()
    _lib.vqkv_decode_attn_mass(mode, H.dev(q), c.k, c.v, H.dev((new + 1).astype(np.int32)), c.dk, c.dv, c.ds,
                               out, mass, ws[1], cap, cap, **c.kw)
    kc, vc = c.all_codes(new + 1)
    ref, w, tol = R.attend(q, kc, vc, c.kcb, c.vcb, c.s, new + 1, lambda b, m, L: np.ones(L, dtype=bool))
    R.check_output(out.cpu().numpy(), ref, tol)
    R.check_mass(mass.cpu().numpy(), before, w, new + 1, R.attend.score_size)
    assert not before[:, :, int(new.max()):].any()      # new tokens start at 0
