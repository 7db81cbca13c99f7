"""Cross attention (vqkv_cross_attn) through the C ABI against a plain fp64
attention over all cached tokens."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import attn_reference as R
from tests import helpers as H
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


class Cross:
    def __init__(self, t, mode, Hq, Hkv, queries, lens, cap=None, dt="fp16", block_tokens=0, seed=0, front=0, back=0, stride=0,
                 qscale=1.0):
        r = np.random.default_rng(seed)
        E, d = vo.GEOMETRY[mode]
        self.t, self.mode, self.Hq, self.Hkv, self.queries, self.lens = t, mode, Hq, Hkv, queries, lens
        B = len(queries)
        self.cap = cap = cap or max(max(lens), 1)
        if block_tokens:
            cap = self.cap = -(-cap // block_tokens) * block_tokens
        self.s, self.kcb, self.vcb = H.random_codebooks(mode, Hkv, seed + 1)
        self.kc = [[r.integers(0, E, size=(cap, 128 // d)) for _ in range(Hkv)] for _ in range(B)]
        self.vc = [[r.integers(0, E, size=(cap, 128 // d)) for _ in range(Hkv)] for _ in range(B)]
        n = front + sum(queries) + back
        self.starts = front + np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
        dtype = t.float16 if dt == "fp16" else t.bfloat16
        q = t.from_numpy((qscale * r.standard_normal((n, Hq, 128))).astype(np.float32)).cuda().to(dtype)
        self.q = q
        if stride:
            buf = t.full((n, Hq * 128 + stride), float("nan"), dtype=dtype, device="cuda")
            buf[:, :Hq * 128] = q.view(n, -1)
            self.q = buf[:, :Hq * 128].unflatten(1, (Hq, 128))
        self.out = t.full((n, Hq, 128), 3.0, dtype=dtype, device="cuda")
        self.dt, self.dtype = dt, dtype
        self.extra = {}
        bufs = [H.pack_cache_role(mode, role, c, cap) for role, c in ((0, self.kc), (1, self.vc))]
        if block_tokens:
            per, bb = cap // block_tokens, vo.code_bytes(mode, block_tokens)
            nblk = B * per + 3
            table = r.permutation(nblk)[:B * per].reshape(B, per).astype(np.int32)
            pools = []
            for x in bufs:
                pool = r.integers(0, 256, size=(nblk, Hkv, bb), dtype=np.uint8)
                for b in range(B):
                    for i in range(per):
                        pool[table[b, i]] = x[b][:, i * bb:(i + 1) * bb]
                pools.append(pool)
            bufs = pools
            self.extra = dict(block_table=H.dev(table), block_tokens=block_tokens, num_blocks=nblk)
        self.k, self.v = (H.dev(x) for x in bufs)
        self.books = (H.dev(self.kcb), H.dev(self.vcb), H.dev(self.s))
        self.dstarts, self.dlens = H.dev(self.starts), H.dev(np.asarray(lens, dtype=np.int32))
        self.most = max(max(queries), 1)
        self.ws = None

    def workspace(self, num_splits=0, max_seq_len=None, most=None):
        return _lib.cross_attn_workspace(self.mode, len(self.queries), self.Hq, self.Hkv, self.q.shape[0], most or self.most, self.cap,
                                         self.cap if max_seq_len is None else max_seq_len, num_splits,
                                         dtype=0 if self.dt == "fp16" else 2)

    def run(self, num_splits=0, scale=0.0, max_seq_len=None, most=None, out=None, ws=None, stream=None):
        self.ws = ws if ws is not None else self.workspace(num_splits, max_seq_len, most)
        out = self.out if out is None else out
        _lib.vqkv_cross_attn(self.mode, self.q, self.dstarts, self.k, self.v, self.dlens, *self.books, out, self.ws, self.cap,
                             self.cap if max_seq_len is None else max_seq_len, most or self.most, softmax_scale=scale,
                             num_splits=num_splits, stream=stream, **self.extra)
        return out

    def flags(self):
        return int(self.ws.view(self.t.int32)[0])

    def reference(self, scale=None, lens=None):
        """(O, bound) of every row; NaN rows for those that no sequence has."""
        n = self.q.shape[0]
        ref, tol = np.full((n, self.Hq, 128), np.nan), np.zeros((n, self.Hq, 128))
        q = self.q.double().cpu().numpy()
        for b, L in enumerate(self.lens if lens is None else lens):
            lo, hi = self.starts[b], self.starts[b + 1]
            if hi > lo:
                o, _, e = R.attend(q[None, lo:hi], [self.kc[b]], [self.vc[b]], self.kcb, self.vcb, self.s, [L],
                                   lambda *_: np.ones(L, dtype=bool), scale)
                if self.dt == "bf16":
                    e = e + 2.0 ** -8 * (np.abs(o) + e)
                ref[lo:hi], tol[lo:hi] = o[0], e[0]
        return ref, tol

    def check(self, got, ref, tol):
        got = got.double().cpu().numpy()
        mine = ~np.isnan(ref)
        assert (np.abs(got - ref)[mine] <= tol[mine]).all(), float(np.nanmax(np.abs(got - ref) - tol))
        norm = np.linalg.norm(ref[mine])
        # rms of the roundings, as in attn_reference.check_output; a bf16 result is eight times as coarse
        if norm > 0:
            assert np.linalg.norm((got - ref)[mine]) <= (2e-3 if self.dt == "fp16" else 4e-3) * norm
        assert (got[~mine] == 3.0).all()     # rows of no sequence


CASES = [
    # mode, Hq, Hkv, queries, lens, options; columns: queries x Hq / Hkv
    (0, 4, 4, [1], [1], dict()),
    (0, 8, 2, [1, 1, 1], [65, 0, 700], dict(back=2)),                                    # one token each, one cache empty
    (1, 10, 2, [1, 0, 3], [300, 50, 64], dict(block_tokens=64)),
    (2, 8, 8, [7, 64, 1], [63, 129, 1], dict(front=1, stride=64)),                       # pairs, 64 columns
    (3, 4, 2, [33, 5], [500, 1000], dict()),                                             # 66 columns: one tile
    (4, 16, 2, [16, 1], [640, 64], dict(block_tokens=128)),                              # 128 columns
    (0, 8, 1, [17, 40, 0, 3], [200, 333, 10, 0], dict(block_tokens=64, back=1)),         # 320 columns: two items
    (1, 2, 2, [129, 300], [257, 64], dict()),
    (2, 6, 2, [90, 1], [130, 900], dict(dt="bf16", stride=8)),
    (3, 5, 1, [52], [777], dict(block_tokens=256)),
    (4, 8, 8, [260, 2], [100, 300], dict(dt="bf16")),
    (0, 8, 4, [5, 1, 2], [90, 64, 3], dict(dt="bf16", front=2, back=3)),
    (0, 1, 1, [600], [1], dict()),                                                       # one token: its value
]


@pytest.mark.parametrize("mode,Hq,Hkv,queries,lens,kw", CASES)
@pytest.mark.parametrize("num_splits", [0, 1, 5])
def test_cross(t, mode, Hq, Hkv, queries, lens, kw, num_splits):
    x = Cross(t, mode, Hq, Hkv, queries, lens, seed=len(queries) + Hq, **kw)
    got = x.run(num_splits)
    x.check(got, *x.reference())
    assert x.flags() == 0
    again = x.run(num_splits, out=t.full_like(x.out, 3.0), ws=x.ws)
    assert t.equal(got, again)                                                           # the same bits, the workspace reused


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("block_tokens", [0, 64])
@pytest.mark.parametrize("queries", [[9, 2], [30, 61], [65, 200]])
def test_every_instance(t, mode, block_tokens, queries):
    x = Cross(t, mode, 4, 2, queries, [400, 210], block_tokens=block_tokens, seed=mode)
    x.check(x.run(), *x.reference())
    assert x.flags() == 0


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,queries,lens,kw", [
    (3, 3, [1], [700], dict()),                                                          # one sequence: the split plan
    (4, 2, [1, 0, 1, 1], [130, 300, 0, 1], dict(back=3, front=1)),                       # without a query, without tokens
    (16, 2, [0, 1, 1], [200, 64, 1000], dict(block_tokens=64, stride=32)),               # eight columns: two groups
    (5, 1, [1, 1], [65, 48], dict(block_tokens=128)),
])
@pytest.mark.parametrize("num_splits", [0, 3])
def test_single_queries(t, mode, dt, Hq, Hkv, queries, lens, kw, num_splits):
    x = Cross(t, mode, Hq, Hkv, queries, lens, dt=dt, seed=mode + Hq, **kw)
    got = x.run(num_splits)
    x.check(got, *x.reference())
    assert x.flags() == 0
    again = x.run(num_splits, out=t.full_like(x.out, 3.0), ws=x.ws)
    assert t.equal(got, again)


def test_single_queries_and_starts_that_make_no_sense(t):
    for mode in (0, 1):
        x = Cross(t, mode, 4, 2, [1, 1, 1], [100, 70, 90], seed=6)
        x.dstarts = H.dev(np.array([0, 1, -7, 3], dtype=np.int32))
        got = x.run()
        assert x.flags() == _lib.VQKV_DEVERR_SEQ_LEN
        ref, tol = x.reference()
        ref[1:] = np.nan
        x.check(got, ref, tol)
        x = Cross(t, mode, 4, 2, [2, 1], [100, 70], seed=6)      # two queries where one was announced
        got = x.run(most=1)
        assert x.flags() == _lib.VQKV_DEVERR_SEQ_LEN
        ref, tol = x.reference()
        ref[1] = np.nan
        x.check(got, ref, tol)


def test_many_single_queries(t):
    """More sequences than the flat plan takes."""
    r = np.random.default_rng(21)
    x = Cross(t, 0, 2, 1, r.integers(0, 2, 1100).tolist(), r.integers(0, 70, 1100).tolist(), cap=80, seed=13, dt="bf16")
    x.check(x.run(), *x.reference())
    assert x.flags() == 0


def test_scale_and_large_scores(t):
    for qscale, scale in ((1.0, 0.5), (12.0, 0.0), (1e-3, 0.0)):
        x = Cross(t, 0, 8, 2, [20, 70], [300, 500], seed=3, qscale=qscale)
        x.check(x.run(scale=scale), *x.reference(scale or None))


def test_equals_the_decode_of_single_tokens(t):
    x = Cross(t, 2, 8, 2, [1, 1, 1], [900, 64, 333], seed=8)
    got = x.run()
    ws = _lib.decode_workspace(2, 3, 8, 2, x.cap, x.cap)
    out = t.empty_like(x.out)
    _lib.vqkv_decode_attn(2, x.q, x.k, x.v, x.dlens, *x.books, out, ws, x.cap, x.cap)
    ref, tol = x.reference()
    assert (np.abs((got.double() - out.double()).cpu().numpy()) <= 2 * tol).all()


def test_lengths_outside_the_range_are_clamped(t):
    x = Cross(t, 0, 4, 2, [3, 40, 2], [100, 128, 50], cap=128, seed=4)
    x.dlens = H.dev(np.array([100, 4000, -7], dtype=np.int32))
    got = x.run(max_seq_len=110)
    x.check(got, *x.reference(lens=[100, 110, 0]))
    assert x.flags() == _lib.VQKV_DEVERR_SEQ_LEN
    assert not got[x.starts[2]:x.starts[3]].any()                                        # nothing to see: zero rows


def test_more_queries_than_announced(t):
    """Rows of a sequence beyond max_queries stay as they are, and the bit says so."""
    x = Cross(t, 0, 4, 2, [10, 3], [100, 70], seed=5)
    got = x.run(most=6)
    ref, tol = x.reference()
    ref[6:10] = np.nan
    x.check(got, ref, tol)
    assert x.flags() == _lib.VQKV_DEVERR_SEQ_LEN


@pytest.mark.parametrize("starts", [[0, 40, 9], [-1, 4, 9], [0, 4, 1000], [9, 4, 4], [2**31 - 1, -2**31, 5]])
def test_starts_that_make_no_sense(t, starts):
    """A sequence whose starts do not ascend within the rows has no queries; the others are computed."""
    x = Cross(t, 1, 4, 2, [4, 5], [100, 70], seed=6)
    x.dstarts = H.dev(np.array(starts, dtype=np.int64).astype(np.int32))
    got = x.run(most=50)
    assert x.flags() == _lib.VQKV_DEVERR_SEQ_LEN
    fine = [0 <= a <= b <= 9 for a, b in zip(starts, starts[1:])]
    x.starts = np.array([4, 4, 9]) if fine == [False, True] and starts[1:] == [4, 9] else np.array([0, 4, 4]) if fine[0] else np.array([0, 0, 0])
    x.check(got, *x.reference())


def test_in_place(t):
    x = Cross(t, 3, 8, 2, [30, 1, 20], [300, 0, 77], seed=7)
    want = x.run().clone()
    q = x.q.clone()
    x.q = q
    got = x.run(out=q)
    assert t.equal(got, want)


def test_more_sequences_than_a_launch_takes(t):
    """1,100 sequences of a few tokens, some without queries, some without tokens."""
    r = np.random.default_rng(11)
    queries, lens = r.integers(0, 4, 1100).tolist(), r.integers(0, 70, 1100).tolist()
    x = Cross(t, 0, 2, 1, queries, lens, cap=80, seed=12, back=4)
    x.check(x.run(), *x.reference())
    assert x.flags() == 0


def test_captured_graphs_and_streams(t):
    """Two captured calls with a workspace each, replayed on two streams at once, and a workspace shared in order."""
    a, b = Cross(t, 0, 8, 2, [3, 70], [500, 300], seed=1), Cross(t, 4, 8, 2, [200], [700], seed=2, dt="bf16")
    want = [x.run().clone() for x in (a, b)]
    graphs = []
    for x in (a, b):
        x.out.zero_()
        ws = x.workspace()
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            x.run(ws=ws)
        graphs.append(g)
    streams = [t.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        a.out.zero_(), b.out.zero_()
        t.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with t.cuda.stream(s):
                g.replay()
        t.cuda.synchronize()
        assert t.equal(a.out, want[0]) and t.equal(b.out, want[1])


def test_workspace_shared_with_decode_and_trees(t):
    """The decode's merge tickets in a shared workspace stay zero."""
    x = Cross(t, 0, 8, 2, [1, 1], [1000, 999], seed=3)
    one = _lib.decode_workspace(0, 2, 8, 2, x.cap, x.cap)
    ws = t.zeros(max(one.numel(), x.workspace().numel()), dtype=t.uint8, device="cuda")
    decode = lambda out: _lib.vqkv_decode_attn(0, x.q, x.k, x.v, x.dlens, *x.books, out, ws, x.cap, x.cap)  # noqa: E731
    first, second = t.empty_like(x.out), t.empty_like(x.out)
    decode(first)
    want = x.run(ws=ws).clone()
    decode(second)
    assert t.equal(first, second) and t.equal(x.run(ws=ws), want)


def test_blocks_outside_the_pool_are_flagged(t):
    x = Cross(t, 0, 4, 2, [3, 70], [128, 100], block_tokens=64, seed=9)
    x.extra["block_table"][0, 1], x.extra["block_table"][1, 0] = x.extra["num_blocks"], -1
    x.run()
    assert x.flags() == _lib.VQKV_DEVERR_BLOCK


def test_refused_by_the_binding(t):
    x = Cross(t, 0, 4, 2, [3, 2], [60, 64], seed=9)
    ws = x.workspace()
    kw = dict(mode=0, q=x.q, row_start=x.dstarts, k_codes=x.k, v_codes=x.v, seq_lens=x.dlens, k_codebook=x.books[0],
              v_codebook=x.books[1], s=x.books[2], out=x.out, workspace=ws, cap_len=64, max_seq_len=64, max_queries=3)
    for bad, kind in ((dict(q=x.q.float()), TypeError), (dict(out=x.out.bfloat16()), TypeError), (dict(out=x.out[:4]), ValueError),
                      (dict(row_start=x.dstarts[:2]), ValueError), (dict(row_start=x.dstarts.long()), TypeError),
                      (dict(q=x.q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError), (dict(q=x.q[:, :, :64]), ValueError),
                      (dict(q=t.cat([x.q, x.q], 1)[:, ::2]), ValueError), (dict(workspace=ws[:256]), _lib.VqkvError),
                      (dict(max_queries=0), _lib.VqkvError), (dict(out=x.out.cpu()), ValueError), (dict(max_seq_len=65), _lib.VqkvError),
                      (dict(k_codes=x.k[:1]), ValueError)):
        with pytest.raises(kind):
            _lib.vqkv_cross_attn(**{**kw, **bad})
    with pytest.raises(_lib.VqkvError):
        _lib.cross_attn_workspace(0, 2, 5, 2, 10, 3, 64, 64)
