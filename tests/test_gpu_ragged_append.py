"""Ragged append (vqkv_append) through the C ABI against the oracle's codes of
the fp64 rotation, and against vqkv_encode."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import helpers as H
from tests import rope_reference as R
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def _dtype(t, name):
    return {"fp16": t.float16, "bf16": t.bfloat16, "fp32": t.float32}[name]


class Batch:
    """Inputs of an append: B sequences with new[b] tokens at pos[b], `front` and `back` padding rows."""

    def __init__(self, t, mode, Hkv, new, pos, cap, dt="fp16", rot=128, interleaved=False, block_tokens=0, seed=0, front=0, back=0,
                 fused=False, shift=None):
        r = np.random.default_rng(seed)
        self.t, self.mode, self.Hkv, self.new, self.pos, self.cap = t, mode, Hkv, new, pos, cap
        self.block_tokens, self.interleaved, self.front = block_tokens, interleaved, front
        B, n = len(new), sum(new)
        T = front + n + back
        self.T, self.B = T, B
        scale = r.uniform(0.5, 3.0, size=(1, Hkv, 128))
        k, v = (r.standard_normal((T, Hkv, 128)) * scale).astype(np.float32), r.standard_normal((T, Hkv, 128)).astype(np.float32)
        for x in (k, v):
            x[:front], x[front + n:] = np.nan, np.nan     # padding is not read
        k, v = (t.from_numpy(x).cuda().to(_dtype(t, dt)) for x in (k, v))
        self.k, self.v = k, v
        if fused:     # slices of a wider buffer, heads first
            buf = t.full((T, 2 * Hkv + 3, 132), float("nan"), dtype=k.dtype, device="cuda")
            buf[:, 1:1 + Hkv, :128], buf[:, 2 + Hkv:2 + 2 * Hkv, :128] = k, v
            self.k, self.v = buf[:, 1:1 + Hkv, :128], buf[:, 2 + Hkv:2 + 2 * Hkv, :128]
        self.s, self.kcb, self.vcb = H.random_codebooks(mode, Hkv, seed + 1)
        self.starts = front + np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.at = np.concatenate([p + np.arange(m) for p, m in zip(pos, new)]) if n else np.zeros(0, dtype=int)
        self.table = self.rope_pos = None
        self.angles = self.at
        if rot:
            n_pos = cap + 1000
            self.table = t.empty((n_pos, rot), device="cuda")
            _lib.vqkv_rope_table(self.table)
            if shift is not None:
                self.angles = self.at + shift
                full = np.full(T, -5, dtype=np.int32)        # not read for padding
                full[front:front + n] = self.angles
                self.rope_pos = H.dev(full)
        self.blocks = None
        if block_tokens:
            per = -(-cap // block_tokens)
            self.num_blocks = B * per + 2
            self.blocks = r.permutation(self.num_blocks)[:B * per].reshape(B, per).astype(np.int32)
            shape = (self.num_blocks, Hkv, vo.code_bytes(mode, block_tokens))
        else:
            shape = (B, Hkv, vo.code_bytes(mode, cap))
        self.before = [r.integers(0, 256, size=shape, dtype=np.uint8) for _ in range(2)]
        self.codes = [H.dev(x) for x in self.before]
        self.err = t.zeros(1, dtype=t.int32, device="cuda")
        self.ties = t.zeros(1, dtype=t.int64, device="cuda")

    def paged(self):
        if self.blocks is None:
            return {}
        return dict(block_table=H.dev(self.blocks), block_tokens=self.block_tokens, num_blocks=self.num_blocks)

    def run(self, **kw):
        args = dict(rope_table=self.table, rope_pos=self.rope_pos, interleaved=self.interleaved, near_tie_count=self.ties,
                    error_flags=self.err, **self.paged())
        args.update(kw)
        _lib.vqkv_append(self.mode, self.k, self.v, H.dev(self.starts), H.dev(np.asarray(self.pos, dtype=np.int32)), H.dev(self.s),
                         H.dev(self.kcb), H.dev(self.vcb), self.codes[0], self.codes[1], self.cap, **args)
        self.t.cuda.synchronize()

    def stream(self, buf, b, h):
        if self.blocks is None:
            return buf[b, h]
        return np.concatenate([buf[i, h] for i in self.blocks[b]])

    def check(self, name, live=None, bounded=True):
        """Every token's codes against the oracle; every other token's codes (and block's bytes) as before."""
        n = len(self.at)
        live = np.ones(n, dtype=bool) if live is None else live
        rows = self.table.double().cpu().numpy()[np.clip(self.angles, 0, len(self.table) - 1)] if self.table is not None else None
        seq = np.repeat(np.arange(self.B), self.new)
        for role, x, cb in ((vo.ROLE_K, self.k, self.kcb), (vo.ROLE_V, self.v, self.vcb)):
            x = x[self.front:self.front + n].double().cpu().numpy()
            ref, d32 = R.append_codes(x, role, self.s, cb, rows, self.interleaved)
            got = self.codes[role].cpu().numpy()
            cap = self.cap if self.blocks is None else self.blocks.shape[1] * self.block_tokens
            for b in range(self.B):
                mine = np.flatnonzero((seq == b) & live)
                for h in range(self.Hkv):
                    new = vo.unpack_stream_fast(self.stream(got, b, h), self.mode, role, cap)
                    old = vo.unpack_stream_fast(self.stream(self.before[role], b, h), self.mode, role, cap)
                    if len(mine):
                        H.check_and_record_codes(f"{name}, mode {self.mode}, role {role}, ({b}, {h})", new[self.at[mine]], ref[mine, h],
                                                 d32[mine, h].reshape(-1, d32.shape[-1]), bounded=bounded)
                    other = np.ones(cap, dtype=bool)
                    other[self.at[mine]] = False
                    assert np.array_equal(new[other], old[other]), (b, h)
            if self.blocks is not None:
                free = np.setdiff1d(np.arange(self.num_blocks), self.blocks)
                assert np.array_equal(got[free], self.before[role][free])


CASES = [
    # new tokens, their positions, capacity, options
    ([1], [0], 64, dict()),                                                               # the first token of all
    ([1], [199], 200, dict(dt="bf16", fused=True)),                                       # the last place
    ([1, 1, 1], [5, 130, 63], 192, dict(block_tokens=64, shift=100)),                     # a decode step
    ([3, 0, 5, 0, 0, 2], [60, 0, 0, 9, 1, 125], 128, dict(rot=64, interleaved=True, back=3, fused=True)),
    ([0, 40, 1], [0, 100, 17], 256, dict(block_tokens=128, dt="bf16", front=2, back=1, rot=96)),
    ([33, 30], [0, 47], 128, dict(dt="fp32", shift=900, rot=120)),
    ([20, 31], [3, 64], 128, dict(rot=0, block_tokens=64)),                               # no rotation
]


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("new,pos,cap,kw", CASES)
@pytest.mark.parametrize("Hkv", [1, 3])
def test_codes(t, mode, Hkv, new, pos, cap, kw):
    b = Batch(t, mode, Hkv, new, pos, cap, seed=7 * mode + len(new), **kw)
    b.run()
    assert int(b.err) == 0
    b.check(f"ragged append {new}, Hkv {Hkv}")


@pytest.mark.parametrize("mode", range(5))
def test_many_rows_equal_single_ones(t, mode):
    """A ragged batch in one call (the many-row kernels) and token by token (the few-row ones): the same bytes."""
    new, pos = [97, 1, 0, 310, 53], [11, 500, 3, 0, 250]
    b = Batch(t, mode, 4, new, pos, 512, dt="bf16", block_tokens=64, seed=mode, rot=128, fused=True, back=5)
    b.run()
    whole = [x.clone() for x in b.codes]
    ties = int(b.ties)
    for x, old in zip(b.codes, b.before):
        x.copy_(H.dev(old))
    seq = np.repeat(np.arange(b.B), new)
    b.ties.zero_()
    k, v = b.k, b.v
    for i in range(0, len(seq), 4):     # up to four tokens of whatever sequences
        part = seq[i:i + 4]
        starts = np.searchsorted(part, np.arange(b.B + 1)).astype(np.int32)
        first = np.array([b.at[np.flatnonzero(seq == s)[0]] if (seq == s).any() else 0 for s in range(b.B)])
        done = np.array([(seq[:i] == s).sum() for s in range(b.B)])
        _lib.vqkv_append(mode, k[i:i + 4][:len(part)], v[i:i + 4][:len(part)], H.dev(starts), H.dev((first + done).astype(np.int32)),
                         H.dev(b.s), H.dev(b.kcb), H.dev(b.vcb), b.codes[0], b.codes[1], b.cap, rope_table=b.table,
                         near_tie_count=b.ties, error_flags=b.err, **b.paged())
    t.cuda.synchronize()
    assert int(b.err) == 0 and int(b.ties) == ties
    assert all(t.equal(x, y) for x, y in zip(whole, b.codes))


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("n", [2, 200])
def test_without_rotation_equals_encode(t, mode, n):
    b = Batch(t, mode, 2, [n, n], [5, 20], 256, rot=0, seed=50 + mode)
    b.run()
    for role, x, cb, s in ((0, b.k, b.kcb, b.s), (1, b.v, b.vcb, None)):
        codes = H.dev(b.before[role])
        rows = x.view(2, n, 2, 128).transpose(1, 2).contiguous()
        _lib.vqkv_encode(mode, role, rows, H.dev(np.array([5, 20], dtype=np.int32)), H.dev(s) if s is not None else None, H.dev(cb),
                         codes, 256)
        assert t.equal(codes, b.codes[role])


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("n", [3, 150])
def test_positions_out_of_range_are_skipped(t, mode, n):
    """Past the capacity, before position 0, and an angle outside the table: neither key nor value is written."""
    b = Batch(t, mode, 2, [n, n, n], [64 - n + 2, -1, 0], 64 if n == 3 else 160, seed=mode, shift=0)
    if n != 3:
        b.pos[0] = 100
        b.at = np.concatenate([p + np.arange(n) for p in b.pos])
        b.angles = b.at
    angles = b.angles.copy()
    angles[2 * n + 1], angles[2 * n + 2] = -1, len(b.table)
    b.rope_pos = H.dev(angles.astype(np.int32))
    b.run()
    assert int(b.err) == _lib.VQKV_DEVERR_POSITION
    ok = (b.at >= 0) & (b.at < b.cap) & (angles >= 0) & (angles < len(b.table))
    assert 0 < ok.sum() < len(ok)
    b.angles = angles
    b.at = np.where(ok, b.at, 0)
    b.check(f"positions out of range, {n}", live=ok)


def test_block_outside_the_pool(t):
    b = Batch(t, 0, 2, [70, 70], [0, 0], 128, block_tokens=64, seed=3)
    b.blocks[0, 1], b.blocks[1, 0] = b.num_blocks, -1
    good = [x.clone() for x in b.codes]
    b.run()
    assert int(b.err) == _lib.VQKV_DEVERR_BLOCK
    touched = {int(b.blocks[0, 0]), int(b.blocks[1, 1])}
    for x, y in zip(b.codes, good):
        changed = (x != y).flatten(1).any(dim=1).nonzero().flatten().tolist()
        assert set(changed) == touched


def test_angles_of_far_positions(t):
    """A table of 200,000 positions; keys there, and their codes, as the oracle's."""
    b = Batch(t, 0, 2, [5, 130], [10, 40], 192, seed=9, shift=199000)
    b.table = t.empty((200000, 128), device="cuda")
    _lib.vqkv_rope_table(b.table, base=500000.0)
    b.run()
    assert int(b.err) == 0
    b.check("far angles")


@pytest.mark.parametrize("mode", range(5))
def test_extreme_rows(t, mode):
    """Values beyond fp16 in fp32 and bf16 rows (an exhaustive search), zero rows, and equal centroids (the lowest wins)."""
    b = Batch(t, mode, 1, [4, 60], [0, 2], 64, dt="fp32", seed=20 + mode)
    b.k[0], b.v[1], b.k[10] = b.k[0] * 1e5, b.v[1] * 1e6, 0
    b.v[11] = 0
    b.kcb[:, 100:103] = b.kcb[:, 7:8]
    b.vcb[:, 200] = b.vcb[:, 8]
    b.run()
    b.check("extreme rows", bounded=False)


def test_captured_and_on_another_stream(t):
    b = Batch(t, 1, 2, [1, 1, 1, 1], [5, 6, 7, 300], 512, dt="bf16", block_tokens=64, seed=2)
    args = (b.mode, b.k, b.v, H.dev(b.starts), H.dev(np.asarray(b.pos, dtype=np.int32)), H.dev(b.s), H.dev(b.kcb), H.dev(b.vcb))
    paged = b.paged()
    want = [x.clone() for x in b.codes]
    _lib.vqkv_append(*args, *want, b.cap, rope_table=b.table, **paged)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        _lib.vqkv_append(*args, *b.codes, b.cap, rope_table=b.table, **paged)
    for _ in range(2):
        for x, old in zip(b.codes, b.before):
            x.copy_(H.dev(old))
        g.replay()
        assert all(t.equal(x, y) for x, y in zip(b.codes, want))
    for x, old in zip(b.codes, b.before):
        x.copy_(H.dev(old))
    s = t.cuda.Stream()
    t.cuda.synchronize()
    _lib.vqkv_append(*args, *b.codes, b.cap, rope_table=b.table, stream=s, **paged)
    s.synchronize()
    assert all(t.equal(x, y) for x, y in zip(b.codes, want))


def test_many_sequences(t):
    """1,500 sequences, most of them without new tokens: every token finds its own."""
    r = np.random.default_rng(5)
    new = (r.random(1500) < 0.3).astype(int) * r.integers(1, 3, 1500)
    new[0], new[-1] = 0, 2
    pos = r.integers(0, 60, 1500)
    b = Batch(t, 2, 1, new.tolist(), pos.tolist(), 64, seed=6, rot=32)
    b.run()
    assert int(b.err) == 0
    rows = b.table.double().cpu().numpy()[b.at]
    seq = np.repeat(np.arange(1500), new)
    got = b.codes[0].cpu().numpy()
    ref, d32 = R.append_codes(b.k.double().cpu().numpy(), 0, b.s, b.kcb, rows)
    new_codes = np.stack([vo.unpack_stream_fast(got[s, 0], 2, 0, 64)[a] for s, a in zip(seq, b.at)])
    H.check_and_record_codes("1,500 sequences", new_codes, ref[:, 0], d32[:, 0].reshape(-1, d32.shape[-1]))
    quiet = np.flatnonzero(new == 0)
    assert np.array_equal(got[quiet], b.before[0][quiet])


def test_refused_by_the_binding(t):
    b = Batch(t, 0, 2, [3, 2], [0, 1], 64)
    kw = dict(mode=0, k=b.k, v=b.v, row_start=H.dev(b.starts), pos=H.dev(np.array([0, 1], dtype=np.int32)), s=H.dev(b.s),
              k_codebook=H.dev(b.kcb), v_codebook=H.dev(b.vcb), k_codes=b.codes[0], v_codes=b.codes[1], cap_len=64,
              rope_table=b.table)
    for bad, kind in ((dict(k=b.k.int()), TypeError), (dict(v=b.v.float()), TypeError), (dict(v=b.v[:4]), ValueError),
                      (dict(k=b.k[..., :64]), ValueError), (dict(row_start=kw["row_start"][:2]), ValueError),
                      (dict(pos=kw["pos"].long()), TypeError), (dict(rope_pos=kw["pos"]), ValueError),
                      (dict(k_codes=b.codes[0][:, :1]), ValueError), (dict(cap_len=80), ValueError),
                      (dict(s=kw["s"].double()), TypeError), (dict(k_codebook=kw["k_codebook"][:, :100]), ValueError),
                      (dict(rope_table=b.table[:, :12]), ValueError), (dict(rope_table=b.table[:, :12].contiguous()), _lib.VqkvError),
                      (dict(v=b.v.cpu()), ValueError), (dict(mode=9), (ValueError, _lib.VqkvError))):
        with pytest.raises(kind):
            _lib.vqkv_append(**{**kw, **bad})
