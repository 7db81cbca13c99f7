"""One workspace for cross attention of single queries and the decode calls of the same B
and Hkv, in every order: each call has the bits that a workspace of its own gives."""
import itertools

import numpy as np
import pytest

from tests import helpers as H
from tests.test_gpu_cross import Cross
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


class Calls:
    """Cross attention of one query (x.run) and of three, a decode, a _multi of eight groups and a draft tree."""
    def __init__(self, t, mode, Hq, Hkv, lens, num_splits, seed=0):
        B = len(lens)
        self.t, self.num_splits, self.mode = t, num_splits, mode
        x = self.x = Cross(t, mode, Hq, Hkv, [1] * B, lens, seed=seed)
        M = 64 * Hkv // Hq
        r = np.random.default_rng(seed)
        some = lambda *shape: H.dev(r.standard_normal((*shape, Hq, 128)).astype(np.float16))  # noqa: E731
        self.q3, self.qm, self.start3 = some(3 * B), some(B, M), H.dev(np.arange(0, 3 * B + 1, 3, dtype=np.int32))
        self.masks = H.dev(np.full((B, M), 2**M - 1, dtype=np.int64))
        self.shape = (mode, B, Hq, Hkv)
        cap = x.cap
        self.sizes = {
            "cross": x.workspace(num_splits), "cross3": _lib.cross_attn_workspace(mode, B, Hq, Hkv, 3 * B, 3, cap, cap, num_splits),
            "decode": _lib.decode_workspace(*self.shape, cap, cap, num_splits),
            "multi": _lib.decode_workspace(*self.shape, cap, cap, num_splits, n_queries=M),
            "tree": _lib.decode_tree_workspace(mode, B, Hq, Hkv, M, cap, cap, num_splits)}

    def run(self, what, ws):
        x, t = self.x, self.t
        rest = (x.k, x.v, x.dlens, *x.books)
        q = {"cross": x.q, "cross3": self.q3, "decode": x.q, "multi": self.qm, "tree": self.qm}[what]
        out = t.full_like(q, float("nan"))
        kw = dict(num_splits=self.num_splits)
        if what in ("cross", "cross3"):
            start, most = (x.dstarts, 1) if what == "cross" else (self.start3, 3)
            _lib.vqkv_cross_attn(self.mode, q, start, *rest, out, ws, x.cap, x.cap, most, **kw)
        elif what == "decode":
            _lib.vqkv_decode_attn(self.mode, q, *rest, out, ws, x.cap, x.cap, **kw)
        elif what == "multi":
            _lib.vqkv_decode_attn_multi(self.mode, q, *rest, out, ws, x.cap, x.cap, **kw)
        else:
            _lib.vqkv_decode_attn_tree(self.mode, q, self.masks, *rest, out, ws, x.cap, x.cap, **kw)
        return out


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("Hq,Hkv,lens,num_splits", [
    (64, 8, [2100, 1900, 2000, 1700], 0),              # shares of all tokens; two groups of columns
    (64, 8, [900, 700, 800, 600, 500, 400, 300, 200], 3),
    (16, 2, [5000], 0),                                # one sequence
    (40, 8, [2100, 1900, 2000, 1700], 0),              # five columns: groups of four and of one
])
def test_shared_with_decode_multi_and_trees(t, mode, Hq, Hkv, lens, num_splits):
    c = Calls(t, mode, Hq, Hkv, lens, num_splits, seed=mode)
    names = list(c.sizes)
    want = {w: c.run(w, c.sizes[w]) for w in names}
    for w in names:
        assert t.isfinite(want[w]).all(), w
    c.x.check(want["cross"], *c.x.reference())
    size = max(w.numel() for w in c.sizes.values())
    # each other call between two of cross attention, of one query and of several
    for cross, other in itertools.product(("cross", "cross3"), names):
        ws = t.zeros(size, dtype=t.uint8, device="cuda")
        for what in (cross, other, cross, other, cross):
            assert t.equal(c.run(what, ws), want[what]), (cross, other, what)
        assert int(ws[:4].view(t.int32)) == 0


@pytest.mark.parametrize("mode", range(5))
def test_single_queries_on_a_used_workspace(t, mode):
    """Whatever lies behind B x Hkv tickets, as a decode of one query per sequence leaves it."""
    x = Cross(t, mode, 16, 2, [1, 1, 0, 1], [3000, 1900, 200, 2500], seed=90 + mode, qscale=12.0)
    for num_splits in (0, 4):
        want = x.run(num_splits).clone()
        x.check(want, *x.reference())
        for value in (1.5, float("nan")):
            ws = t.zeros_like(x.ws)
            behind = (256 + 4 * 4 * 2 + 255) // 256 * 256
            ws[behind:].view(t.float32).fill_(value)
            assert t.equal(x.run(num_splits, out=t.full_like(x.out, 3.0), ws=ws), want)
            assert x.flags() == 0
