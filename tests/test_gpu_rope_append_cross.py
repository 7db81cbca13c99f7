"""The rotary, append and cross-attention calls together, as an encoder-decoder
layer uses them: encoder states into one packed cache, a ragged batch of decoder
prompts into another, then decode steps over both, eager and as a captured graph
that advances its own positions."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import attn_reference as A
from tests import helpers as H
from tests import rope_reference as R
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu

B, HQ, HKV, ROT, BLOCK, CAP, SHIFT = 3, 8, 4, 96, 64, 128, 7   # SHIFT: tokens evicted before, so angles run ahead
ENC, PROMPT, STEPS = [70, 1, 130], [5, 62, 1], 3


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


class Layer:
    def __init__(self, t, mode, seed):
        self.t, self.mode = t, mode
        r = self.r = np.random.default_rng(seed)
        self.s, self.kcb, self.vcb = H.random_codebooks(mode, HKV, seed + 1)
        self.books = [H.dev(x) for x in (self.kcb, self.vcb, self.s)]
        enc_cap = max(ENC)
        self.enc = [t.zeros((B, HKV, _lib.vqkv_code_bytes(mode, enc_cap)), dtype=t.uint8, device="cuda") for _ in range(2)]
        self.enc_cap, self.enc_lens = enc_cap, H.dev(np.array(ENC, dtype=np.int32))
        per = CAP // BLOCK
        self.blocks = r.permutation(B * per).reshape(B, per).astype(np.int32)
        self.paged = dict(block_table=H.dev(self.blocks), block_tokens=BLOCK, num_blocks=B * per)
        self.self_ = [t.zeros((B * per, HKV, _lib.vqkv_code_bytes(mode, BLOCK)), dtype=t.uint8, device="cuda") for _ in range(2)]
        self.table = t.empty((CAP + SHIFT, ROT), device="cuda")
        _lib.vqkv_rope_table(self.table, base=500000.0, scaling=_lib.VQKV_ROPE_WAVELENGTH, factor=8.0, original_len=64)
        self.err = t.zeros(1, dtype=t.int32, device="cuda")
        self.lens = H.dev(np.zeros(B, dtype=np.int32))
        self.one = H.dev(np.arange(B + 1, dtype=np.int32))
        self.ws_self = _lib.decode_workspace(mode, B, HQ, HKV, CAP, CAP)
        self.ws_step = _lib.cross_attn_workspace(mode, B, HQ, HKV, B, 1, enc_cap, enc_cap)
        n = sum(PROMPT)
        self.ws_prompt = _lib.cross_attn_workspace(mode, B, HQ, HKV, n, max(PROMPT), enc_cap, enc_cap)

    def rows(self, n, dtype):     # a projection's output: queries, keys, values side by side
        x = self.r.standard_normal((n, HQ + 2 * HKV, 128)).astype(np.float32)
        return self.t.from_numpy(x).cuda().to(dtype)

    def encode(self, qkv):
        starts = H.dev(np.concatenate([[0], np.cumsum(ENC)]).astype(np.int32))
        _lib.vqkv_append(self.mode, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], starts, self.t.zeros_like(self.lens), self.books[2],
                         *self.books[:2], *self.enc, self.enc_cap, error_flags=self.err)

    def prompt(self, qkv, angles):
        starts = H.dev(np.concatenate([[0], np.cumsum(PROMPT)]).astype(np.int32))
        self.append(qkv, starts, angles)
        self.lens += H.dev(np.array(PROMPT, dtype=np.int32))
        q = qkv[:, :HQ]
        _lib.vqkv_rope(q, angles, self.table, q, error_flags=self.err)      # in place, among the keys and values
        out = self.t.zeros((q.shape[0], HQ, 128), dtype=q.dtype, device="cuda")
        self.cross(q, starts, out, self.ws_prompt, max(PROMPT))
        return q, out

    def append(self, qkv, starts, angles):
        _lib.vqkv_append(self.mode, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], starts, self.lens, self.books[2], *self.books[:2],
                         *self.self_, CAP, rope_table=self.table, rope_pos=angles, error_flags=self.err, **self.paged)

    def cross(self, q, starts, out, ws, most):
        _lib.vqkv_cross_attn(self.mode, q, starts, *self.enc, self.enc_lens, *self.books, out, ws, self.enc_cap, self.enc_cap, most)

    def step(self, qkv, q, own, cross):
        """One token per sequence; positions advance on the device."""
        angles = self.lens + SHIFT
        self.append(qkv, self.one, angles)
        self.lens += 1
        _lib.vqkv_rope(qkv[:, :HQ], angles, self.table, q, error_flags=self.err)
        _lib.vqkv_decode_attn_paged(self.mode, q, *self.self_, self.lens, *self.books, own, self.ws_self, CAP, CAP, **self.paged)
        self.cross(q, self.one, cross, self.ws_step, 1)

    def codes(self, role, b, h, n, enc=False):
        buf = (self.enc if enc else self.self_)[role].cpu().numpy()
        stream = buf[b, h] if enc else np.concatenate([buf[i, h] for i in self.blocks[b]])
        return vo.unpack_stream_fast(stream, self.mode, role, n)


def attend(L, q, b, n, enc):
    """(O, bound) of query rows q [m][Hq][128] over the n tokens that a cache holds for sequence b."""
    kc, vc = ([L.codes(role, b, h, n, enc) for h in range(HKV)] for role in (0, 1))
    o, _, e = A.attend(q[None], [kc], [vc], L.kcb, L.vcb, L.s, [n], lambda *_: np.ones(n, dtype=bool))
    return o[0], e[0]


@pytest.mark.parametrize("mode", range(5))
def test_encoder_decoder_layer(t, mode):
    L = Layer(t, mode, 30 + mode)
    enc = L.rows(sum(ENC), t.bfloat16)
    L.encode(enc)
    edges = np.concatenate([[0], np.cumsum(PROMPT)])
    at = np.concatenate([np.arange(n) for n in PROMPT]) + SHIFT
    qkv = L.rows(sum(PROMPT), t.bfloat16)
    before = qkv.double().cpu().numpy()
    q, out = L.prompt(qkv, H.dev(at.astype(np.int32)))
    steps = [L.rows(B, t.float16) for _ in range(STEPS)]
    eager = []
    for x in steps:
        a = [t.zeros((B, HQ, 128), dtype=t.float16, device="cuda") for _ in range(3)]
        L.step(x, *a)
        eager.append(a)
    t.cuda.synchronize()
    assert int(L.err) == 0 and all(int(w.view(t.int32)[0]) == 0 for w in (L.ws_self, L.ws_step, L.ws_prompt))
    assert L.lens.tolist() == [n + STEPS for n in PROMPT]

    # codes of the encoder's states, the prompts and the steps, as the oracle's
    table = L.table.double().cpu().numpy()
    e = enc.double().cpu().numpy()
    enc_edges = np.concatenate([[0], np.cumsum(ENC)])
    for role, cols, cb in ((0, slice(HQ, HQ + HKV), L.kcb), (1, slice(HQ + HKV, None), L.vcb)):
        ref, d32 = R.append_codes(e[:, cols], role, L.s, cb)
        for b in range(B):
            rows = slice(enc_edges[b], enc_edges[b + 1])
            for h in range(HKV):
                H.check_and_record_codes(f"encoder states, mode {mode}, role {role}", L.codes(role, b, h, ENC[b], True), ref[rows, h],
                                         d32[rows, h].reshape(-1, d32.shape[-1]))
        for b in range(B):
            x = np.concatenate([before[edges[b]:edges[b + 1], cols]] + [y.double().cpu().numpy()[b:b + 1, cols] for y in steps])
            ref, d32 = R.append_codes(x, role, L.s, cb, table[np.arange(len(x)) + SHIFT])
            for h in range(HKV):
                H.check_and_record_codes(f"decoder tokens, mode {mode}, role {role}", L.codes(role, b, h, len(x)), ref[:, h],
                                         d32[:, h].reshape(-1, d32.shape[-1]))

    # rotated queries and the prompts' cross attention
    y, size = R.rotate(before[:, :HQ], table[at])
    assert (np.abs(q.double().cpu().numpy() - y) <= R.rope_bound(y, size, "bf16", ROT)).all()
    assert t.equal(qkv[:, HQ:], t.from_numpy(before[:, HQ:]).cuda().to(qkv.dtype))
    got, rotated = out.double().cpu().numpy(), q.double().cpu().numpy()
    for b in range(B):
        rows = slice(edges[b], edges[b + 1])
        o, tol = attend(L, rotated[rows], b, ENC[b], True)
        assert (np.abs(got[rows] - o) <= tol + 2.0 ** -8 * (np.abs(o) + tol)).all()
    # the steps' attention over both caches
    for i, (sq, own, cross) in enumerate(eager):
        sq, own, cross = (x.double().cpu().numpy() for x in (sq, own, cross))
        for b in range(B):
            for got, n, enc_cache in ((own, PROMPT[b] + i + 1, False), (cross, ENC[b], True)):
                o, tol = attend(L, sq[b:b + 1], b, n, enc_cache)
                assert (np.abs(got[b] - o[0]) <= tol[0]).all()

    # the same steps as replays of one captured step
    final = [x.clone() for x in L.self_]
    L.lens -= STEPS
    x = t.zeros_like(steps[0])
    a = [t.zeros((B, HQ, 128), dtype=t.float16, device="cuda") for _ in range(3)]
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        L.step(x, *a)
    for i in range(STEPS):
        x.copy_(steps[i])
        g.replay()
        assert all(t.equal(p, w) for p, w in zip(a, eager[i])), i
    assert all(t.equal(p, w) for p, w in zip(L.self_, final))
