"""Different calls at once on several streams, each with buffers of its own: the bits of the calls one by one."""
import numpy as np
import pytest

from tests import helpers as H
from tests.test_gpu_tree import case, tree_masks
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def job(mode, kind, seed):
    """(call, its outputs) on buffers of its own; a second call gives the same outputs again."""
    t = H.torch()
    B, Hq, Hkv, cap = 2, 8, 2, 1500
    M = {"tree": 9, "wide tree": 40, "mass": 1, "window": 12}.get(kind, 1)
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed)
    k, v = (H.dev(H.pack_cache_role(mode, role, c, cap)) for role, c in ((0, kc), (1, vc)))
    dq, dl, dk, dv, ds = (H.dev(x) for x in (q, np.array([1500, 777], dtype=np.int32), kcb, vcb, s))
    out = t.zeros_like(dq)
    if "tree" in kind:
        dm = H.dev(tree_masks(r, B, M, "tree").view(np.int64))
        ws = _lib.decode_tree_workspace(mode, B, Hq, Hkv, M, cap, cap)
        return lambda: _lib.vqkv_decode_attn_tree(mode, dq, dm, k, v, dl, dk, dv, ds, out, ws, cap, cap), [out]
    mass = t.zeros((B, Hkv, cap), device="cuda")
    if kind in ("mass", "window"):
        ws = _lib.decode_mass_workspace(mode, B, Hq, Hkv, M, cap, cap)

        def weights():
            mass.zero_()
            _lib.vqkv_decode_attn_mass(mode, dq, k, v, dl, dk, dv, ds, out, mass, ws, cap, cap)
        return weights, [out, mass]
    if kind == "encode":
        x = H.dev(r.standard_normal((B, Hkv, cap, 128)).astype(np.float16))
        pos = t.zeros(B, dtype=t.int32, device="cuda")
        return lambda: _lib.vqkv_encode(mode, 0, x, pos, ds, dk, k, cap), [k]
    weight = H.dev(r.random((B, Hkv, cap), dtype=np.float32))
    first = [x.clone() for x in (k, v)]
    keep, kl = t.zeros((B, Hkv, 600), dtype=t.int32, device="cuda"), t.zeros(B, dtype=t.int32, device="cuda")

    def evict():
        for a, b in zip((k, v, mass), (*first, weight)):
            a.copy_(b)
        _lib.vqkv_evict_select(mass, dl, keep, kl, 4, 64)
        _lib.vqkv_cache_compact(mode, k, v, dl, keep, kl, cap, mass=mass)
    return evict, [k, v, mass, keep]


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_calls_on_six_streams(mode):
    t = H.torch()
    kinds = ["tree", "wide tree", "mass", "window", "encode", "evict"]
    jobs = [job(mode, kind, 50 + i) for i, kind in enumerate(kinds)]
    want = []
    for call, outs in jobs:
        call()
        t.cuda.synchronize()
        want.append([x.clone() for x in outs])
    streams = [t.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(t.cuda.current_stream())
    for _ in range(30):
        for s, (call, _) in zip(streams, jobs):
            with t.cuda.stream(s):
                call()
    t.cuda.synchronize()
    for kind, (_, outs), ref in zip(kinds, jobs, want):
        assert all(t.equal(a, b) for a, b in zip(outs, ref)), kind
