"""Attention calls whose output is the queries' own buffer."""
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


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("call,M", [("multi", 1), ("multi", 6), ("tree", 9), ("tree", 40), ("mass", 1), ("mass", 3), ("mass", 9),
                                    ("mass", 16)])
def test_output_over_the_queries(mode, call, M):
    """The bits of O (and of the weights) that a buffer of its own gives."""
    t = H.torch()
    B, Hq, Hkv, cap = 3, 8, 2, 800
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=15 + mode)
    k, v = (H.dev(H.pack_cache_role(mode, role, c, cap)) for role, c in ((0, kc), (1, vc)))
    dq, dm, dl, dk, dv, ds = (H.dev(x) for x in (q, tree_masks(r, B, M, "tree").view(np.int64),
                                                 np.array([800, 0, 333], dtype=np.int32), kcb, vcb, s))
    sizes = (mode, B, Hq, Hkv)
    ws = {"multi": lambda: _lib.decode_workspace(*sizes, cap, cap, n_queries=M),
          "tree": lambda: _lib.decode_tree_workspace(*sizes, M, cap, cap),
          "mass": lambda: _lib.decode_mass_workspace(*sizes, M, cap, cap)}[call]()

    def run(queries, out):
        mass = t.zeros((B, Hkv, cap), device="cuda")
        args = (k, v, dl, dk, dv, ds, out)
        if call == "multi":
            _lib.vqkv_decode_attn_multi(mode, queries, *args, ws, cap, cap)
        elif call == "tree":
            _lib.vqkv_decode_attn_tree(mode, queries, dm, *args, ws, cap, cap)
        else:
            _lib.vqkv_decode_attn_mass(mode, queries, *args, mass, ws, cap, cap)
        t.cuda.synchronize()
        return out, mass

    want, wmass = run(dq, t.empty_like(dq))
    own = dq.clone()
    got, gmass = run(own, own)
    assert t.equal(got, want) and t.equal(gmass, wmass)
