"""The first call of a process that uses a kernel, made under stream capture."""
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu

BODY = """
import sys
sys.path.insert(0, sys.argv[1])
import numpy as np, torch as t
from tests import helpers as H
from tests.test_gpu_tree import case, tree_masks
from vector_quantized_bit_gb300 import _lib
mode, B, Hq, Hkv, M, cap = 0, 2, 8, 2, 9, 640
r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=1)
k, v = (H.dev(H.pack_cache_role(mode, role, c, cap)) for role, c in ((0, kc), (1, vc)))
dq, dm, dl, dk, dv, ds = (H.dev(x) for x in (q, tree_masks(r, B, M, "tree").view(np.int64), np.array([640, 333], dtype=np.int32),
                                             kcb, vcb, s))
out, one = t.zeros_like(dq), t.zeros_like(dq)
mass = t.zeros((B, Hkv, cap), device="cuda")
keep, kl = t.zeros((B, Hkv, 100), dtype=t.int32, device="cuda"), t.zeros(B, dtype=t.int32, device="cuda")
# device memory as a serving engine holds it: no workspace query of these calls ran before either
tree_ws, mass_ws = (t.zeros(1 << 24, dtype=t.uint8, device="cuda") for _ in range(2))
plain_ws = _lib.decode_workspace(mode, B, Hq, Hkv, cap, cap)
_lib.vqkv_decode_attn(mode, dq[:, 0].contiguous(), k, v, dl, dk, dv, ds, one[:, 0].contiguous(), plain_ws, cap, cap)
t.cuda.synchronize()
state = [x.clone() for x in (k, v, mass)]

def step():
    _lib.vqkv_decode_attn_tree(mode, dq, dm, k, v, dl, dk, dv, ds, out, tree_ws, cap, cap)
    _lib.vqkv_decode_attn_mass(mode, dq, k, v, dl, dk, dv, ds, one, mass, mass_ws, cap, cap)
    _lib.vqkv_evict_select(mass, dl, keep, kl, 4, 8)
    _lib.vqkv_cache_compact(mode, k, v, dl, keep, kl, cap, mass=mass)

def results():
    t.cuda.synchronize()
    return [x.clone() for x in (out, one, mass, keep, kl, k, v)]

g = t.cuda.CUDAGraph()
with t.cuda.graph(g):
    step()
g.replay()
captured = results()
for x, y in zip((k, v, mass), state):
    x.copy_(y)
for x in (out, one, keep, kl):
    x.zero_()
step()
assert all(t.equal(a, b) for a, b in zip(captured, results()))
assert kl.tolist() == [100, 100] and int(out.count_nonzero()) > 0
"""


def test_first_calls_under_capture():
    _build.build()
    r = subprocess.run([sys.executable, "-c", BODY, ROOT], capture_output=True, text=True, timeout=300,
                       cwd=ROOT, env=dict(os.environ))
    assert r.returncode == 0, r.stderr[-3000:]
