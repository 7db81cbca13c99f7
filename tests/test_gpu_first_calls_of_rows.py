"""The first call of a process that encodes many rows, appends, rotates or takes cross
attention, made under stream capture."""
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
mode = int(sys.argv[2])
import numpy as np, torch as t
from tests import helpers as H
from vector_quantized_bit_gb300 import _lib
B, Hq, Hkv, cap, n = 2, 8, 2, 640, 200
r = np.random.default_rng(mode)
s, kcb, vcb = (H.dev(x) for x in H.random_codebooks(mode, Hkv, 1))
rows = lambda *shape: H.dev(r.standard_normal((*shape, 128)).astype(np.float16))
ints = lambda *x: H.dev(np.array(x, dtype=np.int32))
x, k, v, one = rows(B, Hkv, n), rows(2 * n, Hkv), rows(2 * n, Hkv), rows(B, Hkv)
qs = [rows(m * B, Hq) for m in (1, 3, 40)]                     # of the three ways cross attention is laid out
starts = [ints(0, m, 2 * m) for m in (1, 3, 40)]
codes = [t.zeros((B, Hkv, int(_lib.lib().vqkv_code_bytes(mode, cap))), dtype=t.uint8, device="cuda") for _ in range(2)]
pos0, pos1, pos2, lens, split = ints(0, 0), ints(n, n), ints(2 * n, 2 * n), ints(2 * n + 1, 2 * n + 1), ints(0, n, 2 * n)
one_start, at = ints(0, 1, 2), t.arange(2 * n, dtype=t.int32, device="cuda")
table, turned = t.zeros((cap, 128), device="cuda"), t.zeros_like(k)
outs = [t.zeros_like(q) for q in qs]
flags = t.zeros(1, dtype=t.int32, device="cuda")
ws = [t.zeros(1 << 24, dtype=t.uint8, device="cuda") for _ in qs]   # no workspace query prepares anything
t.cuda.synchronize()

def step():
    _lib.vqkv_rope_table(table)
    _lib.vqkv_rope(k, at, table, turned, error_flags=flags)
    for role, (book, c) in enumerate(zip((kcb, vcb), codes)):
        _lib.vqkv_encode(mode, role, x, pos0, s if role == 0 else None, book, c, cap, error_flags=flags)
    _lib.vqkv_append(mode, turned, v, split, pos1, s, kcb, vcb, *codes, cap, error_flags=flags)
    _lib.vqkv_append(mode, one, one, one_start, pos2, s, kcb, vcb, *codes, cap, rope_table=table, error_flags=flags)
    for q, start, out, w, m in zip(qs, starts, outs, ws, (1, 3, 40)):
        _lib.vqkv_cross_attn(mode, q, start, *codes, lens, kcb, vcb, s, out, w, cap, cap, m)

def results():
    t.cuda.synchronize()
    return [y.clone() for y in (table, turned, *codes, *outs, flags)]

g = t.cuda.CUDAGraph()
with t.cuda.graph(g):
    step()
g.replay()
captured = results()
for y in (table, turned, *codes, *outs):
    y.zero_()
step()
assert all(t.equal(a, b) for a, b in zip(captured, results()))
assert int(flags) == 0 and all(int(y.count_nonzero()) > 0 for y in (table, turned, *codes, *outs))
assert not any(int(w[:4].view(t.int32)) for w in ws)
"""


@pytest.mark.parametrize("mode", range(5))
def test_first_calls_under_capture(mode):
    _build.build()
    r = subprocess.run([sys.executable, "-c", BODY, ROOT, str(mode)], capture_output=True, text=True, timeout=300,
                       cwd=ROOT, env=dict(os.environ))
    assert r.returncode == 0, r.stderr[-3000:]
