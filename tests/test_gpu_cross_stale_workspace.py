"""Cross attention does not depend on what earlier calls left behind the tickets of its
workspace: columns past a sequence's last share its warps, and have no q' of their own."""
import numpy as np
import pytest

from tests import helpers as H
from tests.test_gpu_cross import Cross
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def left_behind(t, kind, n):
    """n bytes as other calls leave them: fp32 partials, query images of large values, or bits of any kind."""
    r = np.random.default_rng(n)
    x = {"partials": r.standard_normal(n // 4).astype(np.float32), "images": (300 * r.standard_normal(n // 2)).astype(np.float16),
         "bits": r.integers(0, 256, n, dtype=np.uint8), "nan": np.full(n // 2, np.nan, dtype=np.float16)}[kind]
    return H.dev(x).view(t.uint8)


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,queries", [(8, [3, 2]), (8, [9, 1]), (4, [33, 5]), (8, [41, 70]), (2, [300, 129])])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_same_bits_on_a_used_workspace(t, mode, dt, Hq, queries, num_splits):
    """Scores that climb over the lazy rescale's slack now and then (some 11 nats rms)."""
    x = Cross(t, mode, Hq, 2, queries, [700, 400], seed=80 + mode, qscale=12.0, dt=dt)
    want = x.run(num_splits).clone()
    x.check(want, *x.reference())
    tickets = (256 + 4 * 2 * 2 * 8 + 255) // 256 * 256     # B x Hkv of eight column groups: zero between calls
    for kind in ("partials", "images", "bits", "nan"):
        ws = t.zeros_like(x.ws)
        ws[tickets:] = left_behind(t, kind, ws.numel() + 4)[:ws.numel() - tickets]
        got = x.run(num_splits, out=t.full_like(x.out, 3.0), ws=ws)
        assert t.equal(got, want), kind
        assert x.flags() == 0
