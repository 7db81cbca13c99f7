"""bf16 cross attention of general queries with large scores: its error is that of its
own roundings, whatever the scores and however many queries a sequence has."""
import numpy as np
import pytest

from tests.test_gpu_cross import Cross
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def limit(t, ref):
    """Rms error of the exact result rounded to bf16 (computed here) and of the softmax weights' rounding to fp16,
    uniform within 2^-11 relative: 2^-11 / sqrt(3) at most; independent of each other, and 4 % for the sample."""
    rounded = t.from_numpy(ref).float().bfloat16().double().numpy()
    return 1.04 * np.hypot(np.linalg.norm(rounded - ref) / np.linalg.norm(ref), 2.0 ** -11 / 3 ** 0.5)


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("queries", [[1, 1], [8, 5], [33, 20], [65, 33], [200, 1]])
@pytest.mark.parametrize("qscale", [1.0, 12.0, 24.0])
def test_error_is_the_roundings(t, mode, queries, qscale):
    """Scores of some 1, 11 and 22 nats (rms).  One fp16 part of q' is off by 2^-12 rms: 1.4e-4 of a score, so
    weights by 1.5e-3 at 11 nats, as much as the result's rounding."""
    x = Cross(t, mode, 8, 4, queries, [500, 300], seed=60 + mode, qscale=qscale, dt="bf16")
    got = x.run().double().cpu().numpy()
    ref, _ = x.reference()
    assert np.linalg.norm(got - ref) <= limit(t, ref) * np.linalg.norm(ref)
    assert x.flags() == 0


@pytest.mark.parametrize("queries", [[2, 3], [30, 9], [130, 40]])
def test_the_same_query_alone_and_among_others(t, queries):
    """A query's result does not depend on how many others its sequence has, but for a rounding's direction: at
    most one bf16 step apart, two 2^-8 halves, beside the fp16 roundings of the weights (tolerance of the reference)."""
    x = Cross(t, 2, 8, 2, queries, [300, 70], seed=70, qscale=12.0, dt="bf16")
    many = x.run().double().cpu().numpy()
    first = x.starts[:-1]
    one = Cross(t, 2, 8, 2, [1, 1], [300, 70], seed=70, dt="bf16")
    one.k, one.v, one.books, one.q = x.k, x.v, x.books, x.q[first].contiguous()
    alone = one.run().double().cpu().numpy()
    ref, _ = x.reference()
    got = np.stack([many[first], alone])
    for o in got:
        assert np.linalg.norm(o - ref[first]) <= limit(t, ref[first]) * np.linalg.norm(ref[first])
