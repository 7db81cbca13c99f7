"""Cross attention of one query per sequence where the batch's last sequences have none
and q ends with its last row: every plan, and the rows of the queries that are there."""
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


@pytest.mark.parametrize("mode", range(5))
@pytest.mark.parametrize("dt,Hq,stride,block_tokens", [("fp16", 4, 0, 0), ("bf16", 16, 4096, 64)])
@pytest.mark.parametrize("queries,lens,num_splits", [
    ([1, 1, 0, 0], [300, 64, 500, 70], 0),             # a CTA per sequence
    ([1, 0, 0], [700, 90, 0], 3),                      # splits
    ([1, 0, 1, 0], [6000, 17, 5000, 4000], 0),         # shares of all sequences' tokens
])
def test_last_sequences_without_a_query(t, mode, dt, Hq, stride, block_tokens, queries, lens, num_splits):
    x = Cross(t, mode, Hq, 2, queries, lens, dt=dt, seed=40 + mode, stride=stride, block_tokens=block_tokens)
    assert x.q.shape[0] == x.starts[-1] == sum(queries)
    got = x.run(num_splits)
    x.check(got, *x.reference())
    assert x.flags() == 0


@pytest.mark.parametrize("mode", [0, 1])
def test_more_sequences_than_shares_take(t, mode):
    """1,031 sequences: splits of each, whatever their lengths."""
    x = Cross(t, mode, 2, 1, [1] * 1029 + [0] * 2, [33] * 1031, seed=50)
    x.check(x.run(), *x.reference())
    assert x.flags() == 0
