"""The many-row encoders where a CTA has one tile: at 1.5, 3 and 1.25 bit its four epilogue
warpgroups screen a quarter of the centroids each.  As many rows of 8 KV heads as 19 CTAs a
head have tiles for, or fewer; ties and nearest centroids in every pair of quarters."""
import itertools

import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import helpers as H
from tests.test_gpu_encode import compare
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu
HKV = 8
ROWS = {1: 19 * 8, 3: 19 * 4, 4: 19 * 8}     # of 19 tiles


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode", ROWS)
@pytest.mark.parametrize("role", [0, 1])
@pytest.mark.parametrize("less", [0, 1, 30])
def test_codes(mode, role, less):
    n = ROWS[mode] - less
    s, kcb, vcb = H.random_codebooks(mode, HKV, 40 + mode)
    x = np.random.default_rng(mode + 10 * less).standard_normal((1, HKV, n, 128)).astype(np.float16)
    buf, ties, err = H.gpu_encode(mode, role, x, [5], s if role == 0 else None, kcb if role == 0 else vcb, 192, with_ties=True)
    assert err == 0
    compare(f"one tile, mode {mode}, {n} rows", mode, role, x, s, kcb if role == 0 else vcb, buf, [5], n, ties)


@pytest.mark.parametrize("mode", ROWS)
@pytest.mark.parametrize("a,b", list(itertools.combinations(range(4), 2)))
def test_ties_across_two_quarters(mode, a, b):
    """Quarter b repeats quarter a, and the others are far away: every distance is tied, and the lower index wins."""
    n = ROWS[mode]
    _, _, vcb = H.random_codebooks(mode, HKV, 50 + a + 4 * b)
    E = vcb.shape[1]
    parts = vcb.reshape(HKV, 4, E // 4, -1)
    parts[:, b] = parts[:, a]
    for far in set(range(4)) - {a, b}:
        parts[:, far] += np.float16(40)
    vcb = parts.reshape(vcb.shape)
    x = np.random.default_rng(3).standard_normal((1, HKV, n, 128)).astype(np.float16)
    buf, ties, err = H.gpu_encode(mode, 1, x, [0], None, vcb, 192, with_ties=True)
    assert err == 0 and ties == x.size // vcb.shape[2]
    for h in range(HKV):
        ref, d32 = vo.encode_rows(x[0, h], 1, None, vcb[h])
        got = vo.unpack_stream_fast(buf[0, h], mode, 1, n)
        assert ((got >= a * E // 4) & (got < (a + 1) * E // 4)).all()
        for t, j in zip(*np.nonzero(got != ref)):        # two different centroids as near as fp32 tells
            assert vo.near_tie(d32[t, j], int(got[t, j]))


@pytest.mark.parametrize("mode", ROWS)
@pytest.mark.parametrize("quarter", range(4))
def test_the_nearest_in_any_quarter(mode, quarter):
    """Rows made of one quarter's centroids: the nearest is at distance 0."""
    n = ROWS[mode]
    _, _, vcb = H.random_codebooks(mode, HKV, 60)
    E, d = vcb.shape[1:]
    picks = np.random.default_rng(7).integers(quarter * E // 4, (quarter + 1) * E // 4, size=(HKV, n, 128 // d))
    x = np.stack([vcb[h][picks[h]].reshape(n, 128) for h in range(HKV)])[None]
    buf, _, err = H.gpu_encode(mode, 1, x, [0], None, vcb, 192, with_ties=True)
    assert err == 0
    for h in range(HKV):
        got = vo.unpack_stream_fast(buf[0, h], mode, 1, n)
        assert np.array_equal(vcb[h][got], vcb[h][picks[h]])
