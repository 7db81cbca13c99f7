"""The many-row encoders where a CTA has one tile (64 rows of 8 KV heads): at 1.5, 3 and
1.25 bit both epilogue warpgroups screen it, half of the centroids each."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import helpers as H
from tests.test_gpu_encode import compare
from vector_quantized_bit_gb300 import _build

pytestmark = pytest.mark.gpu
HKV, N = 8, 64
MODES = [1, 3, 4, 0, 2]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("role", [0, 1])
@pytest.mark.parametrize("n", [N, 33, 127])
def test_codes(mode, role, n):
    s, kcb, vcb = H.random_codebooks(mode, HKV, 40 + mode)
    x = np.random.default_rng(mode).standard_normal((1, HKV, n, 128)).astype(np.float16)
    buf, ties, err = H.gpu_encode(mode, role, x, [5], s if role == 0 else None, kcb if role == 0 else vcb, 192, with_ties=True)
    assert err == 0
    compare(f"one tile, mode {mode}, {n} rows", mode, role, x, s, kcb if role == 0 else vcb, buf, [5], n, ties)


@pytest.mark.parametrize("mode", MODES)
def test_ties_across_the_halves(mode):
    """The upper half of the codebook repeats the lower: every distance is tied, and the lowest index wins."""
    _, _, vcb = H.random_codebooks(mode, HKV, 50)
    E = vcb.shape[1]
    vcb[:, E // 2:] = vcb[:, :E // 2]
    x = np.random.default_rng(3).standard_normal((1, HKV, N, 128)).astype(np.float16)
    buf, ties, err = H.gpu_encode(mode, 1, x, [0], None, vcb, N, with_ties=True)
    assert err == 0 and ties == x.size // vcb.shape[2]
    for h in range(HKV):
        ref, d32 = vo.encode_rows(x[0, h], 1, None, vcb[h])
        got = vo.unpack_stream_fast(buf[0, h], mode, 1, N)
        assert (got < E // 2).all()
        for t, j in zip(*np.nonzero(got != ref)):        # two different centroids as near as fp32 tells
            assert vo.near_tie(d32[t, j], int(got[t, j]))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("half", [0, 1])
def test_the_nearest_in_either_half(mode, half):
    """Rows made of one half's centroids: the nearest is at distance 0."""
    _, _, vcb = H.random_codebooks(mode, HKV, 60)
    E, d = vcb.shape[1:]
    r = np.random.default_rng(7)
    picks = r.integers(half * E // 2, (half + 1) * E // 2, size=(HKV, N, 128 // d))
    x = np.stack([vcb[h][picks[h]].reshape(N, 128) for h in range(HKV)])[None]
    buf, _, err = H.gpu_encode(mode, 1, x, [0], None, vcb, N, with_ties=True)
    assert err == 0
    for h in range(HKV):
        got = vo.unpack_stream_fast(buf[0, h], mode, 1, N)
        assert np.array_equal(vcb[h][got], vcb[h][picks[h]])


@pytest.mark.parametrize("mode", MODES)
def test_values_beyond_fp16_and_codebooks_beyond_the_table(mode):
    """Both fall back to the exhaustive search, of all centroids by the first warpgroup."""
    s, kcb, vcb = H.random_codebooks(mode, HKV, 70)
    x = np.random.default_rng(8).standard_normal((1, HKV, N, 128)).astype(np.float16)
    s[:, :16] = 1e-5
    big = (kcb.astype(np.float32) * 50).astype(np.float16)
    buf, ties, err = H.gpu_encode(mode, 0, x, [0], s, big, N, with_ties=True)
    assert err == 0
    compare(f"one tile, mode {mode}, beyond fp16", mode, 0, x, s, big, buf, [0], N, ties, bounded=False)
    far = vcb.copy()
    far[:, -1] = 900.0
    buf, ties, err = H.gpu_encode(mode, 1, x, [0], None, far, N, with_ties=True)
    assert err == 0
    compare(f"one tile, mode {mode}, far centroid", mode, 1, x, s, far, buf, [0], N, ties)
