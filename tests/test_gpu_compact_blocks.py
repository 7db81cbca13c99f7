"""vqkv_cache_compact over a block table with entries outside the pool: codes and weights stay together."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import helpers as H
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode,page", [(0, 64), (1, 64), (1, 128), (2, 64), (3, 128), (4, 256)])
def test_weights_stay_with_the_codes_that_stay(mode, page):
    t = H.torch()
    r = np.random.default_rng(20 + mode)
    E, d = vo.GEOMETRY[mode]
    Hkv, per, nblk = 2, 8, 9
    cap = per * page
    L, n = cap - 5, 5 * page + 17
    toks = [r.integers(0, E, size=(nblk, Hkv, page, 128 // d)) for _ in range(2)]
    pools = [np.stack([np.stack([vo.pack_stream_fast(x[i, h], mode, role, page) for h in range(Hkv)]) for i in range(nblk)])
             for role, x in enumerate(toks)]
    table = r.permutation(nblk)[:per].astype(np.int32)
    gone = [1, 4, 6]                                   # destinations and sources, destinations, sources only
    table[gone] = [nblk, -1, 2**31 - 1]
    mass = r.random((1, Hkv, cap), dtype=np.float32)
    src = np.sort(np.stack([r.permutation(np.arange(n // 2, L))[:n] if L - n // 2 >= n else r.permutation(L)[:n]
                            for _ in range(Hkv)]), axis=1)[None].astype(np.int32)
    want_t, want_m = [x.copy() for x in toks], mass.copy()
    for h in range(Hkv):
        for i in range(n):
            s = int(src[0, h, i])
            if i // page in gone or s // page in gone or not i <= s < L:
                continue
            for w, x in zip(want_t, toks):
                w[table[i // page], h, i % page] = x[table[s // page], h, s % page]
            want_m[0, h, i] = mass[0, h, s]
        want_m[0, h, n:L] = 0.0
    k, v, m = H.dev(pools[0]), H.dev(pools[1]), H.dev(mass)
    err = t.zeros(1, dtype=t.int32, device="cuda")
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    _lib.vqkv_cache_compact(mode, k, v, i32(L), H.dev(src), i32(n), cap, mass=m, error_flags=err,
                            block_table=H.dev(table[None]), block_tokens=page, num_blocks=nblk)
    assert int(err.item()) & _lib.VQKV_DEVERR_BLOCK
    for role, buf in ((0, k), (1, v)):
        got = buf.cpu().numpy()
        for i in range(nblk):
            for h in range(Hkv):
                assert np.array_equal(got[i, h], vo.pack_stream_fast(want_t[role][i, h], mode, role, page)), (role, i, h)
    assert np.array_equal(m.cpu().numpy(), want_m)
