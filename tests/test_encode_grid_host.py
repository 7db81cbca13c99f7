"""The grids of the encode against the stand-in for the CUDA runtime (152 SMs): one wave of
CTAs, each with work.  No GPU needed."""
from tests.test_prepare_host import run  # noqa: F401  (a fixture)

BODY = """
ROWS = {0: 4, 1: 8, 2: 2, 3: 4, 4: 8}      # rows of a tile of the many-row kernels
for mode in range(5):
    for B, Hkv, n in ((1, 8, 64), (1, 8, 20), (4, 8, 33), (2, 3, 500), (1, 5, 4000), (1, 6, 1000), (1, 7, 90), (1, 1, 153), (3, 200, 7),
                      (1, 1, 152), (2, 8, 9), (1, 77, 40)):
        a = _lib.EncodeArgs(mode=mode, role=1, B=B, Hkv=Hkv, head_dim=128, n_rows=n, cap_len=8192, x=0x1000, pos=0x2000, s=0x3000,
                            codebook=0x4000, codes=0x5000)
        log()
        assert L.vqkv_encode(ctypes.byref(a), None) == 0
        x, y, z = (int(v) for v in [l for l in log() if l.startswith("launch")][0].split()[-3:])
        few = B * n * Hkv <= 152
        tiles = -(-B * n // ROWS[mode])
        assert (y, z) == (Hkv, 1)
        assert x == (B * n if few else min(tiles, max(152 // Hkv, 1))), (mode, B, Hkv, n, x)
        assert x * Hkv <= 152 or x == 1
"""


def test_one_wave_of_ctas_with_work(run):  # noqa: F811
    run(BODY)
