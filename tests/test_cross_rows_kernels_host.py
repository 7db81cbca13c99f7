"""What cross attention of single queries prepares and launches, against the stand-in for
the CUDA runtime: one kernel a call, which merges by itself.  No GPU needed."""
from tests.test_cross_prepare_host import CALLS
from tests.test_prepare_host import run  # noqa: F401  (a fixture)


def test_one_kernel_per_call(run):  # noqa: F811
    run(CALLS + """
for m in range(5):
    for B, Hkv, cap, splits in ((1, 2, 65536, 0), (3, 1, 65536, 0), (16, 16, 1024, 0), (2, 2, 1024, 5), (1100, 2, 64, 0), (4, 8, 65536, 0)):
        a = cross(m, B, 1, B=B, Hq=8 * Hkv, Hkv=Hkv, cap_len=cap, max_seq_len=cap, num_splits=splits, workspace_bytes=1 << 34,
                  q=0x10000000)
        a.q_row_stride = 8 * Hkv * 128
        log()
        assert L.vqkv_cross_attn(ctypes.byref(a), None, None) == 0
        launched = [x for x in log() if x.startswith("launch")]
        assert len(launched) == 1 and "decode_vq" in launched[0], launched
        x, y, z = (int(v) for v in launched[0].split()[-3:])
        assert y == Hkv and z in (2, 2 * B), (x, y, z)     # two column groups; a CTA takes one sequence, or a share of all
""")
