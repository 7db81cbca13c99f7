"""The plan of cross attention of single queries against the stand-in for the CUDA runtime:
where its workspace ends, and how many CTAs a sequence gets.  No GPU needed."""
from tests.test_cross_prepare_host import CALLS
from tests.test_prepare_host import run  # noqa: F401  (a fixture)


def test_partials_lie_behind_the_tickets_of_every_decode(run):  # noqa: F811
    """Word 0 to byte 256, then B x Hkv tickets of eight groups, rounded up to 256 bytes, then 132 floats per
    split and column; the tickets that the call uses are the first B x Hkv."""
    run(CALLS + """
for m in range(5):
    for B, Hq, Hkv, splits in ((2, 8, 2, 3), (64, 64, 8, 2), (1, 5, 1, 7), (3, 2, 2, 1)):
        a = cross(m, B, 1, B=B, Hq=Hq, Hkv=Hkv, cap_len=4096, max_seq_len=4096, num_splits=splits)
        d = dec(m, B=B, Hq=Hq, Hkv=Hkv, cap_len=4096, max_seq_len=4096, num_splits=splits)
        n = L.vqkv_decode_num_splits(ctypes.byref(d))
        tickets = (256 + 4 * B * Hkv * 8 + 255) // 256 * 256
        need = L.vqkv_cross_attn_workspace_bytes(ctypes.byref(a))
        assert need == tickets + 4 * B * Hq * n * 132, (m, B, Hq, Hkv, need, n)
""")


def test_splits_fit_half_a_ticket(run):  # noqa: F811
    out = run(CALLS + """
for m in range(5):
    a = cross(m, 2, 1, cap_len=1 << 23, max_seq_len=1 << 23, num_splits=1 << 20, workspace_bytes=1 << 40)
    log()
    assert L.vqkv_cross_attn(ctypes.byref(a), None, None) == 0
    print([x.split()[-3] for x in log() if x.startswith("launch")][0])
""")
    assert out and all(1000 < int(x) <= 65535 for x in out), out
