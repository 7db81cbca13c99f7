"""Which kernels the append and cross-attention calls prepare on the host, against
the stand-in for the CUDA runtime.  No GPU needed."""
from tests.test_prepare_host import run  # noqa: F401  (a fixture)

CALLS = """
def append(mode, n=3, **kw):
    a = _lib.AppendArgs(mode=mode, dtype=2, B=2, Hkv=2, head_dim=128, n_tokens=n, cap_len=1024, rot_dim=64, n_pos=2048,
                        k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128, k=0x10000, v=0x20000,
                        row_start=0x1000, pos=0x2000, rope_table=0x4000, s=0x5000, k_codebook=0x6000, v_codebook=0x7000,
                        k_codes=0x8000, v_codes=0x9000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a

def cross(mode, n=5, most=3, dtype=0, **kw):
    return _lib.CrossArgs(decode=dec(mode, out=0x90000000, **kw), dtype=dtype, n_rows=n, max_queries=most, q_row_stride=1024, row_start=0xb000)

calls = [lambda m: L.vqkv_append(ctypes.byref(append(m)), None, None),
         lambda m: L.vqkv_append(ctypes.byref(append(m, 4000)), None, None),
         lambda m: L.vqkv_cross_attn(ctypes.byref(cross(m)), None, None),
         lambda m: L.vqkv_cross_attn(ctypes.byref(cross(m, 90, 30)), None, None),
         lambda m: L.vqkv_cross_attn(ctypes.byref(cross(m, 900, 300)), None, None),
         lambda m: L.vqkv_cross_attn(ctypes.byref(cross(m, 2, 1)), None, None)]
"""


def test_plain_calls_prepare_none_of_their_kernels(run):  # noqa: F811
    out = run(CALLS + """
for mode in range(5):
    assert L.vqkv_decode_attn(ctypes.byref(dec(mode)), None) == 0
print("\\n".join(log()))
""")
    for word in ("cross", "AppendParams", "rows_combine"):
        assert not [x for x in out if word in x], word


def test_every_call_prepares_its_kernels_once(run):  # noqa: F811
    out = run(CALLS + """
prepared = set()
log()
for again in (False, True):
    for m in range(5):
        for call in calls:
            assert call(m) == 0
            lines = log()
            done = {x.split()[1] for x in lines if x.startswith("attribute")}
            prepared |= done
            print(again, len(done))
            for x in lines:
                assert not x.startswith("launch") or "decode_" not in x or x.split()[1] in prepared, x
""")
    assert all(x.split()[1] == "0" for x in out if x.startswith("True"))
    assert sum(int(x.split()[1]) for x in out if x.startswith("False")) > 0


def test_kernels_whose_registers_do_not_cover_their_split_are_refused(run):  # noqa: F811
    run(CALLS + """
fake.fake_registers(64)
for m in range(5):
    assert [call(m) for call in calls] == [0, 4, 4, 4, 4, 0]
    assert L.vqkv_cross_attn_workspace_bytes(ctypes.byref(cross(m))) == 0
    assert L.vqkv_cross_attn_workspace_bytes(ctypes.byref(cross(m, 2, 1))) > 0
""")


def test_workspaces_cover_the_plan(run):  # noqa: F811
    """Sizes are enough for the call, one byte less is refused; fp16's covers bf16's up to the layout."""
    run(CALLS + """
for m in range(5):
    for n, most in ((5, 3), (90, 30), (900, 300), (2, 1), (4096, 4096)):
        for dtype in (0, 2):
            a = cross(m, n, most, dtype)
            need = L.vqkv_cross_attn_workspace_bytes(ctypes.byref(a))
            assert need > 0
            a.decode.workspace_bytes = need
            assert L.vqkv_cross_attn(ctypes.byref(a), None, None) == 0
            a.decode.workspace_bytes = need - 1
            assert L.vqkv_cross_attn(ctypes.byref(a), None, None) == 3
            a.decode.workspace_bytes = need
            a.decode.workspace = 0x8080
            assert L.vqkv_cross_attn(ctypes.byref(a), None, None) == 1
""")
