"""Which kernels vqkv_decode_attn_mass launches, by columns and by how much the
batch holds (stand-in CUDA runtime, no GPU needed)."""
import pytest

from tests.test_prepare_host import run  # noqa: F401  (fixture)

FEW, MANY = "decode_mass_kernel", "mass_tile_kernel"


@pytest.mark.parametrize("mode,M,B,L,kernel", [
    (0, 4, 1, 196608, FEW), (0, 5, 1, 500, MANY), (2, 4, 1, 196608, FEW), (3, 3, 1, 196608, FEW), (3, 4, 1, 500, MANY),
    (1, 3, 1, 196608, FEW), (1, 4, 1, 500, MANY),
    # 1.25 bit: 16 columns of much are quicker on the tiles, of little on the decode's kernels
    (4, 3, 1, 196608, FEW), (4, 4, 1, 16384, FEW), (4, 4, 1, 32768, MANY), (4, 4, 1, 196608, MANY), (4, 4, 8, 1000, FEW),
    (4, 4, 32, 1000, MANY),
])
def test_path(run, mode, M, B, L, kernel):
    out = run(f"""
kw = dict(B={B}, Hq=32, Hkv=8, cap_len={L}, max_seq_len={L})
a = mass({mode}, M={M}, **kw)
a.decode.workspace_bytes = 0
assert L.vqkv_decode_attn_mass(ctypes.byref(a), None, None) == 3          # VQKV_ERR_WORKSPACE
a.decode.workspace_bytes = L.vqkv_decode_mass_workspace_bytes(ctypes.byref(a))
log()
assert L.vqkv_decode_attn_mass(ctypes.byref(a), None, None) == 0
print("\\n".join(x for x in log() if x.startswith("launch")))
""")
    assert [x for x in out if kernel in x] and not [x for x in out if (MANY if kernel == FEW else FEW) in x]
