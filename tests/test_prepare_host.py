"""Which kernels a call prepares on the host, against a stand-in for the CUDA
runtime (fake_cudart.c) that reports a device and launches nothing: a plain
decode neither loads nor depends on the kernels of other calls.  No GPU needed."""
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from vector_quantized_bit_gb300 import _build

PRELUDE = """
import ctypes, sys
sys.modules["torch"] = None          # the library must find the stand-in, not PyTorch's runtime
fake = ctypes.CDLL({fake!r}, mode=ctypes.RTLD_GLOBAL)
fake.fake_log.restype = ctypes.c_char_p
sys.path.insert(0, {root!r})
from vector_quantized_bit_gb300 import _lib
L = _lib.lib()

def dec(mode, **kw):
    a = _lib.DecodeArgs(mode=mode, B=2, Hq=8, Hkv=2, head_dim=128, cap_len=1024, max_seq_len=1024, q=0x1000, k_codes=0x2000,
                        v_codes=0x3000, seq_lens=0x4000, k_codebook=0x5000, v_codebook=0x6000, s=0x7000, num_splits=0,
                        workspace=0x8000, workspace_bytes=1 << 30, out=0x9000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a

def tree(mode, M=8, **kw):
    return _lib.DecodeTreeArgs(decode=dec(mode, **kw), n_queries=M, tree_mask=0xa000)

def mass(mode, M=1, **kw):
    return _lib.DecodeMassArgs(decode=dec(mode, **kw), n_queries=M, mass=0xa000)

def select():
    return _lib.EvictSelectArgs(B=2, Hkv=2, cap_len=1024, max_seq_len=1024, n_keep=100, n_sink=1, n_recent=1, mass=0x1000,
                                seq_lens=0x2000, keep=0x3000, keep_lens=0x4000)

def compact(mode):
    return _lib.CacheCompactArgs(mode=mode, B=2, Hkv=2, cap_len=1024, n_src=64, src_heads=2, k_codes=0x1000, v_codes=0x2000,
                                 seq_lens=0x3000, src=0x4000, counts=0x5000, mass=0x7000)

def log():
    text = fake.fake_log().decode()
    fake.fake_clear()
    return text.splitlines()
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    _build.build()
    d = tmp_path_factory.mktemp("fake")
    fake, version = str(d / "libcudart.so.13"), d / "version"
    version.write_text("libcudart.so.13 { global: *; };\n")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-I", cuda, "-Wl,-soname,libcudart.so.13",
                    f"-Wl,--version-script={version}", os.path.join(ROOT, "tests", "fake_cudart.c"), "-o", fake], check=True)

    def go(body):
        r = subprocess.run([sys.executable, "-c", PRELUDE.format(fake=fake, root=ROOT) + body], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout.splitlines()
    return go


def test_plain_calls_prepare_no_other_calls_kernels(run):
    out = run("""
for mode in range(5):
    assert L.vqkv_decode_workspace_bytes(ctypes.byref(dec(mode))) > 0
    assert L.vqkv_decode_attn(ctypes.byref(dec(mode)), None) == 0
print("\\n".join(log()))
""")
    assert sum(x.startswith("launch") for x in out) >= 5
    for word in ("tree", "mass", "compact", "evict"):
        assert not [x for x in out if word in x], word


def test_plain_calls_do_not_fail_with_other_calls_kernels(run):
    """Kernels whose registers do not cover their split are refused; the calls that do not use them go on."""
    run("""
fake.fake_registers(64)
for mode in range(5):
    assert L.vqkv_decode_attn_tree(ctypes.byref(tree(mode)), None, None) == 4        # VQKV_ERR_CUDA
    assert L.vqkv_decode_tree_workspace_bytes(ctypes.byref(tree(mode))) == 0
    assert L.vqkv_decode_attn_mass(ctypes.byref(mass(mode, M=16)), None, None) == 4
    assert L.vqkv_decode_attn(ctypes.byref(dec(mode)), None) == 0
    assert L.vqkv_decode_attn_mass(ctypes.byref(mass(mode, M=1)), None, None) == 0   # few columns: other kernels
    assert L.vqkv_cache_compact(ctypes.byref(compact(mode)), None, None) == 0
assert L.vqkv_evict_select(ctypes.byref(select()), None) == 0
assert not [x for x in log() if x.startswith("launch") and ("tree_kernel" in x or "mass_tile" in x)]
""")


def test_every_call_prepares_its_kernels_once(run):
    out = run("""
calls = [lambda m: L.vqkv_decode_attn_tree(ctypes.byref(tree(m)), None, None),
         lambda m: L.vqkv_decode_attn_tree(ctypes.byref(tree(m, M=40)), None, None),
         lambda m: L.vqkv_decode_attn_mass(ctypes.byref(mass(m)), None, None),
         lambda m: L.vqkv_decode_attn_mass(ctypes.byref(mass(m, M=16)), None, None),
         lambda m: L.vqkv_cache_compact(ctypes.byref(compact(m)), None, None),
         lambda m: L.vqkv_evict_select(ctypes.byref(select()), None)]
prepared = set()
need = ("decode_tree_kernel", "mass_tile_kernel", "decode_vq", "compact_kernel", "evict_select_kernel")
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
                assert not x.startswith("launch") or not any(w in x for w in need) or x.split()[1] in prepared, x
""")
    assert all(x.split()[1] == "0" for x in out if x.startswith("True"))
    assert sum(int(x.split()[1]) for x in out if x.startswith("False")) > 0
