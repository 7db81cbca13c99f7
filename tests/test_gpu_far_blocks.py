"""Paged caches whose blocks lie past 4 GiB of the pools: the same bits as from
a pool that holds those blocks alone."""
import numpy as np
import pytest

from oracle import vqkv_oracle as vo
from tests import helpers as H
from tests.test_gpu_tree import case, tree_masks
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("mode", [0, 1, 2, 3, 4])
def test_blocks_past_four_gibibytes(mode):
    t = H.torch()
    B, Hq, Hkv, M, page, per = 2, 8, 2, 9, 512, 3
    cap = page * per
    r, q, kc, vc, s, kcb, vcb = case(mode, B, Hq, Hkv, M, cap, seed=30 + mode)
    bb = vo.code_bytes(mode, page)
    streams = [H.dev(H.pack_cache_role(mode, role, c, cap)) for role, c in ((0, kc), (1, vc))]
    small = [x.view(B, Hkv, per, bb).transpose(1, 2).reshape(B * per, Hkv, bb).contiguous() for x in streams]
    first = 2 ** 32 // (Hkv * bb) + 2                          # its bytes begin past 2^32
    order = r.permutation(B * per)
    big = []
    for x in small:
        y = t.empty((first + B * per, Hkv, bb), dtype=t.uint8, device="cuda")
        y[first + t.from_numpy(order).cuda()] = x
        big.append(y)
    dq, dm, dl, dk, dv, ds = (H.dev(x) for x in (q, tree_masks(r, B, M, "tree").view(np.int64),
                                                 np.array([cap, 700], dtype=np.int32), kcb, vcb, s))
    results = []
    for pools, table in ((small, np.arange(B * per)), (big, first + order)):
        kw = {"block_table": H.dev(table.reshape(B, per).astype(np.int32)), "block_tokens": page,
              "num_blocks": pools[0].shape[0]}
        mass = t.zeros((B, Hkv, cap), device="cuda")
        outs = []
        ws = _lib.decode_tree_workspace(mode, B, Hq, Hkv, M, cap, cap)
        outs.append(t.empty_like(dq))
        _lib.vqkv_decode_attn_tree(mode, dq, dm, *pools, dl, dk, dv, ds, outs[-1], ws, cap, cap, **kw)
        for n in (1, M):
            ws = _lib.decode_mass_workspace(mode, B, Hq, Hkv, n, cap, cap)
            outs.append(t.empty_like(dq[:, :n]))
            _lib.vqkv_decode_attn_mass(mode, dq[:, :n].contiguous(), *pools, dl, dk, dv, ds, outs[-1], mass, ws, cap, cap, **kw)
        outs.append(mass.clone())
        keep, kl = t.zeros((B, Hkv, 400), dtype=t.int32, device="cuda"), t.zeros(B, dtype=t.int32, device="cuda")
        _lib.vqkv_evict_select(mass, dl, keep, kl, 4, 64)
        err = t.zeros(1, dtype=t.int32, device="cuda")
        _lib.vqkv_cache_compact(mode, *pools, dl, keep, kl, cap, mass=mass, error_flags=err, **kw)
        t.cuda.synchronize()
        assert int(err.item()) == 0
        rows = kw["block_table"].long().flatten()
        results.append(outs + [mass, keep] + [x[rows] for x in pools])
    assert all(t.equal(a, b) for a, b in zip(*results))
