"""Rotary positions (vqkv_rope_table, vqkv_rope) through the C ABI against fp64."""
import numpy as np
import pytest

from tests import rope_reference as R
from vector_quantized_bit_gb300 import _build, _lib

pytestmark = pytest.mark.gpu
TYPES = ("fp16", "bf16", "fp32")


@pytest.fixture(scope="module", autouse=True)
def t():
    _build.build()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def _dtype(t, name):
    return {"fp16": t.float16, "bf16": t.bfloat16, "fp32": t.float32}[name]


def make_table(t, n_pos, rot, **kw):
    out = t.full((n_pos, rot), float("nan"), device="cuda")
    names = {"low": "low_turns", "high": "high_turns", "old": "original_len", "scaling": "scaling"}
    args = {names.get(k, k): v for k, v in kw.items()}
    if "scaling" in args:
        args["scaling"] = ("none", "linear", "base", "wavelength", "ramp").index(args["scaling"])
    _lib.vqkv_rope_table(out, **args)
    return out


@pytest.mark.parametrize("n_pos,rot,kw", [
    (1, 8, {}), (1000, 128, {}), (513, 72, dict(base=500000.0)), (4096, 64, dict(scaling="linear", factor=4.0)),
    (777, 96, dict(scaling="base", factor=8.0)), (3001, 128, dict(scaling="wavelength", factor=8.0, old=8192, base=5e5)),
    (3001, 128, dict(scaling="ramp", factor=32.0, low=1.0, high=32.0, old=4096, amplitude=1.3466)),
    (100, 8, dict(scaling="ramp", factor=4.0, low=1.0, high=32.0, old=64)),           # no pair between the borders
    (100, 16, dict(scaling="ramp", factor=4.0, low=1e-9, high=1.0, old=1 << 20)),     # the ramp ends at the last pair
    (50, 16, dict(scaling="wavelength", factor=0.5, old=100)), (50, 16, dict(amplitude=-2.0)), (50, 16, dict(amplitude=0.0)),
    (100, 8, dict(scaling="linear", factor=1e-6)),                                    # many turns per position
])
def test_table(t, n_pos, rot, kw):
    got = make_table(t, n_pos, rot, **kw).cpu().numpy().astype(np.float64)
    ref = R.table(n_pos, rot, **kw)
    f = R.frequencies(rot, **{k: v for k, v in kw.items() if k != "amplitude"})
    amp = abs(kw.get("amplitude", 1.0))
    # sine and cosine of an eighth of a turn at most: 2 ulp of the result (below 1), the argument's own rounding, the
    # amplitude's product: under 2^-22; the frequencies and the reference's angles in fp64: p f 2^-50
    tol = (2.0 ** -22 + np.arange(n_pos)[:, None] * np.tile(f, 2) * 2.0 ** -50) * amp
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) - tol).max())


def test_far_positions(t):
    n, rot = 1 << 21, 16
    got = make_table(t, n, rot, base=1e6)
    at = np.unique(np.concatenate([np.arange(5), np.random.default_rng(1).integers(0, n, 2000), [n - 1]]))
    a = at[:, None] * R.frequencies(rot, base=1e6)
    d = np.abs(got[t.from_numpy(at).cuda()].cpu().numpy() - np.concatenate([np.cos(a), np.sin(a)], axis=1))
    assert (d <= 2.0 ** -22 + np.tile(a, 2) * 2.0 ** -50).all()
    assert np.isfinite(got.sum().item())


def _views(t, T, H, dt, layout, r):
    """(x values fp64, x view, out view, buffers) of a strides' layout."""
    x = t.from_numpy(r.standard_normal((T, H, 128)).astype(np.float32)).cuda().to(_dtype(t, dt))
    if layout == "contiguous":
        return x, t.full_like(x, float("nan"))
    if layout == "in place":
        y = x.clone()
        return y, y
    if layout == "slices":     # queries and keys side by side in one projection, rotated into another slice of it
        buf = t.full((T, 3 * H + 1, 128), float("nan"), dtype=x.dtype, device="cuda")
        buf[:, :H] = x
        return buf[:, :H], buf[:, 2 * H:3 * H]
    if layout == "head major":
        buf = x.transpose(0, 1).contiguous()
        return buf.transpose(0, 1), t.full((H, T, 128), float("nan"), dtype=x.dtype, device="cuda").transpose(0, 1)
    if layout == "padded":     # rows 132 elements apart
        a, b = (t.full((T, H, 132), float("nan"), dtype=x.dtype, device="cuda") for _ in range(2))
        a[..., :128] = x
        return a[..., :128], b[..., :128]
    one = x[:1, :1].expand(T, H, 128)   # one row for all
    return one, t.full((T, H, 128), float("nan"), dtype=x.dtype, device="cuda")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H,rot,interleaved,transpose,layout", [
    (1, 1, 128, False, False, "contiguous"), (1, 32, 128, False, False, "in place"), (7, 5, 64, True, False, "slices"),
    (7, 5, 64, False, True, "head major"), (33, 17, 8, False, False, "padded"), (33, 17, 8, True, True, "contiguous"),
    (129, 3, 96, False, True, "in place"), (129, 3, 120, True, False, "padded"), (700, 40, 128, False, False, "slices"),
    (700, 40, 72, True, True, "in place"), (900, 65, 128, True, False, "contiguous"), (5, 9, 128, False, False, "expanded"),
])
def test_rope(t, dt, T, H, rot, interleaved, transpose, layout):
    r = np.random.default_rng(T + H + rot)
    x, out = _views(t, T, H, dt, layout, r)
    xv = x.double().cpu().numpy()
    table = make_table(t, 300, rot)
    pos = r.integers(0, 300, T).astype(np.int32)
    pos[0], pos[-1] = 299, 0
    err = t.zeros(1, dtype=t.int32, device="cuda")
    around = out._base.clone() if layout in ("slices", "padded") and out._base is not None else None
    _lib.vqkv_rope(x, t.from_numpy(pos).cuda(), table, out, interleaved=interleaved, transpose=transpose, error_flags=err)
    rows = table.double().cpu().numpy()[pos]
    y, size = R.rotate(xv, rows, interleaved, transpose)
    tol = R.rope_bound(y, size, dt, rot)
    got = out.double().cpu().numpy()
    assert (np.abs(got - y) <= tol).all(), float((np.abs(got - y) - tol).max())
    assert int(err) == 0
    if around is not None:     # nothing else was written
        mark = around.clone()
        view = mark.as_strided(out.shape, out.stride(), out.storage_offset())
        view.copy_(out)
        assert t.equal(mark.nan_to_num(7.0), out._base.nan_to_num(7.0))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_transpose_is_the_gradient(t, dt, interleaved):
    """<w, R(x + d) - R(x)> = <R^T w, d>: R^T w is the gradient of <w, R x>, here against differences."""
    T, H, rot = 50, 6, 96
    r = np.random.default_rng(4)
    table = make_table(t, 5000, rot, amplitude=1.2)
    pos = t.from_numpy(r.integers(0, 5000, T).astype(np.int32)).cuda()
    x, d, w = (t.from_numpy(r.standard_normal((T, H, 128)).astype(np.float32)).cuda().to(_dtype(t, dt)) for _ in range(3))
    x2 = (x.float() + d.float()).to(x.dtype)
    grad, y, y2 = (t.empty_like(x) for _ in range(3))
    _lib.vqkv_rope(w, pos, table, grad, interleaved=interleaved, transpose=True)
    _lib.vqkv_rope(x, pos, table, y, interleaved=interleaved)
    _lib.vqkv_rope(x2, pos, table, y2, interleaved=interleaved)
    rows = table.double().cpu().numpy()[pos.cpu().numpy()]

    def n(a):
        return a.double().cpu().numpy()
    left, right = (n(w) * (n(y2) - n(y))).sum(), (n(grad) * (n(x2) - n(x))).sum()
    # every output is off by its bound at most; the fp64 sums add nothing to speak of
    bound = 0.0
    for rows_in, back, factor in ((x, False, n(w)), (x2, False, n(w)), (w, True, n(x2) - n(x))):
        v, size = R.rotate(n(rows_in), rows, interleaved, back)
        bound += (np.abs(factor) * R.rope_bound(v, size, dt, rot)).sum()
    assert abs(left - right) <= bound
    assert bound <= 8 * R.HALF_STEP[dt] * 4 * np.abs(n(w)).sum()     # and that says something


def test_forward_then_transpose_returns(t):
    """Amplitude 1: the transposed map undoes the rotation, to two fp32 roundings of each."""
    table = make_table(t, 200000, 128, base=500000.0)
    x = t.randn((64, 8, 128), device="cuda")
    pos = t.randint(0, 200000, (64,), device="cuda", dtype=t.int32)
    y = t.empty_like(x)
    _lib.vqkv_rope(x, pos, table, y)
    _lib.vqkv_rope(y, pos, table, y, transpose=True)
    # the table's rows are off unit length by 2^-21 at most, the two maps add 6 2^-24 of the pair's length twice
    length = (x[..., :64] ** 2 + x[..., 64:] ** 2).sqrt().repeat(1, 1, 2)
    assert bool(((y - x).abs() <= 2.0 ** -20 * length).all())


def test_positions_outside_the_table(t):
    table = make_table(t, 10, 64)
    pos = t.tensor([3, -1, 10, 2**31 - 1, -2**31, 9], dtype=t.int32, device="cuda")
    x = t.randn((6, 33, 128), device="cuda")
    out = t.full_like(x, 5.0)
    err = t.zeros(1, dtype=t.int32, device="cuda")
    _lib.vqkv_rope(x, pos, table, out, error_flags=err)
    assert int(err) == _lib.VQKV_DEVERR_POSITION
    assert bool((out[1:5] == 5.0).all()) and bool((out[[0, 5]] != 5.0).any())
    out2 = t.full_like(x, 5.0)
    _lib.vqkv_rope(x, pos, table, out2)      # no error word
    assert t.equal(out, out2)


def test_special_values_stay_in_their_pair(t):
    """NaN and infinities reach their own pair's channels only; those that pass through keep their bits."""
    table = make_table(t, 10, 64)
    for dtype in (t.float16, t.bfloat16, t.float32):
        x = t.randn((2, 3, 128), device="cuda").to(dtype)
        clean = t.empty_like(x)
        pos = t.tensor([1, 7], dtype=t.int32, device="cuda")
        _lib.vqkv_rope(x, pos, table, clean)
        bad = x.clone()
        bad[0, 1, 5] = float("nan")
        bad[1, 2, 100] = float("inf")
        bad[1, 0, 127] = float("nan")
        out = t.empty_like(x)
        _lib.vqkv_rope(bad, pos, table, out)
        same = out == clean
        hit = ~same
        assert sorted(map(tuple, hit.nonzero().tolist())) == [(0, 1, 5), (0, 1, 37), (1, 0, 127), (1, 2, 100)]
        assert bool(out[1, 2, 100].isinf()) and bool(out[0, 1, 37].isnan())


def test_refused_by_the_binding(t):
    table = make_table(t, 10, 64)
    x = t.randn((4, 2, 128), device="cuda").half()
    pos = t.zeros(4, dtype=t.int32, device="cuda")
    out = t.empty_like(x)
    call = _lib.vqkv_rope
    for bad, kind in ((dict(positions=pos.long()), TypeError), (dict(positions=pos[:3]), ValueError),
                      (dict(table=table.double()), TypeError), (dict(table=table.t()), ValueError), (dict(table=table[0]), ValueError),
                      (dict(out=out.float()), TypeError), (dict(out=out[:3]), ValueError), (dict(x=x.int()), TypeError),
                      (dict(x=x[..., :64]), ValueError), (dict(x=x.cpu()), ValueError), (dict(out=out.cpu()), ValueError),
                      (dict(x=x.transpose(0, 2).contiguous().transpose(0, 2)), ValueError),
                      (dict(out=x.flip(0)[:1].expand(4, 2, 128)), _lib.VqkvError), (dict(out=x.view(-1)[4:].as_strided((4, 2, 128), (128, 128, 1))), _lib.VqkvError)):
        kw = {**dict(x=x, positions=pos, table=table, out=out), **bad}
        with pytest.raises(kind):
            call(**kw)
    with pytest.raises(_lib.VqkvError):
        _lib.vqkv_rope_table(t.empty((4, 60), device="cuda"))
    with pytest.raises(TypeError):
        _lib.vqkv_rope_table(t.empty((4, 64), device="cuda", dtype=t.float16))


def test_captured_and_on_another_stream(t):
    table = make_table(t, 100, 128)
    x = t.randn((300, 12, 128), device="cuda").half()
    pos = t.randint(0, 100, (300,), device="cuda", dtype=t.int32)
    want, out = t.empty_like(x), t.zeros_like(x)
    _lib.vqkv_rope(x, pos, table, want)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        _lib.vqkv_rope_table(table)
        _lib.vqkv_rope(x, pos, table, out)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert t.equal(out, want)
    s = t.cuda.Stream()
    out.zero_()
    t.cuda.synchronize()
    _lib.vqkv_rope(x, pos, table, out, stream=s)
    s.synchronize()
    assert t.equal(out, want)


def test_no_tokens(t):
    table = make_table(t, 1, 8)
    x = t.empty((0, 4, 128), device="cuda")
    _lib.vqkv_rope(x, t.empty(0, dtype=t.int32, device="cuda"), table, t.empty_like(x))
    _lib.vqkv_rope_table(t.empty((0, 8), device="cuda"))
