"""Plain fp64 attention over a packed cache with any visibility, for the tests
of the draft-tree and attention-weight calls, and bounds on their errors."""
import math

import numpy as np

from oracle import vqkv_oracle as vo

HALF_STEP = 2.0 ** -11     # fp16 rounding, relative


def rows(codes, cb, s=None):
    """Dequantised rows of one (sequence, KV head), keys in their own domain when s is given."""
    x = vo.dequantize(codes, cb)
    return vo.untransform_keys(x, s) if s is not None else x


def attend(q, kc, vc, kcb, vcb, s, lens, visible, scale=None):
    """q fp16 [B][M][Hq][128]; kc / vc [b][h] code arrays; visible(b, m, L) -> bool [L].

    Returns O fp64 [B][M][Hq][128], the weights summed over queries and heads
    [b][h] -> fp64 [L], and a bound on |dO| of fp16-rounded q' and P (below).
    attend.score_size is the largest scale * sum |q'_c K'_tc| seen.
    """
    attend.score_size = 0.0
    B, M, Hq, D = q.shape
    Hkv = kcb.shape[0]
    g = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    mass = [[None] * Hkv for _ in range(B)]
    for b in range(B):
        L = int(lens[b])
        for h in range(Hkv):
            k, v = rows(kc[b][h][:L], kcb[h], s[h]), rows(vc[b][h][:L], vcb[h])
            kr = vo.dequantize(kc[b][h][:L], kcb[h])
            mass[b][h] = np.zeros(L)
            for m in range(M):
                see = visible(b, m, L)
                if not see.any():
                    continue
                qh = q[b, m, h * g:(h + 1) * g].astype(np.float64)
                sc = np.where(see, scale * (qh @ k.T), -np.inf)
                p = np.exp(sc - sc.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                o = p @ v
                out[b, m, h * g:(h + 1) * g] = o
                mass[b][h] += p.sum(axis=0)
                # Rounding q' moves score t by at most e = 2^-11 sum |q'_c K'_tc| (x scale), and
                # with it each normalised weight by a factor within exp(+-2e); rounding P (against
                # an unrounded sum) by another 2^-11.  dO = sum dp (v - o) + o sum dp, and the
                # result is rounded to fp16 once more.  fp32 sums add a few 2^-20 at these lengths.
                qr = vo.transform_query(qh, s[h])
                size = scale * (np.abs(qr) @ np.abs(kr[see]).T).max(axis=1)
                attend.score_size = max(attend.score_size, float(size.max()))
                e = HALF_STEP * size + 2.0 ** -18
                spread = np.einsum("ht,td->hd", p[:, see], np.abs(v[see]))
                rel = (np.exp(2 * e) - 1 + HALF_STEP + 2.0 ** -16)[:, None]
                tol[b, m, h * g:(h + 1) * g] = rel * (spread + np.abs(o)) + HALF_STEP * np.abs(o) * (1 + rel) + 2.0 ** -24
    return out, mass, tol


def check_output(got, ref, tol):
    """Every element within its bound; the whole within 2e-3 in the 2-norm: rounding
    errors are 2^-11 / sqrt(3) rms each (q' through score errors near 4e-4, P, O), 7e-4
    together for scores of unit size, so 2e-3 leaves a factor near three."""
    assert np.isfinite(got).all()
    d = np.abs(got.astype(np.float64) - ref)
    assert (d <= tol).all(), (float((d - tol).max()), np.unravel_index(int((d - tol).argmax()), d.shape))
    if np.linalg.norm(ref) > 0:
        assert np.linalg.norm(d) <= 2e-3 * np.linalg.norm(ref), np.linalg.norm(d) / np.linalg.norm(ref)


def check_mass(got, before, ref, lens, score_size):
    """Accumulated weights against before + the fp64 weights.

    Scores carry fp32 accuracy: q' = hi + lo to 2^-22, its transform 10
    roundings of 2^-24, the tensor-core sum of 128 products in fp32 up to 40
    steps of 2^-23; together under 2^-17 of scale * sum |q' K'| = score_size.
    A normalised weight moves by at most twice that, plus exp2, the sum l, its
    reciprocal and the sum over columns (under 2^-17 in all), and the
    addition to the old value rounds once.  Rounding errors average out, so
    the 2-norm holds at 1e-5.
    """
    rel = 2 * 2.0 ** -17 * score_size + 2.0 ** -17
    for b in range(got.shape[0]):
        L = int(lens[b])
        for h in range(got.shape[1]):
            want = before[b, h, :L].astype(np.float64) + ref[b][h]
            d = np.abs(got[b, h, :L] - want)
            assert (d <= rel * ref[b][h] + 2.0 ** -23 * np.abs(want) + 1e-37).all(), (b, h, float(d.max()))
            if L:
                assert np.linalg.norm(d) <= 1e-5 * np.linalg.norm(want)
            assert np.array_equal(got[b, h, L:], before[b, h, L:])
