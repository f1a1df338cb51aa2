"""Plain 64-bit forms of the operators around the weight products, and how far
a kernel may be from them.

A rounding is off by at most half a step: HALF[type] relative to the value,
and TINY[type] where the value is below the type's normal range."""
import numpy as np
import torch

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TYPE_ID = {"fp32": 0, "fp16": 1, "bf16": 2}
HALF = {"fp32": 2.0**-24, "fp16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"fp32": 2.0**-150, "fp16": 2.0**-25, "bf16": 2.0**-134}
F32 = HALF["fp32"]


def f64(t):
    return t.detach().cpu().double().numpy()


def rounded(tol_before, ref, kind):
    """Tolerance of a value that is off by tol_before and then rounded to `kind`."""
    return tol_before + HALF[kind] * (np.abs(ref) + tol_before) + TINY[kind]


def within(got, ref, tol, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any(), \
        f"{what}: infinities in other places"
    fine = np.isfinite(ref)
    err, tol = np.abs(got - ref)[fine], np.broadcast_to(tol, ref.shape)[fine]
    if err.size:
        i = int(np.argmax(err - tol))
        assert err[i] <= tol[i], f"{what}: off by {err[i]:.3e}, {tol[i]:.3e} allowed, at {i} of {err.size}"


def quantise_rows(x):
    """Codes and scales of the rows of fp32 x: scale and quotient are 32-bit numbers."""
    x = x.astype(np.float32)
    s = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
    d = np.where(s > 0, s, 1).astype(np.float64)[:, None]
    r = (x.astype(np.float64) / d).astype(np.float32).astype(np.float64)
    q = np.sign(r) * np.floor(np.abs(r) + 0.5)
    return np.where(s[:, None] > 0, np.clip(q, -127, 127), 0).astype(np.int8), s


def product(q, sx, w, sw, bias, kind):
    """(y, tolerance): the int32 sum becomes fp32 (one rounding), two factors and a bias (one each)."""
    acc = q.astype(np.int64) @ w.astype(np.int64).T
    p = acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    y = p if bias is None else p + bias.astype(np.float64)
    return y, rounded(3 * F32 * np.abs(p) + (0 if bias is None else F32 * np.abs(y)) + 1e-37, y, kind)


def rope(x, pos, inv_freq, rot, pairs, kind):
    """x [T, heads, D] fp64 -> (rotated, tolerance).  Sine and cosine are off by a few
    2^-24 of one turn's radian measure, each product and the sum by one rounding."""
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    ang = pos.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y, tol = x.copy(), np.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    tol[..., a] = tol[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * 12 * F32
    return y, rounded(tol, y, kind)


def attend(q, k, v, p, window, sinks, scale, kind, out_kind, absent=()):
    """One sequence: q [n, Hq, D], k, v [L, H, D] in 64 bits, p [n] the queries' places.
    Returns (out, its tolerance, lse, its tolerance).

    x = scale q.k: D products summed in fp32 (any order), then a factor: off by dx.  A
    weight exp(x - m) has that as a relative error, a few roundings of its own, and one
    rounding to the cache's type; below the type's normal range that is TINY of the largest
    weight's scale.  The sums over L keys are fp32.  One rounding to the output's type."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    tol, tol_lse = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    j = np.arange(L)
    for i in range(n):
        seen = j <= p[i]
        if window > 0:
            seen &= (p[i] - j < window) | (j < sinks)
        seen[[a for a in absent if a < L]] = False
        at = np.nonzero(seen)[0]
        if not len(at):
            continue
        for h in range(Hq):
            kk, vv = k[at, h // (Hq // H)], v[at, h // (Hq // H)]
            x = scale * (kk @ q[i, h])
            m = x.max()
            if m == -np.inf:
                continue
            e = np.exp(x - m)
            l = e.sum()
            out[i, h], lse[i, h] = e @ vv / l, m + np.log(l)
            dx = (D + 3) * F32 * np.max(abs(scale) * (np.abs(kk) @ np.abs(q[i, h]))) + 8 * F32
            with np.errstate(invalid="ignore"):
                mass, flat = e @ np.abs(vv) / l, np.abs(vv).sum(0) / l
                before = mass * (HALF[kind] + 2 * dx + 2 * len(at) * F32 + 8 * F32) + TINY[kind] * flat
            tol[i, h] = rounded(before, out[i, h], out_kind)
            tol_lse[i, h] = dx + (len(at) + 8) * F32 + 4 * F32 * abs(lse[i, h])
    return out, tol, lse, tol_lse
