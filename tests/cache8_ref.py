"""Plain 64-bit forms of the 8-bit cache's operators and of the verification of drafted
tokens, and how far a kernel may be from them."""
import numpy as np
import torch

from gpu_util import DEV
from layer_ref import F32, HALF, TYPES, quantise_rows, rounded


def codes_of(y):
    """Codes and scales of the rows (last axis) of fp32 y."""
    q, s = quantise_rows(y.reshape(-1, y.shape[-1]))
    return q.reshape(y.shape), s.reshape(y.shape[:-1])


def rope8(x, pos, inv_freq, rot, pairs):
    """x [T, heads, D] in 64 bits -> the rotated rows as fp32: sine and cosine are fp32 numbers,
    products and sums 64-bit ones (the products exact), rounded once."""
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    ang = pos.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    c, s = (f(ang).astype(np.float32).astype(np.float64)[:, None] for f in (np.cos, np.sin))
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y.astype(np.float32)


def to_type(y, kind):
    """fp32 numpy values rounded to `kind`, as a tensor on the CPU."""
    return torch.from_numpy(np.ascontiguousarray(y)).to(TYPES[kind])


def pools8(g, pages, page, heads, D, by_head=False, fill=None):
    """(k, v, k_scale, v_scale) on the device: random codes and scales, or codes of `fill` and NaN scales."""
    def shaped(t):
        return t.transpose(1, 2) if by_head else t
    lead = (pages, heads, page) if by_head else (pages, page, heads)
    if fill is None:
        codes = [torch.from_numpy(g.integers(-127, 128, (*lead, D)).astype(np.int8)).to(DEV) for _ in range(2)]
        scales = [torch.from_numpy((g.random(lead) * 0.03 + 0.005).astype(np.float32)).to(DEV) for _ in range(2)]
    else:
        codes = [torch.full((*lead, D), fill, dtype=torch.int8, device=DEV) for _ in range(2)]
        scales = [torch.full(lead, float("nan"), device=DEV) for _ in range(2)]
    return [shaped(t) for t in codes + scales]


#: Weights are scaled so that a row's largest is 2^7 at least, times a power of two that takes the
#: largest scale of a seen value to 1/2 at least: what fp16 loses of one is half of 2^-24 of that.
LOST = 2.0**-31


def attend8(q, ck, sk, cv, sv, p, window, sinks, scale, out_kind, absent=()):
    """One sequence: q [n, Hq, D], codes [L, H, D], scales [L, H] in 64 bits, p [n] the queries'
    places.  Returns (out, its tolerance, lse, its tolerance).

    x = scale s (q . c): products of q and codes are exact, D of them are summed in fp32 (any
    order), then two or three factors: off by dx.  (A bf16 row is taken as fp16 values with the
    row's largest at 2^14 or more: 2^-39 of it may be lost from each.)  A weight exp(x - m) has
    that as a relative error and a few roundings of its own; times s it is rounded to fp16.  The
    sums over L keys are fp32.  One rounding to the output's type."""
    n, Hq, D = q.shape
    L, H = ck.shape[:2]
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
            g = h // (Hq // H)
            kk, vv = ck[at, g] * sk[at, g, None], cv[at, g] * sv[at, g, None]
            x = scale * (kk @ q[i, h])
            m = x.max()
            if m == -np.inf:
                continue
            e = np.exp(x - m)
            l = e.sum()
            out[i, h], lse[i, h] = e @ vv / l, m + np.log(l)
            small = 2.0**-39 * np.abs(q[i, h]).max()
            dx = np.max(abs(scale) * ((D + 4) * F32 * (np.abs(kk) @ np.abs(q[i, h])) + small * np.abs(kk).sum(1))) + 8 * F32
            with np.errstate(invalid="ignore"):
                mass = e @ np.abs(vv) / l
                flat = np.abs(cv[at, g]).sum(0) * sv[at, g].max() / l
                before = mass * (HALF["fp16"] + 2 * dx + 2 * len(at) * F32 + 8 * F32) + LOST * flat
            tol[i, h] = rounded(before, out[i, h], out_kind)
            tol_lse[i, h] = dx + (len(at) + 8) * F32 + 4 * F32 * abs(lse[i, h])
    return out, tol, lse, tol_lse


def probabilities(x, t):
    """p of one row of 64-bit logits, all 0 where the row has no mass."""
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    if m == -np.inf:
        return np.zeros_like(x)
    if not t > 0:
        return (np.arange(len(x)) == np.argmax(x)).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        d = x - m
        e = np.where(x == m, 1.0, np.where(d == -np.inf, 0.0, np.exp(d / t)))
    return e / e.sum()


def verify(logits, start, max_q, tokens, draft, u, temperature):
    """(accepted, next) by the definition, in 64 bits; arguments are numpy arrays."""
    T, V = logits.shape
    accepted, following = [], []
    for b in range(len(start) - 1):
        s0 = min(max(int(start[b]), 0), T)
        n = min(min(max(int(start[b + 1]), s0), T) - s0, max_q)
        t = 1.0 if temperature is None else float(temperature[b])
        done, token = 0, -1
        for i in range(n):
            p = probabilities(logits[s0 + i], t)
            w = p
            if i + 1 < n:
                r = s0 + i + 1
                q = np.zeros(V)
                if draft is not None:
                    with np.errstate(invalid="ignore"):
                        q = np.where(draft[r] > 0, draft[r], 0.0)
                elif 0 <= tokens[r] < V:
                    q[tokens[r]] = 1.0
                if 0 <= tokens[r] < V and u[r] * q[tokens[r]] < p[tokens[r]]:
                    done += 1
                    continue
                left = np.maximum(p - q, 0.0)
                w = left if left.sum() > 0 else p
            if w.sum() > 0:
                sums = np.cumsum(w)
                over = np.nonzero(sums > max(float(u[s0]), 0.0) * sums[-1])[0]
                token = int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])
            break
        accepted.append(done)
        following.append(token)
    return np.array(accepted, np.int32), np.array(following, np.int32)
