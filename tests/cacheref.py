"""Plain 64-bit reference of the cache operators, and the bounds their outputs are held to."""
import math

import numpy as np
import torch

FP8 = torch.float8_e4m3fn


def pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e.to(torch.int32))


def quantise(x):
    """(codes, scale bytes) of bf16 vectors x [..., D] on the CPU, from the definition."""
    x = x.double()
    finite = torch.isfinite(x)
    amax = torch.where(finite, x.abs(), 0.0).amax(-1)
    e = torch.full(amax.shape, -40, dtype=torch.int32)
    for k in range(-39, 121):  # the smallest whole number with amax <= 448 * 2^e
        e = torch.where(amax > 448.0 * math.ldexp(1.0, k - 1), k, e).to(torch.int32)
    y = torch.where(finite, x, math.nan) * pow2(-e)[..., None]
    # nearest e4m3 value, ties to even: steps of 2^(k-3) in [2^k, 2^(k+1)), of 2^-9 below 2^-6
    k = (torch.frexp(torch.where(finite, y, 0.0).abs())[1] - 1).clamp(min=-6)
    step = pow2(k - 3)
    codes = (torch.round(y / step) * step).float().to(FP8)  # exact: already an e4m3 value
    return codes, (e + 127).to(torch.uint8)


def values(codes, scale):
    """The float64 values that a cache stands for (bf16 without scales)."""
    x = codes.double()
    return x if scale is None else x * pow2(scale.int() - 127)[..., None]


def ancestors(parent):
    """[T, T] bool: column j is row t's ancestor or t itself."""
    T = len(parent)
    see = np.zeros((T, T), bool)
    for t in range(T):
        j = t
        while j >= 0:
            see[t, j] = True
            j = parent[j]
    return torch.from_numpy(see)


def attention(q, k, v, lens, k_new=None, v_new=None, parent=None, k_prefix=None, v_prefix=None, ks=None, vs=None,
              kps=None, vps=None, scale=None):
    """(out, lse, tol_out, tol_lse) in float64 on the CPU.

    The bounds, per element.  Scores: products of bf16 (or of bf16 and codes) are exact in float32; summing D of them
    there is off by at most D * 2^-23 * sum|q k| (2^-23 a step: a whole step for each addition, tensor cores
    truncate), and for e4m3 keys a query is held as two e4m3 terms, off by at most 2^-18 of the largest query element
    that shares its tile; with the scaling, the subtraction and the exponential's own error (2^-21 in all, relative to
    1 + |score|), dx bounds the error of an exponent, and every weight is off by a factor within 1 +- 2 dx.  Weights
    are rounded to bf16 for the product with the values: half a step, 2^-8 (e4m3 values: f16 and three e5m2 terms,
    2^-9, and 2^-28 of the largest weight).  The output is rounded to bf16: 2^-8 of its value.  With A = sum p |v| /
    sum p: |error| <= (2^-8 + 4 dx) A + 2^-8 |o|, and 2^-22 A a key for the float32 sums of the values."""
    q = q.double()
    B, T, Hq, D = q.shape
    H = k.shape[2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    e4 = ks is not None or kps is not None
    for b in range(B):
        n = int(lens[b])
        kk, vv = [], []
        if k_prefix is not None:
            kk.append(values(k_prefix, kps))
            vv.append(values(v_prefix, vps))
        kk.append(values(k[b, :n], None if ks is None else ks[b, :n]))
        vv.append(values(v[b, :n], None if vs is None else vs[b, :n]))
        if k_new is not None:
            kk.append(k_new[b].double())
            vv.append(v_new[b].double())
        kk, vv = torch.cat(kk), torch.cat(vv)
        N = kk.shape[0]
        see = torch.ones((T, N), dtype=torch.bool)
        if k_new is not None:
            see[:, N - T:] = ancestors(parent[b].tolist() if parent is not None else list(range(-1, T - 1)))
        if N == 0:
            continue
        for hq in range(Hq):
            h = hq // G
            K, V, Q = kk[:, h], vv[:, h], q[b, :, hq]
            x = (Q @ K.T) * scale
            x = torch.where(see, x, -math.inf)
            mag = torch.where(see, (Q.abs() @ K.abs().T) * scale, 0.0)
            mag = torch.where(torch.isfinite(mag), mag, 0.0)
            dx = D * 2.0 ** -23 * mag.amax(1) + 2.0 ** -21 * (1 + mag.amax(1))
            if e4:
                Kf = torch.where(torch.isfinite(K), K, 0.0)
                dx = dx + scale * 2.0 ** -18 * q.abs().amax() * Kf.abs().sum(1).amax()
            m = x.amax(1, keepdim=True)
            m = torch.where(torch.isfinite(m), m, 0.0)
            p = torch.exp(x - m)
            s = p.sum(1, keepdim=True)
            some = see.any(1)
            # an unseen value does not matter, whatever it is
            o = torch.zeros((T, D), dtype=torch.float64)
            A = torch.zeros((T, D), dtype=torch.float64)
            for t in range(T):
                if some[t]:
                    o[t] = (p[t, see[t]] @ V[see[t]]) / s[t]
                    A[t] = (p[t, see[t]] @ V[see[t]].abs()) / s[t]
            out[b, :, hq] = o
            lse[b, :, hq] = torch.where(some, (m + s.log())[:, 0], -math.inf)
            rel = 2.0 ** -8 + 4 * dx[:, None] + 2.0 ** -22 * N
            tol[b, :, hq] = rel * A + 2.0 ** -8 * o.abs()
            if e4:
                Vf = torch.where(torch.isfinite(V), V, 0.0)
                tol[b, :, hq] += 2.0 ** -28 * N * Vf.abs().amax(0)
            tol_lse[b, :, hq] = 2 * dx + 2.0 ** -22 * N + 2.0 ** -22 * lse[b, :, hq].abs().nan_to_num(0, 0, 0)
    return out, lse, tol, tol_lse


def assert_close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), f"{what}: infinities"
    d = (got - want).abs()[fin]
    over = d > tol[fin]
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} off, worst {float((d / tol[fin].clamp(min=1e-300)).max()):.3g} of the bound"
