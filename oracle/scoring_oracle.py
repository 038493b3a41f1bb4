"""Plain fp64 forms of the scoring path: RMSNorm with the residual's addition
and e4m3 output, block-scaled e4m3 products, token log-probabilities."""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def bf16_round(x):
    """fp32 values to the nearest bf16 (ties to even), as fp64."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def e4m3_round(x):
    """To the nearest e4m3 number (ties to even), saturated at +-448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.sign(x) * np.minimum(np.rint(a / step) * step, E4M3_MAX)


def e4m3_quotients(v, m):
    """448 v / m to the nearest e4m3 number, ties to even, in whole numbers: v and m
    (m > 0, |v| <= m) have at most 24 significant bits."""
    v, m = np.broadcast_arrays(np.asarray(v, np.float64), np.asarray(m, np.float64))
    fv, ev = np.frexp(np.abs(v))
    fm, em = np.frexp(m)
    num = 448 * np.ldexp(fv, 24).astype(np.int64)  # the quotient is num / den * 2^(ev - em)
    den = np.ldexp(fm, 24).astype(np.int64)
    sh = ev - em
    # leading power of two: 2^e <= quotient
    e = np.floor(np.log2(np.where(num > 0, num / den, 1.0))).astype(np.int64) + sh
    step = np.maximum(e, -6) - 3
    up = np.clip(sh - step, -60, 60)
    num = np.where(up > 0, num << np.clip(up, 0, 25), num)  # (num / den 2^up < 16)
    den = np.where(up < 0, den << np.clip(-up, 0, 38), den)
    n, r = num // den, num % den
    n = n + ((2 * r > den) | ((2 * r == den) & (n % 2 == 1)))
    return np.sign(v) * np.ldexp(n.astype(np.float64), step.astype(np.int32))


def _blocks(k):
    return [(i, min(i + 128, k)) for i in range(0, k, 128)]


def block_scales(x, block_rows):
    """max |x| / 448 of each block_rows x 128 block (1 where it is below 2^-100)."""
    n, k = x.shape
    out = np.ones((-(-n // block_rows), len(_blocks(k))))
    for i in range(out.shape[0]):
        for j, (a, b) in enumerate(_blocks(k)):
            m = np.abs(x[i * block_rows:(i + 1) * block_rows, a:b]).max()
            out[i, j] = m / E4M3_MAX if m >= 2.0 ** -100 else 1.0
    return out


def spread(scale, n, k, block_rows):
    return np.repeat(np.repeat(scale, block_rows, 0)[:n], 128, 1)[:, :k]


def add_rms_norm(x, residual, w, eps, dtype):
    """(y, h) with h rounded to dtype ("fp32" | "bf16") and y in fp64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = (h + np.asarray(residual, np.float64)).astype(np.float32)
        h = bf16_round(h) if dtype == "bf16" else h.astype(np.float64)
    r = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h / r * np.asarray(w, np.float64), h


def add_rms_norm_backward(dy, dh, h, w, eps):
    """(dX, dW) of y = w h / rms(h) plus dh passed through."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, w))
    r = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = dy * w
    dx = g / r - h * (g * h).mean(-1, keepdims=True) / r ** 3
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h / r).sum(0)


def block_matmul(a, sa, b, sb, bias=None):
    """(D, sum of |terms|) of decoded codes a, b and their scales."""
    a = a * spread(np.asarray(sa, np.float64), *a.shape, 1)
    b = b * spread(np.asarray(sb, np.float64), *b.shape, 128)
    d = a @ b.T
    if bias is not None:
        d = d + np.asarray(bias, np.float64)
    return d, np.abs(a) @ np.abs(b).T


def token_logprobs(z, target=None, ignore_index=-100, temperature=1.0, top_k=0):
    """Row by row from the definition; see include/flkl.h for the edge rules."""
    rows, V = z.shape
    out = {"logp": np.zeros(rows), "entropy": np.zeros(rows), "lse": np.zeros(rows),
           "top_logp": np.zeros((rows, top_k)), "top_ids": np.full((rows, top_k), -1)}
    for r in range(rows):
        if target is not None and target[r] == ignore_index:
            continue
        zr = np.asarray(z[r], np.float64)
        bad = np.isnan(zr).any() or np.isposinf(zr).any()
        # NaN first, then by value, ties to the lower index
        order = np.lexsort((np.arange(V), -np.where(np.isnan(zr), 0.0, zr), ~np.isnan(zr)))
        ids = order[:top_k]
        out["top_ids"][r] = ids
        t = int(target[r]) if target is not None else -1
        if bad:
            logq, out["entropy"][r], out["lse"][r] = np.full(V, np.nan), np.nan, np.nan
        elif np.isneginf(zr).all():
            logq, out["lse"][r] = np.full(V, -np.inf), -np.inf
        else:
            u = (zr - zr.max()) / temperature
            ln = np.log(np.exp(u).sum())
            logq = u - ln
            p = np.exp(logq)
            out["entropy"][r] = -(p[p > 0] * logq[p > 0]).sum()
            out["lse"][r] = zr.max() / temperature + ln
        out["top_logp"][r] = logq[ids]
        out["logp"][r] = logq[t] if 0 <= t < V else 0.0
    return out


def token_logprobs_backward(z, target, fwd, dlogp=None, dentropy=None, dtop=None,
                            ignore_index=-100, temperature=1.0):
    """(dz, magnitude of the terms that were added up)."""
    rows, V = z.shape
    dz, mag = np.zeros((rows, V)), np.zeros((rows, V))
    for r in range(rows):
        t = int(target[r]) if target is not None else -1
        if target is not None and t == ignore_index or np.isneginf(z[r]).all():
            continue
        zr = np.asarray(z[r], np.float64)
        u = (zr - zr.max()) / temperature
        logq = u - np.log(np.exp(u).sum())
        p = np.exp(logq)
        lq = np.where(p > 0, logq, 0.0)
        gl = dlogp[r] if dlogp is not None and 0 <= t < V else 0.0
        ge = dentropy[r] if dentropy is not None else 0.0
        gt = dtop[r] if dtop is not None else np.zeros(0)
        ent = fwd["entropy"][r]
        d = -(gl + gt.sum()) * p - ge * p * (lq + ent)
        m = (abs(gl) + np.abs(gt).sum() + abs(ge) * (np.abs(lq) + abs(ent))) * p
        if gl:
            d[t] += gl
            m[t] += abs(gl)
        for j, g in enumerate(gt):
            d[fwd["top_ids"][r][j]] += g
            m[fwd["top_ids"][r][j]] += abs(g)
        dz[r], mag[r] = d / temperature, m / temperature
    return dz, mag
