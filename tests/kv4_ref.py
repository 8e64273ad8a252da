"""Plain 64-bit references of the norm/rotation, the 4-bit cache and attention over it (numpy, no kernel code)."""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def subnormal(dtype) -> float:
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps


def quantise(x):
    """(codes uint8 [..., D/2], scales float16 [..., D/32]) of values [..., D]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    finite = np.isfinite(b).all(-1)
    with np.errstate(all="ignore"):
        # a 24-bit amax over 7 never rounds to a midpoint of two f16 values through fp32, so this is the direct rounding
        d = np.minimum((np.abs(b).max(-1) / 7).astype(np.float32), np.float32(65504)).astype(np.float16)
        dd = d.astype(np.float64)[..., None]
        q = np.where(dd > 0, np.clip(np.rint(b / dd), -7, 7), 0.0)
    q = np.where(finite[..., None], q, 0.0)
    d = np.where(finite, d, np.float16(np.nan))
    q = (q + 8).astype(np.uint8)
    qs = (q[..., :16] | (q[..., 16:] << 4)).reshape(*x.shape[:-1], x.shape[-1] // 2)
    return qs, d


def values(qs, d):
    """float64 values [..., D] of codes and scales."""
    b = qs.reshape(*qs.shape[:-1], -1, 16)
    q = np.concatenate([b & 15, b >> 4], -1).astype(np.float64) - 8
    return (q * d.astype(np.float64)[..., None]).reshape(*qs.shape[:-1], -1)


def cache_rows(qs, d, pages, offs, h):
    return values(qs[pages, h, offs], d[pages, h, offs])


def rope(x, gamma, eps, cos_sin, positions, interleaved):
    """(result, bound of the pair's terms) for x [T, H, D]; cos_sin None: no rotation."""
    x = np.asarray(x, np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma.astype(np.float64)
    y, size = x.copy(), np.abs(x)
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        row = cos_sin.astype(np.float64)[positions][:, None, :]
        c, s = row[..., :rot // 2], row[..., rot // 2:]
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = np.abs(a * c) + np.abs(b * s)
        size[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, size


def attention(q, k_qs, k_d, v_qs, v_d, table, lens, scale, window):
    """q [B, M, Hq, D] float64. Returns (out, lse, tolerance of fp32 arithmetic for out, and for lse).

    The tolerance. With u = 2^-24: a score is a sum of D products of codes 0..15 with q, less 8 times the sum of q, so
    its error is at most (2 D + 32) u S with S = scale sum_i |q_i| 16 d_i (two roundings a step, also where a matrix
    instruction adds with a step of 2^-23). An error of e in every score moves a softmax weight by a factor within
    exp(+-2e). The weighted sum runs over n tokens, 16 or fewer at a step: at most (n / 4 + 64) u of W = sum p 16 d_v,
    its terms with the offset of 8 in them. lse moves by e and the sum's own roundings, and is stored with u of its size.
    """
    B, M, Hq, D = q.shape
    page, Hkv = k_qs.shape[2], k_qs.shape[1]
    out, lse = np.zeros(q.shape), np.full((B, M, Hq), -math.inf)
    tol, tol_lse = np.zeros(q.shape), np.zeros((B, M, Hq))
    for b in range(B):
        for m in range(M):
            end = int(lens[b]) - M + m + 1
            start = max(0, end - window) if window else 0
            if end <= start:
                continue
            t = np.arange(start, end)
            pages, offs = table[b][t // page], t % page
            n = end - start
            for h in range(Hkv):
                k, v = cache_rows(k_qs, k_d, pages, offs, h), cache_rows(v_qs, v_d, pages, offs, h)
                kd = np.repeat(k_d[pages, h, offs].astype(np.float64), 32, -1)
                vd = np.repeat(v_d[pages, h, offs].astype(np.float64), 32, -1)
                g = Hq // Hkv
                for hq in range(h * g, h * g + g):
                    s = scale * (k @ q[b, m, hq])
                    e = (2 * D + 32) * U * scale * (kd @ np.abs(q[b, m, hq])).max() * 16 + 4 * U * np.abs(s).max()
                    top = s.max()
                    p = np.exp(s - top)
                    out[b, m, hq] = p @ v / p.sum()
                    lse[b, m, hq] = top + np.log(p.sum())
                    tol[b, m, hq] = 2 * e * (p @ np.abs(v)) / p.sum() + (n / 4 + 64) * U * (p @ (16 * vd)) / p.sum()
                    tol_lse[b, m, hq] = e + (n / 4 + 64) * U + 2 * U * abs(lse[b, m, hq])
    return out, lse, tol, tol_lse
