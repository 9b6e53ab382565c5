"""Plain implementations of the rotary table, the append to the paged 8-bit
cache and attention, for the tests: fp32 steps in the documented order where
the result is exact (numpy's elementwise operations round once, to nearest
even), 64 bits for attention, with error bounds that follow from the formulas."""
from __future__ import annotations

import numpy as np
import torch


def bf16(x: np.ndarray) -> np.ndarray:
    """fp32 -> the nearest bf16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()


def rounded(x: np.ndarray, dtype) -> np.ndarray:
    return bf16(x) if dtype == torch.bfloat16 else x.astype(np.float32)


def rope_table(first, n, rot, theta, factor=1.0, low=0.0, high=0.0, orig=0, mag=1.0) -> np.ndarray:
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / rot)
    if high > 0:
        b = np.clip((orig * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = (1 - b) * f / factor + b * f
    else:
        f = f / factor
    a = (first + np.arange(n, dtype=np.float64))[:, None] * f
    return mag * np.stack((np.cos(a), np.sin(a)), -1)


def rotate(x: np.ndarray, cs: np.ndarray, pairs: bool) -> np.ndarray:
    """x [T, H, D] fp32, cs [T, rot/2, 2] fp32; every step rounded to fp32."""
    rot = 2 * cs.shape[1]
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    y = x.copy()
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def codes_of(x: np.ndarray, s: np.ndarray) -> np.ndarray:
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, x / s, np.float32(0))
    return np.clip(np.rint(q), -127, 127).astype(np.int8)


def append(codes, scales, x, pages, ctx, cu, limit=None):
    """In place on codes [P, H, ps, D], scales [P, H, nsb]; x [T, H, D] fp32."""
    ps, sb = codes.shape[2], codes.shape[2] // scales.shape[2]
    for b in range(len(ctx)):
        end = ctx[b] + cu[b + 1] - cu[b]
        end = end if limit is None else min(end, limit)
        for s0 in range(ctx[b] // sb * sb, end, sb):
            lo, hi = max(s0, ctx[b]), min(s0 + sb, end)
            if lo >= hi:
                continue
            page, blk, slot = pages[b][s0 // ps], s0 % ps // sb, s0 % ps
            if not 0 <= page < codes.shape[0]:
                continue
            new = x[cu[b] + lo - ctx[b]:cu[b] + hi - ctx[b]].transpose(1, 0, 2)     # [H, n, D]
            scale = np.abs(new).max((1, 2)).astype(np.float32) / np.float32(127)
            if lo > s0:
                old = scales[page, :, blk]
                scale = np.maximum(old, scale)
                held = codes[page, :, slot:slot + lo - s0]
                grown = codes_of(held.astype(np.float32) * old[:, None, None], scale[:, None, None])
                codes[page, :, slot:slot + lo - s0] = np.where((scale != old)[:, None, None], grown, held)
            codes[page, :, slot + lo - s0:slot + hi - s0] = codes_of(new, scale[:, None, None])
            scales[page, :, blk] = scale


def held(codes, scales, pages, lo, hi) -> np.ndarray:
    """Tokens lo .. hi-1 of a sequence as fp32 values [n, H, D]."""
    ps, sb = codes.shape[2], codes.shape[2] // scales.shape[2]
    p = np.arange(lo, hi)
    page, slot = np.asarray(pages)[p // ps], p % ps
    return codes[page, :, slot].astype(np.float32) * scales[page, :, slot // sb][..., None]


def attention(q, k, v, scale, seen, p_step, out_step, q_step=0.0):
    """q [R, D] over k, v [n, D] in 64 bits; seen [R, n] booleans -> (out, lse,
    bound of |out - computed|, bound of |lse - computed|).

    Where the bound comes from: a score's fp32 sum of D products is off by at
    most D 2^-23 sum|q k| (2^-23 a step: the tensor core may cut instead of
    rounding), its scaling and the exponent's argument by some 2^-22 of their
    size, q itself by q_step of the row's largest |q|; a relative change of e
    in every weight moves the result by at most 2 e sum(p |v|) / sum(p); the
    weights are rounded by p_step (half a step) for the second product, weights
    below fp16's or bf16's normal range by an absolute 2^-25 of the largest;
    the sums over n add n 2^-23 of sum(p |v|); the result is rounded by
    out_step. A second-order factor of 1.1 covers products of these."""
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    s = q @ k.T * scale
    sabs = np.abs(q) @ np.abs(k).T * abs(scale)
    n, d = k.shape[0], k.shape[1]
    s_seen = np.where(seen, s, -np.inf)
    any_seen = seen.any(1)
    m = np.where(any_seen, s_seen.max(1, initial=-np.inf), 0.0)
    p = np.exp(s_seen - m[:, None])
    tot = p.sum(1)
    safe = np.where(any_seen, tot, 1.0)
    out = p @ v / safe[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(any_seen, m + np.log(np.where(any_seen, tot, 1.0)), -np.inf)
    top = np.where(seen, sabs, 0.0).max(1, initial=0.0)
    qk = np.abs(q).max(1, initial=0.0) * q_step * np.abs(k).sum(1).max(initial=0.0) * abs(scale)
    e = d * 2.0 ** -23 * top + qk + 2.0 ** -21 * (top + 8.0)
    a = p @ np.abs(v) / safe[:, None]
    vmax = np.abs(v).max(initial=0.0)
    weights = (p_step + 2 * e + n * 2.0 ** -23)[:, None] * a + (n * 2.0 ** -25 * vmax / safe)[:, None]
    bound = 1.1 * (weights + out_step * np.abs(out)) + 1e-38
    lse_bound = 1.1 * (e + n * 2.0 ** -23) + 2.0 ** -22 * np.where(any_seen, np.abs(lse), 0.0) + 2.0 ** -22
    return out, lse, bound, lse_bound
