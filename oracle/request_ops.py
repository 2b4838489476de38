"""The operators around the 16-bit decode step in float64 on the CPU: causal attention over packed prompts, the 4-bit format of
the paged cache, log probabilities. Written from the definitions in include/bpw.h; test infrastructure only. Arguments are numpy
arrays (16-bit types converted to float64 by the caller)."""
import math

import numpy as np

NUMBERS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def prompt(q, k, v, starts, scale):
    """-> out [tokens, q_heads, dim], lse [tokens, q_heads], and the mean of |v| under the same weights (what rounding errors
    scale with); NaN rows for tokens of no sequence. Each token's own positions alone are looked at."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    for a, b in zip(starts, starts[1:]):
        a, b = min(max(int(a), 0), T), min(max(int(b), 0), T)
        for t in range(a, b):
            for h in range(Hq):
                with np.errstate(invalid="ignore"):
                    s = k[a:t + 1, h // G] @ q[t, h] * scale
                    w = np.exp(s - s.max())
                    x = v[a:t + 1, h // G]
                    out[t, h], mag[t, h] = w @ x / w.sum(), w @ np.abs(x) / w.sum()
                    lse[t, h] = s.max() + math.log(w.sum())
    return out, lse, mag


def to_codes(x):
    """x [..., dim] -> codes (one a byte) [..., dim], power bytes [..., dim / 32], and how near each element is to the border of
    another code, relative to its block's power of two."""
    shape = x.shape
    b = np.array(x, np.float64).reshape(*shape[:-1], shape[-1] // 32, 32)
    codes, power, near = np.zeros(b.shape, np.uint8), np.zeros(b.shape[:-1], np.uint8), np.full(b.shape, np.inf)
    borders = [(NUMBERS[i] + NUMBERS[i + 1]) / 2 for i in range(7)]
    for at in np.ndindex(*b.shape[:-1]):
        row = b[at]
        if not np.isfinite(row).all():
            power[at] = 255
            continue
        most = np.abs(row).max()
        e = -125
        while e < 125 and most > 7 * 2.0 ** e:
            e += 1
        power[at] = e + 127
        a = np.abs(row) / 2.0 ** e
        c = np.zeros(32, np.uint8)
        for i, border in enumerate(borders):
            c += (a > border) | ((a == border) & (i % 2 == 1))  # a border itself goes to the even code
            near[at] = np.minimum(near[at], np.abs(a - border))
        near[at] = np.minimum(near[at], abs(most / 2.0 ** e - 7)) if e > -125 else near[at]
        near[at] = np.minimum(near[at], abs(most / 2.0 ** e - 3.5)) if e > -125 else near[at]
        codes[at] = c + np.where(row < 0, 8, 0)
    return codes.reshape(shape), power, near.reshape(shape)


def from_codes(codes, power):
    """The values that codes (one a byte) and power bytes stand for."""
    b = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32).astype(np.int64)
    unit = np.where(power == 255, np.nan, 2.0 ** (power.astype(np.float64) - 127))
    return (np.where(b >= 8, -1, 1) * NUMBERS[b % 8] * unit[..., None]).reshape(codes.shape)


def unpacked(codes):
    """Bytes of two codes, the lower half first, as codes one a byte."""
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def logprobs(x, tokens, n_top, scale):
    """-> logprobs [rows], entropy [rows], top tokens and their log probabilities [rows, n_top], and what float32 errors scale
    with: the largest scaled distance to the row's largest logit among the entries named."""
    T, V = x.shape
    lp, ent = np.full(T, -np.inf), np.zeros(T)
    top, top_lp = np.full((T, n_top), -1, np.int64), np.full((T, n_top), -np.inf)
    for t in range(T):
        row = x[t]
        bad = np.isnan(row).any() or (row == np.inf).any()
        order = np.lexsort((np.arange(V), np.where(np.isnan(row), np.inf, -row)))
        order = [i for i in order[:n_top + int(np.isnan(row).sum())] if not np.isnan(row[i]) and row[i] > -np.inf][:n_top]
        top[t, :len(order)] = order
        if bad:
            lp[t], ent[t], top_lp[t] = np.nan, np.nan, np.nan
            continue
        if not (row > -np.inf).any():
            continue
        d = scale * (row - row.max())
        p = np.exp(d)
        log_l = math.log(p.sum())
        with np.errstate(invalid="ignore"):
            ent[t] = log_l - np.where(p > 0, p * d, 0.0).sum() / p.sum()
        if 0 <= tokens[t] < V:
            lp[t] = d[tokens[t]] - log_l
        top_lp[t, :len(order)] = d[order] - log_l
    return lp, ent, top, top_lp
