"""The decode-step operators in float64 on the CPU, one token, head and position at a time where that is
affordable: head norms with rotation, the paged append, attention over a shared prefix and
per-sequence suffixes, and draft verification. Written from the definitions in include/bpw.h; test
infrastructure only. Arguments are numpy arrays (16-bit types converted to float64 by the caller)."""
import math

import numpy as np


def norm_rope(x, gain, positions, inv_freq, eps, interleaved):
    """x [tokens, heads, dim] -> the normed and rotated heads. gain None: no norm. Also returns, per
    element, |a| + |b| of the normed pair it was made from (what float32 rounding errors scale with)."""
    x = np.array(x, np.float64)
    T, H, D = x.shape
    if gain is not None:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps) * np.asarray(gain, np.float64)
    y, mag = x.copy(), np.abs(x)
    R = 2 * len(inv_freq)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        for t in range(T):
            # the angle reduced exactly: position and frequency as rationals would be overkill, float64 is 29 bits finer
            c, s = math.cos(float(positions[t]) * float(inv_freq[i])), math.sin(float(positions[t]) * float(inv_freq[i]))
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
            mag[t, :, a] = mag[t, :, b] = np.abs(x[t, :, a]) + np.abs(x[t, :, b])
    return y, mag


def rows(pages, page_list, n):
    """Positions 0 .. n-1 of a page list: ([heads, n, dim], usable [n]); a page that is not one of the cache's
    gives unusable zeros."""
    n_pages, H, P, D = pages.shape
    out, ok = np.zeros((H, n, D)), np.zeros(n, bool)
    for i in range(n):
        page = int(page_list[i // P])
        if 0 <= page < n_pages:
            out[:, i] = pages[page, :, i % P]
            ok[i] = True
    return out, ok


def attention(q, k_pages, v_pages, prefix_pages, prefix_len, table, lens, q_starts, max_q, scale):
    """-> out [tokens, q_heads, dim], lse [tokens, q_heads], and the mean of |V| under the same weights (what
    rounding errors scale with); NaN rows for tokens of no sequence."""
    T, Hq, D = q.shape
    Hk, P = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hk
    out, mag = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    pk, ok_p = rows(k_pages, prefix_pages, prefix_len) if prefix_len else (np.zeros((Hk, 0, D)), np.zeros(0, bool))
    pv = rows(v_pages, prefix_pages, prefix_len)[0] if prefix_len else np.zeros((Hk, 0, D))
    for b in range(len(lens)):
        t0 = min(max(int(q_starts[b]), 0), T)
        n = min(min(max(int(q_starts[b + 1]), t0), T) - t0, max_q)
        L = min(max(int(lens[b]), 0), table.shape[1] * P)
        sk, ok_s = rows(k_pages, table[b], L)
        sv, _ = rows(v_pages, table[b], L)
        for j in range(n):
            sees = max(0, L - (n - 1 - j))
            use = np.concatenate([ok_p, ok_s[:sees]])
            for h in range(Hq):
                k = np.concatenate([pk[h // G], sk[h // G, :sees]])[use]
                v = np.concatenate([pv[h // G], sv[h // G, :sees]])[use]
                if not len(k):
                    out[t0 + j, h], mag[t0 + j, h], lse[t0 + j, h] = 0.0, 0.0, -np.inf
                    continue
                s = k @ q[t0 + j, h] * scale
                top = s.max()
                w = np.exp(s - top)
                out[t0 + j, h], mag[t0 + j, h] = w @ v / w.sum(), w @ np.abs(v) / w.sum()
                lse[t0 + j, h] = top + math.log(w.sum())
    return out, lse, mag


def verify(target, draft, tokens, n_draft, accept_u, sample_u):
    """-> out_tokens [sequences, drafts + 1], accepted [sequences]. draft None: certain tokens."""
    B, K1, V = target.shape
    K = K1 - 1
    out, acc = np.full((B, K1), -1, np.int64), np.zeros(B, np.int64)
    for b in range(B):
        most = K if n_draft is None else min(max(int(n_draft[b]), 0), K)
        n = 0
        while n < most:
            x = int(tokens[b, n])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, n, x])
            if not float(accept_u[b, n]) * q < float(target[b, n, x]):
                break
            out[b, n] = x
            n += 1
        acc[b] = n

        def masses(m):
            return np.where(np.isfinite(m) & (m > 0), m, 0.0)

        m = masses(target[b, n].astype(np.float64))
        if n < most:
            if draft is None:
                rest = m.copy()
                if 0 <= int(tokens[b, n]) < V:
                    rest[int(tokens[b, n])] = 0.0
            else:
                with np.errstate(invalid="ignore"):
                    rest = masses(target[b, n].astype(np.float64) - draft[b, n].astype(np.float64))
            if rest.sum() > 0:
                m = rest
        cum = np.cumsum(m)
        if cum[-1] > 0:
            above = np.nonzero((cum > float(sample_u[b]) * cum[-1]) & (m > 0))[0]
            out[b, n] = above[0] if len(above) else np.nonzero(m > 0)[0][-1]
    return out, acc
