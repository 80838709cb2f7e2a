"""Plain 64-bit forms of the token-by-token operators, on the CPU: the e4m3 cache
(append, attend) and linear attention with a decay for each head (forward,
gradients), each written straight from its definition.  Test infrastructure only.
"""

from __future__ import annotations

import math

import numpy as np

# the 127 magnitudes of e4m3 in code order
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def e4m3_round(x):
    """x (float64) to the nearest e4m3 value, ties to the even code, at most 448."""
    a = np.minimum(np.abs(x), 448.0)
    lo = np.clip(np.searchsorted(E4M3, a, side="right") - 1, 0, 125)
    up, down = E4M3[lo + 1] - a, a - E4M3[lo]
    take = (up < down) | ((up == down) & (lo % 2 == 1))
    return np.where(take, E4M3[lo + 1], E4M3[lo]) * np.sign(x)


def page_scale(amax):
    """The least power of two s, not below 2^-126, with amax <= 448 s; 0 for 0."""
    if amax == 0:
        return 0.0
    e = -126
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, codes, scale, table, lens, n_new, num_pages):
    """x (B, H, T, d) into codes (P, H, page, d) and scale (P, H), float64, in place.
    Bad pages are skipped; returns whether one was met."""
    page, bad = codes.shape[2], False
    for b in range(x.shape[0]):
        if lens[b] < 0 or n_new[b] < 0 or n_new[b] > x.shape[2]:
            bad = True
            continue
        at, end = int(lens[b]), int(lens[b] + n_new[b])
        while at < end:
            s0 = at % page
            s1 = min(page, s0 + end - at)
            entry = at // page
            p = int(table[b, entry]) if entry < table.shape[1] else -1
            if 0 <= p < num_pages:
                for h in range(x.shape[1]):
                    rows = x[b, h, at - int(lens[b]):at - int(lens[b]) + s1 - s0]
                    s = page_scale(float(np.abs(rows).max()))
                    old = scale[p, h] if s0 else 0.0
                    s = max(s, old)
                    if s0 and 0 < old < s:
                        codes[p, h, :s0] = e4m3_round(codes[p, h, :s0] * (old / s))
                    codes[p, h, s0:s1] = e4m3_round(rows / s) if s else 0.0
                    scale[p, h] = s
            else:
                bad = True
            at += s1 - s0
    return bad


def attend(q, k8, v8, ks, vs, table, lens, q_lens, causal, scale):
    """(o, lse, weight) with weight = sum_j p_j |v_j|, what roundings of the
    probabilities act on, and the largest sum |q k| scale of each row; rows past
    q_lens NaN.  Keys in bad pages are not seen."""
    B, Hq, T, d = q.shape
    P, Hkv, page = k8.shape[:3]
    o = np.full(q.shape, np.nan)
    w, mag = np.zeros(q.shape), np.zeros((B, Hq, T))
    lse = np.full((B, Hq, T), np.nan)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        nq = min(max(int(q_lens[b]), 0), T)
        pos = np.arange(n)
        ids = np.asarray(table[b], dtype=np.int64)[pos // page] if n else np.zeros(0, np.int64)
        good = (ids >= 0) & (ids < P)
        ids, slots = ids[good], pos[good] % page
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            k = k8[ids, hk, slots] * ks[ids, hk][:, None]
            v = v8[ids, hk, slots] * vs[ids, hk][:, None]
            for t in range(nq):
                see = pos[good] < (n - (nq - 1 - t) if causal else n)
                if not see.any():
                    o[b, h, t], lse[b, h, t] = 0.0, -np.inf
                    continue
                x = k[see] @ q[b, h, t] * scale
                m = x.max()
                p = np.exp(x - m)
                lse[b, h, t] = m + math.log(p.sum())
                p /= p.sum()
                o[b, h, t] = p @ v[see]
                w[b, h, t] = p @ np.abs(v[see])
                mag[b, h, t] = (np.abs(k[see]) @ np.abs(q[b, h, t])).max() * scale
    return o, lse, w, mag


def decay_forward(q, k, v, log_decay, state, lens, scale):
    """(o, state): S <- g S + k v^T, o = scale q S, token by token; rows of o past
    lens NaN."""
    B, H, N, d = q.shape
    g = np.exp(log_decay)
    o, out = np.full(q.shape, np.nan), np.array(state, dtype=np.float64)
    for b in range(B):
        for h in range(H):
            S = out[b, h].copy()
            for t in range(int(lens[b])):
                S = g[h] * S + np.outer(k[b, h, t], v[b, h, t])
                o[b, h, t] = scale * (q[b, h, t] @ S)
            out[b, h] = S
    return o, out


def decay_backward(q, k, v, log_decay, dout, state, dstate, lens, scale):
    """Gradients of sum(o dout) + sum(state_out dstate); rows past lens NaN."""
    B, H, N, d = q.shape
    g = np.exp(log_decay)
    dq, dk, dv = (np.full(q.shape, np.nan) for _ in range(3))
    ds = np.array(dstate, dtype=np.float64)
    for b in range(B):
        for h in range(H):
            S, n = np.array(state[b, h], dtype=np.float64), int(lens[b])
            for t in range(n):
                S = g[h] * S + np.outer(k[b, h, t], v[b, h, t])
                dq[b, h, t] = scale * (S @ dout[b, h, t])
            G = ds[b, h].copy()
            for t in range(n - 1, -1, -1):
                G = G + scale * np.outer(q[b, h, t], dout[b, h, t])
                dk[b, h, t], dv[b, h, t] = G @ v[b, h, t], k[b, h, t] @ G
                G = g[h] * G
            ds[b, h] = G
    return dq, dk, dv, ds
