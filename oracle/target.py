"""The target's verification pass in plain float64: appending to a paged cache with the head norm and the rotation,
attention of a pass's rows over that cache, and the verification of drafted tokens.

Everything goes row by row (or draft by draft) from the formulas, on numpy arrays; a row's attention takes only the
keys in its view, so nothing outside it can reach the result.
"""
from __future__ import annotations

import numpy as np


def rows_of(n_seqs: int, n_rows: int, row_start=None):
    """[(sequence, first row, rows)]: starts clamped to the call's rows, and none before one ahead of it."""
    if row_start is None:
        per = n_rows // n_seqs if n_seqs else 0
        return [(s, s * per, per) for s in range(n_seqs)]
    at = np.maximum.accumulate(np.clip(np.asarray(row_start, np.int64)[:n_seqs + 1], 0, n_rows))
    return [(s, int(at[s]), int(at[s + 1] - at[s])) for s in range(n_seqs)]


def slot_of(table_row, page_size: int, n_pages: int, p: int):
    """(page, slot) of position p, or None where it is not held."""
    if p < 0 or p >= len(table_row) * page_size:
        return None
    page = int(table_row[p // page_size])
    return (page, p % page_size) if 0 <= page < n_pages else None


def rms_head(x, gain, eps):
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gain


def rotate(x, pos: int, inv_freq, interleaved: bool, scale: float):
    """x [heads][head_dim] at position pos."""
    r = 2 * len(inv_freq)
    cos, sin = np.cos(pos * inv_freq), np.sin(pos * inv_freq)
    i = np.arange(len(inv_freq))
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    y = x.copy()
    y[:, a] = scale * (x[:, a] * cos - x[:, b] * sin)
    y[:, b] = scale * (x[:, a] * sin + x[:, b] * cos)
    return y


def paged_append(k, v, q, table, kv_len, page_size, n_pages, row_start=None, inv_freq=None, interleaved=False,
                 scale=1.0, q_norm=None, k_norm=None, eps=1e-6):
    """({(page, slot): (k' [kv_heads][hd], v)}, q' or None, held rows): the new rows' values before any rounding."""
    k, v = np.asarray(k, np.float64), np.asarray(v, np.float64)
    q_out = None if q is None else np.array(q, np.float64)
    slots, touched = {}, []
    for s, a, n in rows_of(len(kv_len), len(k), row_start):
        for i in range(n):
            p = int(kv_len[s]) - n + i
            kk = k[a + i]
            if k_norm is not None:
                kk = rms_head(kk, k_norm, eps)
            if inv_freq is not None:
                kk = rotate(kk, p, inv_freq, interleaved, scale)
            if q is not None:
                qq = q_out[a + i]
                if q_norm is not None:
                    qq = rms_head(qq, q_norm, eps)
                if inv_freq is not None:
                    qq = rotate(qq, p, inv_freq, interleaved, scale)
                q_out[a + i] = qq
            touched.append(a + i)
            at = slot_of(table[s], page_size, n_pages, p)
            if at is not None:
                slots[at] = (kk, v[a + i])
    return slots, q_out, touched


def paged_attention(q, k_cache, v_cache, table, kv_len, row_start=None, scale=None, window=0):
    """(out, lse, softmax-weighted |v|, touched rows); caches [pages][page_size][kv_heads][hd] in float64."""
    q = np.asarray(q, np.float64)
    n_pages, page_size, kvh, hd = k_cache.shape
    heads = q.shape[1]
    g = heads // kvh
    scale = hd ** -0.5 if scale is None else scale
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full(q.shape[:2], -np.inf)
    touched = []
    for s, a, n in rows_of(len(kv_len), len(q), row_start):
        held = {}
        for i in range(n):
            p = int(kv_len[s]) - n + i
            touched.append(a + i)
            lo = max(0, p - window + 1) if window else 0
            keys = []
            for j in range(lo, p + 1):
                if j not in held:
                    held[j] = slot_of(table[s], page_size, n_pages, j)
                if held[j] is not None:
                    keys.append(held[j])
            if not keys:
                continue
            pg, sl = (np.array(x) for x in zip(*keys))
            for h in range(heads):
                kk, vv = k_cache[pg, sl, h // g], v_cache[pg, sl, h // g]
                with np.errstate(all="ignore"):
                    sc = scale * (kk @ q[a + i, h])
                    m = sc.max()
                    if m == -np.inf:  # scores of -inf alone: nothing to weigh
                        continue
                    e = np.exp(sc - m)
                    out[a + i, h] = (e / e.sum()) @ vv
                    mag[a + i, h] = (e / e.sum()) @ np.abs(vv)
                    lse[a + i, h] = m + np.log(e.sum())
    return out, lse, mag, touched


def _weights(x, temperature):
    """softmax(x / T) (T <= 0 or NaN: all at the first largest); None for a row without any probability."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    if m == -np.inf:
        return None
    if not temperature > 0:
        y = np.zeros_like(x)
        y[int(np.argmax(x))] = 1.0
        return y
    if m == np.inf:
        y = (x == m).astype(np.float64)
    else:
        y = np.exp((x - m) / min(max(float(temperature), 1e-30), 1e30))
    return y / y.sum()


def verify(target, draft_tok, accept_u, sample_u, draft_logits=None, draft_start=None, temperature=None):
    """[(accepted, token, margin)] per sequence and prob per draft.  The margin says how far the numbers that decide
    are from their borders, relative to the probabilities compared: a result of 32-bit sums can differ from this one
    only where it is at that rounding's level."""
    n, d = len(sample_u), len(draft_tok)
    V = np.asarray(target).shape[1]
    prob = np.zeros(d)
    res = []
    for s, a, cnt in rows_of(n, d, draft_start):
        T = 1.0 if temperature is None else float(temperature[s])
        greedy = not T > 0
        acc, margin, rest = cnt, np.inf, None
        for i in range(cnt):
            x = int(draft_tok[a + i])
            p = _weights(target[a + s + i], T)
            px = p[x] if p is not None and 0 <= x < V else 0.0
            q, qx = None, 1.0
            if draft_logits is not None and not greedy:
                q = _weights(draft_logits[a + i], T)
                qx = q[x] if q is not None and 0 <= x < V else 0.0
            prob[a + i] = px / qx if px < qx else float(px > 0)
            if acc < cnt:
                continue
            u = float(accept_u[a + i])
            if not greedy:
                margin = min(margin, abs(u * qx - px) / max(u * qx, px, 1e-300))
            if not u * qx < px:
                acc = i
                rest = p
                if p is not None and not greedy:
                    if draft_logits is not None:
                        rest = np.maximum(p - (q if q is not None else 0.0), 0.0)
                    elif 0 <= x < V:
                        rest = p.copy()
                        rest[x] = 0.0
                    if rest.sum() == 0:
                        rest = p
        if acc == cnt:
            rest = _weights(target[a + s + cnt], T)
        if rest is None:
            res.append((acc, -1, margin))
            continue
        c = np.cumsum(rest)
        want = float(sample_u[s]) * c[-1]
        tok = int(np.argmax(c > want)) if (c > want).any() else int(np.nonzero(rest)[0][-1])
        if not greedy and want > 0:
            margin = min(margin, float(np.min(np.abs(c - want))) / c[-1])
        res.append((acc, tok, margin))
    return res, prob
