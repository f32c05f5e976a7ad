"""TEST INFRASTRUCTURE ONLY -- fp64 CPU oracle of the attention layers' cache.

Plain numpy in float64 on the stored values, one token or row at a time; it
shares no code with the CUDA path.  ``kv_append`` norms, rotates and places
new tokens, ``kv_read`` collects cached ones, ``paged_attention`` is the
softmax over the positions a row sees.  Quantised values are returned as what
they round (``kv_append``), and read as code * scale.
"""
from __future__ import annotations

import math

import numpy as np

CODE_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96


def norm_rotate(x, weight=None, cos=None, sin=None, interleaved=False, eps=1e-6):
    """One head's row x [D]: RMS norm (weight None: none), then the rotation of
    its first 2 len(cos) places (cos None: none)."""
    x = np.asarray(x, np.float64).copy()
    if weight is not None:
        x = x * np.asarray(weight, np.float64) / math.sqrt(float(np.mean(x * x)) + eps)
    if cos is not None:
        half = len(cos)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            u, w = x[a], x[b]
            x[a] = u * cos[i] - w * sin[i]
            x[b] = w * cos[i] + u * sin[i]
    return x


def row_scale(row):
    """The scale of one quantised row."""
    return max(float(np.max(np.abs(row))), AMAX_FLOOR) / CODE_MAX


def kv_append(q, k, v, slots, nslots, positions=None, cos=None, sin=None, interleaved=False,
              q_weight=None, k_weight=None, eps=1e-6):
    """(q_out [T,Hq,D], {slot: (k [Hkv,D], v [Hkv,D])}) before any rounding; padding tokens'
    q_out rows are NaN and their slots absent."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    out, held = np.full(q.shape, np.nan), {}
    for t in range(q.shape[0]):
        slot = int(slots[t])
        if not 0 <= slot < nslots:
            continue
        c = s = None
        if cos is not None:
            p = int(positions[t])
            if not 0 <= p < len(cos):
                continue
            c, s = np.asarray(cos[p], np.float64), np.asarray(sin[p], np.float64)
        for h in range(q.shape[1]):
            out[t, h] = norm_rotate(q[t, h], q_weight, c, s, interleaved, eps)
        held[slot] = (np.stack([norm_rotate(k[t, h], k_weight, c, s, interleaved, eps)
                                for h in range(k.shape[1])]), v[t])
    return out, held


def cached(pool, scale, table_row, ps, pos):
    """Row [Hkv,D] of position pos, or None where there is none."""
    if not 0 <= pos < len(table_row) * ps:
        return None
    page = int(table_row[pos // ps])
    if not 0 <= page < pool.shape[0]:
        return None
    row = np.asarray(pool[page, :, pos % ps], np.float64)
    return row if scale is None else row * np.asarray(scale[page, :, pos % ps], np.float64)[:, None]


def kv_read(pool, scale, table, cu_lens, tokens, starts=None):
    """Rows [tokens,Hkv,D] of one pool."""
    out = np.zeros((tokens, pool.shape[1], pool.shape[3]))
    for b in range(len(table)):
        for i in range(int(cu_lens[b]), min(int(cu_lens[b + 1]), tokens)):
            pos = (0 if starts is None else int(starts[b])) + i - int(cu_lens[b])
            row = cached(pool, scale, table[b], pool.shape[2], pos)
            if row is not None:
                out[i] = row
    return out


def paged_attention(q, k, v, table, lens, k_scale=None, v_scale=None, scale=None, window=0):
    """out [B,T,Hq,D], lse [B,T,Hq], and what error bounds need, [B,T,Hq] each: the largest
    |v| a row sees, the largest sum |q_i k_i| scale over its keys, and how many it sees."""
    q = np.asarray(q, np.float64)
    Bn, T, Hq, D = q.shape
    ps, G = k.shape[2], Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    vmax, smax, seen = np.zeros(q.shape[:3]), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    for b in range(Bn):
        n = int(lens[b])
        rows = {}
        for t in range(T):
            e = n - T + t
            first = max(0, e - window + 1) if window > 0 else 0
            at = []
            for j in range(first, min(e + 1, len(table[b]) * ps)):
                if j not in rows:
                    kr = cached(k, k_scale, table[b], ps, j)
                    rows[j] = None if kr is None else (kr, cached(v, v_scale, table[b], ps, j))
                if rows[j] is not None:
                    at.append(j)
            if not at:
                continue
            K, V = (np.stack([rows[j][i] for j in at]) for i in (0, 1))   # [n, Hkv, D]
            for h in range(Hq):
                kk, vv = K[:, h // G], V[:, h // G]
                s = kk @ q[b, t, h] * scale
                m = s.max()
                p = np.exp(s - m)
                lse[b, t, h] = m + math.log(p.sum())
                out[b, t, h] = p @ vv / p.sum()
                vmax[b, t, h] = np.abs(vv).max()
                smax[b, t, h] = (np.abs(kk) @ np.abs(q[b, t, h])).max() * abs(scale)
                seen[b, t, h] = len(at)
    return out, lse, vmax, smax, seen
