"""64-bit references of the serving operators, in numpy, from their definitions:
the 4-bit cache page, the three-zone attention over row values, and the page
tables built from request lengths."""
from __future__ import annotations

import numpy as np

LOW, HIGH = 2.0 ** -120, 2.0 ** 126


def quantise(x):
    """(codes int64 [..., D/32, 32], scales float64 [..., D/32]) of rows x [..., D]."""
    v = np.asarray(x, dtype=np.float64)
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    top = np.abs(v).max(-1)
    good = (top >= LOW) & (top < HIGH)              # False for NaN
    want = np.where(good, top, 7.0) / 7
    unit = np.exp2(np.floor(np.log2(want)) - 4)
    s = np.rint(want / unit) * unit
    c = np.where(good[..., None], np.rint(np.where(good[..., None], v, 0.0) / s[..., None]), 0.0).astype(np.int64)
    return c, np.where(good, s, np.where(top < LOW, 0.0, np.nan))


def values(x):
    """The values that rows x stand for once stored."""
    c, s = quantise(x)
    return (c * s[..., None]).reshape(np.shape(x))


def _places(D, is_key):
    n = D // 32
    d = np.arange(D)
    G, y, i, h = d // 32, (d % 32) // 8, (d % 8) // 2, d % 2
    return G, y * 2 * n + (2 * G + h if is_key else h * n + G), i


def pack(rows, is_key):
    """Page bytes of rows [..., ps, D] -> uint8 [..., page_bytes]."""
    rows = np.asarray(rows, dtype=np.float64)
    ps, D = rows.shape[-2:]
    c, s = quantise(rows)
    c = c.reshape(rows.shape) & 15
    G, unit, i = _places(D, is_key)
    units = np.zeros((*rows.shape[:-1], D // 4), dtype=np.uint16)
    for d in range(D):
        units[..., unit[d]] |= (c[..., d] << (4 * i[d])).astype(np.uint16)
    sc = (s.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    flat = np.concatenate([units.reshape(*rows.shape[:-2], -1), sc.reshape(*rows.shape[:-2], -1)], -1)
    return np.ascontiguousarray(flat).view(np.uint8)


def unpack(pages, ps, D, is_key):
    """Row values float64 [..., ps, D] of page bytes [..., page_bytes]."""
    u = np.ascontiguousarray(pages).view(np.uint16)
    units = u[..., :ps * D // 4].reshape(*u.shape[:-1], ps, D // 4)
    sc = (u[..., ps * D // 4:].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    sc = sc.reshape(*u.shape[:-1], ps, D // 32)
    G, unit, i = _places(D, is_key)
    c = (units[..., unit].astype(np.int64) >> (4 * i)) & 15
    return np.where(c > 7, c - 16, c) * sc[..., G]


def sees(k):
    """[R][R]: which step keys a row sees."""
    R = 1 if k == 0 else k + k * k
    m = np.zeros((R, R), dtype=bool)
    for r in range(R):
        if r < max(k, 1):
            m[r, :r + 1] = True
        else:
            j = (r - k) // k + 1
            m[r, :j] = True
            m[r, k + (j - 1) * k:k + j * k] = True
    return m


def attention(q, k_blk, v_blk, prefix_k, prefix_v, k, step_keys=True):
    """One sequence: q [R][Hq][D], k_blk/v_blk [R][Hkv][D], prefix rows [P][Hkv][D].
    Returns (out, lse, spread, mag): spread = sum of p |v| (what a relative error
    of every p can move the output by), mag = the largest sum of |q| |k| scale."""
    R, Hq, D = q.shape
    H = k_blk.shape[1]
    K = np.concatenate([prefix_k, k_blk]) if step_keys else prefix_k
    V = np.concatenate([prefix_v, v_blk]) if step_keys else prefix_v
    mask = np.ones((R, len(K)), dtype=bool)
    if step_keys:
        mask[:, len(prefix_k):] = sees(k)
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf)
    spread, mag = np.zeros((R, Hq, D)), 0.0
    if len(K) == 0:
        return out, lse, spread, mag
    for h in range(Hq):
        g = h // (Hq // H)
        s = np.where(mask, q[:, h] @ K[:, g].T / np.sqrt(D), -np.inf)
        mag = max(mag, float((np.abs(q[:, h]) @ np.abs(K[:, g]).T).max() / np.sqrt(D)))
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        l = p.sum(1, keepdims=True)
        out[:, h] = p @ V[:, g] / l
        spread[:, h] = p @ np.abs(V[:, g]) / l
        lse[:, h] = (top + np.log(l))[:, 0]
    return out, lse, spread, mag


def tables(table, ctx, new, free, count, ps, num_pages, max_rows):
    """(table, count, row_starts, slots, positions, error bits) as tidar_build_tables."""
    BAD_PAGE, BAD_LEN, BAD_COUNT, POOL = 1, 2, 4, 32
    B, width = table.shape
    out, bits = table.copy(), 0
    wants, rows = [], []
    for b in range(B):
        c, m = int(ctx[b]), int(new[b])
        rows.append(max(m, 0))
        wants.append([])
        if c < 0 or m < 0 or c + m > width * ps:
            bits |= BAD_LEN
            continue
        if m == 0:
            continue
        for e in range(c // ps, -(-(c + m) // ps)):
            if 0 <= table[b, e] < num_pages:
                continue
            if table[b, e] == -1 and e >= -(-c // ps):
                wants[b].append(e)
            else:
                bits |= BAD_PAGE
                wants[b] = []
                break
    total, need = sum(rows), sum(map(len, wants))
    ok = True
    if not 0 <= count <= len(free) or need > count:
        bits, ok = bits | POOL, False
    if total > max_rows:
        bits, ok = bits | BAD_COUNT, False
    left = count
    if ok:
        for b in range(B):
            for e in wants[b]:
                left -= 1
                out[b, e] = free[left]
    starts = np.minimum(np.concatenate([[0], np.cumsum(rows)]), max_rows).astype(np.int32)
    slots, pos = np.full(max_rows, -1, dtype=np.int64), np.full(max_rows, -1, dtype=np.int32)
    for b in range(B):
        for r in range(starts[b], starts[b + 1]):
            p = int(ctx[b]) + r - int(starts[b])
            if ctx[b] < 0 or p >= width * ps:
                continue
            pos[r] = p
            page = int(out[b, p // ps])
            if 0 <= page < num_pages:
                slots[r] = page * ps + p % ps
            else:
                bits |= BAD_PAGE
    return out, left, starts, slots, pos, bits
