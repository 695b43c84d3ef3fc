"""64-bit definitions of the serving operators: head norms with rotation,
window attention with first tokens, the 4-bit key/value cache and the block
tables of paged caches.  Written from the formulas in ``include/csa.h``, row by
row; shares no code with the CUDA path."""
import numpy as np


# ------------------------------------------------------- head norms, rotation ---

def qk_norm_rope(x, gamma, pos, sections, R, halves, eps=1e-6, base=10000.0):
    """x [T, heads, c]; gamma None, [c] or [heads, c]; pos [axes, T]."""
    x = np.asarray(x, np.float64)
    c = x.shape[-1]
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    y = x.copy()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for j in range(R // 2):
        ang = np.asarray(pos[axis[j]], np.float64) * base ** (-2.0 * j / R)
        cs, sn = np.cos(ang)[:, None], np.sin(ang)[:, None]
        m, n = (c - R + j, c - R // 2 + j) if halves else (c - R + 2 * j, c - R + 2 * j + 1)
        y[..., m] = x[..., m] * cs - x[..., n] * sn
        y[..., n] = x[..., m] * sn + x[..., n] * cs
    return y


# ------------------------------------------------------------------ attention ---

def visible(t, window, first):
    """Ascending positions that a query at position t sees (window 0: all)."""
    u = np.arange(t + 1)
    return u if window == 0 else u[(u > t - window) | (u < first)]


def attend(q, k, v, scale, sink=None):
    """One query head [c] over rows k, v [m, c]: (output, sum of weight * |v|,
    largest sum |q k|)."""
    if k.shape[0] == 0:
        z = np.zeros(v.shape[-1])
        return z, z, 0.0
    l = scale * (k @ q)
    top = l.max() if sink is None else max(l.max(), sink)
    p = np.exp(l - top)
    p /= p.sum() + (0.0 if sink is None else np.exp(sink - top))
    return p @ v, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max())


def window_attn(q, k, v, window, first, sink, scale, rows=None):
    """q [n_q, nh, c], k, v [n_k, nkv, c] of one sequence -> out, spread
    (sum of weight * |v|) and the largest sum |q k| per (query, head)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    nq, nh, _ = q.shape
    nk, nkv = k.shape[:2]
    g = nh // nkv
    rows = range(nq) if rows is None else rows
    out = np.zeros((len(rows), nh, v.shape[-1]))
    spread, reach = np.zeros_like(out), np.zeros((len(rows), nh, 1))
    for r, i in enumerate(rows):
        u = visible(nk - nq + i, window, first)
        for h in range(nh):
            out[r, h], spread[r, h], reach[r, h] = attend(
                q[i, h], k[u, h // g], v[u, h // g], scale, None if sink is None else float(sink[h]))
    return out, spread, reach


# ---------------------------------------------------------------- 4-bit cache ---

_E4M3 = None


def e4m3_table():
    """The 127 non-negative finite E4M3 values, ascending (code = index)."""
    global _E4M3
    if _E4M3 is None:
        e, m = np.divmod(np.arange(127), 8)
        _E4M3 = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return _E4M3


def nearest_even(x, values):
    """Index of the value nearest to each x, the even index between two."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo, up = x - values[hi - 1], values[hi] - x
    return np.where((up < lo) | ((up == lo) & (hi % 2 == 0)), hi, hi - 1)


def quantise(row):
    """One row [c] -> (codes -7..7, E4M3 scale codes [c/16], E)."""
    row = np.asarray(row, np.float64)
    c = row.shape[0]
    if not np.all(np.isfinite(row)):
        return np.zeros(c, np.int64), np.zeros(c // 16, np.int64), 255
    top = np.abs(row).max()
    field = 0 if top < 2.0 ** -126 else int(np.floor(np.log2(top))) + 127
    E = min(max(field - 10, 1), 254)
    r = 2.0 ** (E - 127)
    grp = row.reshape(-1, 16)
    s = nearest_even(np.abs(grp).max(1) / (7 * r), e4m3_table())
    step = e4m3_table()[s][:, None] * r
    code = np.where(step > 0, np.rint(grp / np.where(step > 0, step, 1.0)), 0)
    return np.clip(code, -7, 7).astype(np.int64).reshape(c), s, E


def dequantise(codes, s, E):
    r = np.nan if E == 255 else 2.0 ** (E - 127)
    return (np.asarray(codes, np.float64).reshape(-1, 16) * e4m3_table()[s][:, None] * r).reshape(-1)


def write_row(image, u, c, is_v, codes, s, E):
    """Puts one quantised row of token u into a 16-token image (uint8 [18 c + 32])."""
    t, h, b = u // 4, (u // 2) % 2, u % 2
    slot, D = 8 * h + 2 * t + b, c // 8
    nib = (codes + 8).astype(np.uint8)
    by = nib[0::2] | (nib[1::2] << 4)
    if not is_v:
        image[slot * (c // 2):(slot + 1) * (c // 2)] = by
        image[16 * c + slot * (c // 16):16 * c + (slot + 1) * (c // 16)] = s
    else:
        for i in range(c // 2):
            d = 2 * i
            image[8 * c + h * 32 * D + (d // D) * 4 * D + t * D + ((d % D) // 4) * 4 + 2 * b
                  + (d % 4) // 2] = by[i]
        for g in range(c // 16):
            image[17 * c + g * 16 + u] = s[g]
    image[18 * c + 2 * slot + (1 if is_v else 0)] = E


def read_row(image, u, c, is_v):
    """The values of token u's K or V row."""
    t, h, b = u // 4, (u // 2) % 2, u % 2
    slot, D = 8 * h + 2 * t + b, c // 8
    if not is_v:
        by = image[slot * (c // 2):(slot + 1) * (c // 2)]
        s = image[16 * c + slot * (c // 16):16 * c + (slot + 1) * (c // 16)]
    else:
        d = 2 * np.arange(c // 2)
        by = image[8 * c + h * 32 * D + (d // D) * 4 * D + t * D + ((d % D) // 4) * 4 + 2 * b
                   + (d % 4) // 2]
        s = image[17 * c + np.arange(c // 16) * 16 + u]
    codes = np.stack([by & 15, by >> 4], -1).reshape(-1).astype(np.int64) - 8
    return dequantise(codes, s.astype(np.int64), int(image[18 * c + 2 * slot + (1 if is_v else 0)]))


def kv4_image(cache, table, b, h, u):
    """The image (a view) that holds position u of sequence b, or None."""
    tiles = cache.shape[2]
    j, r = divmod(u, 16 * tiles)
    if u < 0 or j >= table.shape[1] or not 0 <= table[b, j] < cache.shape[0]:
        return None
    return cache[table[b, j], h, r // 16]


def kv4_store(cache, table, pos, k, v, count=None):
    """In place on cache (uint8 [num_blocks, nkv, tiles, bytes])."""
    B, n, nkv, c = k.shape
    for b in range(B):
        if pos[b] < 0:
            continue
        for i in range(n if count is None else min(n, max(0, int(count[b])))):
            u = int(pos[b]) + i
            for h in range(nkv):
                img = kv4_image(cache, table, b, h, u)
                if img is not None:
                    write_row(img, u % 16, c, False, *quantise(k[b, i, h]))
                    write_row(img, u % 16, c, True, *quantise(v[b, i, h]))


def kv4_rows(cache, table, b, h, us, c):
    """K, V [m, c] of the positions us that are there, and r of the V rows."""
    ks, vs, rs = [], [], []
    for u in us:
        img = kv4_image(cache, table, b, h, int(u))
        if img is not None:
            t = int(u) % 16
            ks.append(read_row(img, t, c, False))
            vs.append(read_row(img, t, c, True))
            rs.append(2.0 ** (int(img[18 * c + 2 * (8 * ((t >> 1) & 1) + 2 * (t >> 2) + (t & 1)) + 1]) - 127))
    return np.array(ks).reshape(-1, c), np.array(vs).reshape(-1, c), np.array(rs)


def kv4_decode(q, cache, table, pos, scale, window, first, sink):
    """q [B, nh, c] -> (out, spread, reach) as window_attn, the largest
    max|q| * sum|k| per head, and max_u(p_u r_u) * sum_u |v_u| / r_u."""
    q = np.asarray(q, np.float64)
    B, nh, c = q.shape
    nkv = cache.shape[1]
    g = nh // nkv
    out, reach, far = np.zeros(q.shape), np.zeros((B, nh, 1)), np.zeros((B, nh, 1))
    spread, under = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        if pos[b] < 0:
            continue
        us = visible(int(pos[b]), window, first)
        for h in range(nkv):
            k, v, r = kv4_rows(cache, table, b, h, us, c)
            for x in range(h * g, (h + 1) * g):
                out[b, x], spread[b, x], reach[b, x] = attend(
                    q[b, x], k, v, scale, None if sink is None else float(sink[x]))
                if len(k):
                    far[b, x] = np.abs(q[b, x]).max() * np.abs(k).sum(1).max()
                    l = scale * (k @ q[b, x])
                    p = np.exp(l - l.max())
                    p /= p.sum() + (0.0 if sink is None else np.exp(float(sink[x]) - l.max()))
                    under[b, x] = (p * r).max() * (np.abs(v) / r[:, None]).sum(0)
    return out, spread, reach, far, under


# --------------------------------------------------------------- block tables ---

def blocks_copy(region, src, dst, n=None):
    """In place on region [num_blocks, ...]."""
    old = region.copy()
    for s, d in list(zip(src, dst))[:n]:
        if 0 <= s < len(region) and 0 <= d < len(region):
            region[d] = old[s]


def blocks_fork(table, src, dst, tokens, fresh, block_tokens):
    rows, mb = table.shape
    out = table.copy()
    cs, cd = np.full(len(src), -1), np.full(len(src), -1)
    for i in range(len(src)):
        if not 0 <= dst[i] < rows or dst[i] in list(dst[i + 1:]):
            continue
        out[dst[i]] = -1
        if not 0 <= src[i] < rows:
            continue
        full, part = divmod(max(0, int(tokens[i])), block_tokens)
        full = min(full, mb)
        out[dst[i], :full] = table[src[i], :full]
        if full < mb and part:
            out[dst[i], full] = fresh[i]
            if table[src[i], full] >= 0 and fresh[i] >= 0:
                cs[i], cd[i] = table[src[i], full], fresh[i]
    return out, cs, cd


def _named(rows, num_blocks):
    return sorted({int(v) for v in rows.ravel() if 0 <= v < num_blocks})


def blocks_free(table, seqs, num_blocks):
    out = table.copy()
    gone = sorted({int(s) for s in seqs if 0 <= s < table.shape[0]})
    out[gone] = -1
    kept = set(_named(out, num_blocks))
    freed = [v for v in _named(table[gone], num_blocks) if v not in kept]
    return out, np.array(freed + [-1] * (num_blocks - len(freed))), len(freed)


def blocks_compact(table, num_blocks):
    used = _named(table, num_blocks)
    live = len(used)
    src = [v for v in used if v >= live]
    dst = [v for v in range(live) if v not in set(used)]
    to = {v: v for v in used} | dict(zip(src, dst))
    out = np.array([[to.get(int(v), -1) for v in row] for row in table], np.int64).reshape(table.shape)
    return out, src, dst, live
