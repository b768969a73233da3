"""Float64 oracle of the paged 4-bit history cache: block tables, head norms with rotation, the
4-bit records and grouped attention over them.  Written from the definitions in include/rocs.h, one
request, row or group at a time; test infrastructure only."""
from __future__ import annotations

import math

import numpy as np

GROUP = 32
SCALE_MIN, SCALE_MAX = 2.0 ** -120, 2.0 ** 120


# ---- block tables -------------------------------------------------------------------------------
def block_tables(past, new, page, free, n_pages, table, rows):
    """(table, kv_len, row_offsets, slots, positions, pages_used, statuses): statuses is the set of
    device statuses ("counts", "index") that the call may set."""
    past = np.zeros(len(new), np.int64) if past is None else np.asarray(past, np.int64)
    table = np.array(table, np.int32)
    max_blocks = table.shape[1]
    kv_len, offsets = np.zeros(len(new), np.int32), np.zeros(len(new) + 1, np.int32)
    slots, positions = np.full(rows, -1, np.int64), np.full(rows, -1, np.int32)
    row = taken = 0
    st = set()
    for r, n in enumerate(int(x) for x in new):
        p = int(past[r])
        offsets[r] = row
        ok = p >= 0 and n >= 0 and p + n <= max_blocks * page
        held = p if 0 <= p <= max_blocks * page else 0
        need = math.ceil((p + n) / page) - math.ceil(p / page) if ok else 0
        fits = need == 0 or taken + need <= len(free)
        if not ok or not fits:
            st.add("counts")
        kv_len[r] = held + n if ok and fits else held
        if ok and fits:
            first = math.ceil(p / page)
            for b in range(need):
                if row + (first + b) * page - p >= rows:
                    break                        # the page begins in a row that is not there
                if 0 <= free[taken + b] < n_pages:
                    table[r, first + b] = free[taken + b]
                else:
                    st.add("index")
            for j in range(n):
                if row + j >= rows:
                    break
                b, o = divmod(p + j, page)
                pg = free[taken + b - first] if b >= first else table[r, b]
                if 0 <= pg < n_pages:
                    slots[row + j], positions[row + j] = int(pg) * page + o, p + j
                else:
                    st.add("index")
            taken += need                        # one that does not fit leaves the pages to those behind it
        row += max(n, 0)
    offsets[len(new)] = row
    if row > rows:
        st.add("counts")
    return table, kv_len, offsets, slots, positions, taken, st


# ---- head norms and rotation ---------------------------------------------------------------------
def angles(max_pos, d_rot, base=10000.0):
    """The cos_sin table [max_pos, d_rot] in fp32: cosines, then sines."""
    a = np.arange(max_pos, dtype=np.float64)[:, None] * base ** (-np.arange(0, d_rot, 2) / d_rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def qk_norm_rope(x, gamma, eps, cos_sin, positions, interleaved):
    """x [rows, H, d] -> (y, scale): y as defined (rows at position -1 are not touched) and, per
    element, the sum of the magnitudes that make it up, which rounding errors are relative to."""
    rows, H, d = x.shape
    rot = cos_sin.shape[1]
    y, mag = np.array(x, np.float64), np.abs(np.array(x, np.float64))
    g = np.ones(d) if gamma is None else np.asarray(gamma, np.float64)
    for i in range(rows):
        if positions[i] < 0 or positions[i] >= cos_sin.shape[0]:
            continue
        n = np.asarray(x[i], np.float64)
        n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps) * g
        y[i], mag[i] = n, np.abs(n)
        c, s = np.asarray(cos_sin[positions[i]], np.float64).reshape(2, -1)
        for t in range(rot // 2):
            a, b = (2 * t, 2 * t + 1) if interleaved else (t, t + rot // 2)
            y[i, :, a], y[i, :, b] = n[:, a] * c[t] - n[:, b] * s[t], n[:, b] * c[t] + n[:, a] * s[t]
            mag[i, :, a] = np.abs(n[:, a] * c[t]) + np.abs(n[:, b] * s[t])
            mag[i, :, b] = np.abs(n[:, b] * c[t]) + np.abs(n[:, a] * s[t])
    return y, mag


# ---- 4-bit records --------------------------------------------------------------------------------
def scale_of(top):
    """The smallest number of four significant bits >= top / 7, within the scale's range."""
    top = np.asarray(top, np.float64)
    m, e = np.frexp(np.where(top > 0, top, 1.0) / 7.0)
    s = np.ceil(m * 16.0) * np.exp2(e - 4.0)
    return np.clip(np.where(top > 0, s, 0.0), SCALE_MIN, SCALE_MAX)


def quantize(x):
    """[..., d] -> (codes 1..15, scales [..., d / 32]); a group with a non-finite value is zeros."""
    g = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, GROUP))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    s = scale_of(np.abs(g).max(-1))
    q = np.sign(g) * np.minimum(7, np.floor(np.abs(g) / s[..., None] + 0.5))
    return (q + 8).astype(np.uint8).reshape(x.shape), s


def dequantize(codes, scales):
    q = codes.astype(np.float64).reshape(codes.shape[:-1] + (-1, GROUP)) - 8
    return (q * np.asarray(scales, np.float64)[..., None]).reshape(codes.shape)


def _bf16_bytes(x):
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    assert not (u & 0xFFFF).any()
    return (u >> 16).astype("<u2")


def record_bytes(page, d):
    return page * d * 9 // 8


def _part(cache, page, d, kv):
    """Views (codes [n_pages, H, page, d / 2], scales as u2 [n_pages, H, page, d / 32]) of the keys
    (kv = 0) or values (1) of a cache [n_pages, H, record] of bytes."""
    half = record_bytes(page, d) // 2
    c = cache[:, :, kv * half:kv * half + page * d // 2].reshape(cache.shape[:2] + (page, d // 2))
    s = cache[:, :, kv * half + page * d // 2:(kv + 1) * half].reshape(cache.shape[:2] + (page, d // 16))
    return c, s


def append(cache, page, K, V, slots):
    """K, V [rows, H, d] into a copy of the cache [n_pages, H, record]."""
    cache = np.array(cache)
    d = K.shape[-1]
    half = record_bytes(page, d) // 2
    for kv, x in enumerate((K, V)):
        codes, scales = quantize(x)
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        sb = _bf16_bytes(scales).view(np.uint8).reshape(scales.shape[:-1] + (-1,))
        for i, s in enumerate(slots):
            if 0 <= s < cache.shape[0] * page:
                pg, o = divmod(int(s), page)
                at = kv * half + o * (d // 2)
                cache[pg, :, at:at + d // 2] = packed[i]
                at = kv * half + page * d // 2 + o * (d // 16)
                cache[pg, :, at:at + d // 16] = sb[i]
    return cache


def values(cache, page, d):
    """(K, V) float64 [n_pages, H, page, d] of a cache of bytes."""
    out = []
    for kv in (0, 1):
        c, s = _part(cache, page, d, kv)
        codes = np.empty(c.shape[:-1] + (d,), np.uint8)
        codes[..., 0::2], codes[..., 1::2] = c & 15, c >> 4
        u = np.ascontiguousarray(s).view("<u2").astype(np.uint32) << 16
        out.append(dequantize(codes, u.view(np.float32)))
    return out


# ---- attention -------------------------------------------------------------------------------------
def attention(Q, H_kv, K, V, table, kv_len, offsets, page, scale, causal):
    """Q [rows, H_q, d], K and V [n_pages, H_kv, page, d] -> (O, mag): O [rows, H_q, d], and the same
    sum with |v|, which errors of the weights are relative to."""
    rows, H_q, d = Q.shape
    O, mag = np.zeros((rows, H_q, d)), np.zeros((rows, H_q, d))
    share = H_q // H_kv
    for r in range(len(kv_len)):
        q0, q1, n = int(offsets[r]), int(offsets[r + 1]), int(kv_len[r])
        if q1 == q0 or n == 0:
            continue
        pages = [int(p) for p in table[r, :(n + page - 1) // page]]
        for h in range(H_q):
            k = K[pages, h // share].reshape(-1, d)[:n]
            v = V[pages, h // share].reshape(-1, d)[:n]
            s = np.asarray(Q[q0:q1, h], np.float64) @ k.T * scale
            if causal:
                s = np.where(np.arange(n)[None] <= n - (q1 - q0) + np.arange(q1 - q0)[:, None], s, -np.inf)
            top = s.max(-1, keepdims=True)
            w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            tot = w.sum(-1, keepdims=True)
            w = w / np.where(tot > 0, tot, 1.0)
            O[q0:q1, h], mag[q0:q1, h] = w @ v, w @ np.abs(v)
    return O, mag
