"""Float64 definition of serving over a paged KV cache held in 8 bits (sa_page_plan,
sa_kv8_write, sa_kv8_fwd), one request, page and query row at a time."""

from __future__ import annotations

import numpy as np

FORMATS = ("e4m3", "int8")
TOP = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The 256 code values: sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 127) == 127 else v
        if c & 128:
            out[c] = -out[c]
    return out


_E4M3 = e4m3_values()


def values(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Code bytes (uint8) -> the numbers they stand for."""
    return _E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def round_codes(x: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code (ties to even), saturated, as bytes.  NaN: 0x7f in e4m3, 0 in integers."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.where(np.isnan(x), 0, np.rint(np.clip(x, -127, 127))).astype(np.int8).view(np.uint8)
    pos = _E4M3[:127]                                   # 0 .. 448, ascending, code = index
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    c = np.where(np.signbit(x), c | 128, c).astype(np.uint8)
    return np.where(np.isnan(x), 127, c).astype(np.uint8)


def scale_for(a: float, fmt: str) -> float:
    """The least power of two s in [2^-60, 2^60] with a <= top * s."""
    s = 2.0 ** -60
    while s < 2.0 ** 60 and a > TOP[fmt] * s:
        s *= 2
    return s


def power_at_least(s: float) -> float:
    r = 2.0 ** -60
    while r < 2.0 ** 60 and r < s:
        r *= 2
    return r


def read_scale(s):
    return np.clip(np.where(np.isnan(s), 0.0, s), 2.0 ** -60, 2.0 ** 60)


def plan(old, new, table, free, n_free, page_size, n_tokens):
    """(table, seq_lens, cu, slots, n_free, n_served)."""
    table = table.copy()
    B, max_pages = table.shape
    lens, cu, slots = np.array(old), np.zeros(B + 1, np.int64), np.full(n_tokens, -1, np.int64)
    left = min(max(n_free, 0), len(free))
    served, tok = 0, 0
    for b in range(B):
        o, n = int(old[b]), int(new[b])
        if o < 0 or n < 0:
            break
        held, pages = -(-o // page_size), -(-(o + n) // page_size)
        if pages > max_pages or tok + n > n_tokens or pages - held > left:
            break
        for j in range(held, pages):
            left -= 1
            table[b, j] = free[left]
        for i in range(n):
            p = int(table[b, (o + i) // page_size])
            if p >= 0:
                slots[tok + i] = p * page_size + (o + i) % page_size
        tok += n
        lens[b] = o + n
        cu[b + 1] = tok
        served += 1
    cu[served + 1:] = tok
    return table, lens, cu, slots, left, served


def write(x, codes, scale, table, lens, cu, fmt):
    """Write x [T, H, d] (float64) into codes [P, ps, H, d] (bytes) and scale [P, H], in place."""
    P, ps, H, _ = codes.shape
    T = x.shape[0]
    for b in range(table.shape[0]):
        t0, n = cu[b], cu[b + 1] - cu[b]
        L = min(max(int(lens[b]), 0), table.shape[1] * ps)
        runs = {}
        for i in range(n):
            pos = L - n + i
            if pos >= 0 and t0 + i < T:
                runs.setdefault(pos // ps, []).append((pos % ps, t0 + i))
        for j, rows in runs.items():
            p = int(table[b, j])
            if not 0 <= p < P:
                continue
            off, ts = rows[0][0], [t for _, t in rows]
            for h in range(H):
                part = x[ts, h]
                a = np.where(np.isfinite(part), np.abs(part), 0.0).max()
                s = scale_for(a, fmt)
                if off:
                    before = read_scale(np.float64(scale[p, h]))
                    s = max(s, power_at_least(before))
                    if s != before:
                        codes[p, :off, h] = round_codes(values(codes[p, :off, h], fmt) * (before / s), fmt)
                codes[p, [r for r, _ in rows], h] = round_codes(part / s, fmt)
                scale[p, h] = s
    return codes, scale


def attend(q, k, v, table, lens, cu, page_size, scale, *, idx=None, block_size=1, topk_len=None, window=None,
           sinks=None):
    """q [T, Hq, d], k / v [P, ps, H, d] (float64, dequantised).  Returns (o, lse, spread, seen): spread [T, Hq, d_v] is
    sum p |v| and seen [T, Hq] the largest scale * sum |q||k| over the visible rows (for error bounds)."""
    T, Hq, d = q.shape
    P, ps, H, dv = v.shape
    G = Hq // H
    o, lse = np.zeros((T, Hq, dv)), np.full((T, Hq), np.inf)
    spread, big = np.zeros((T, Hq, dv)), np.zeros((T, Hq))
    kf, vf = k.reshape(P * ps, H, d), v.reshape(P * ps, H, dv)
    for b in range(table.shape[0]):
        t0, n = cu[b], cu[b + 1] - cu[b]
        L = min(max(int(lens[b]), 0), table.shape[1] * ps)
        for i in range(n):
            t, ta = t0 + i, L - n + i
            for h in range(H):
                if ta < 0:
                    rows = np.zeros(0, np.int64)
                elif idx is None:
                    rows = np.arange(ta + 1)
                else:
                    x = idx[t, h].astype(np.int64)
                    if topk_len is not None:
                        x = x[:max(0, int(topk_len[t, h]))]
                    x = x[x >= 0]
                    rows = (x[:, None] * block_size + np.arange(block_size)).ravel()
                rows = rows[(rows <= ta) & (rows < L)]
                if window is not None:
                    rows = rows[rows >= ta - window]
                page = table[b, rows // ps].astype(np.int64)
                ok = (page >= 0) & (page < P)
                at = page[ok] * ps + rows[ok] % ps
                for g in range(G):
                    hq = h * G + g
                    kk, vv = kf[at, h], vf[at, h]
                    z = scale * (kk @ q[t, hq])
                    e = z if sinks is None else np.append(z, sinks[hq])
                    if e.size == 0:
                        continue
                    m = e.max()
                    l = np.exp(e - m).sum()
                    p = np.exp(z - m) / l
                    o[t, hq] = p @ vv
                    lse[t, hq] = m + np.log(l)
                    spread[t, hq] = p @ np.abs(vv)
                    if z.size:
                        big[t, hq] = abs(scale) * (np.abs(kk) @ np.abs(q[t, hq])).max()
    return o, lse, spread, big
