"""Oracle of the 8-bit paged key/value cache, in numpy float64: page plans, quantised writes,
reads and causal attention, each written from its definition in plain loops."""

from __future__ import annotations

import math

import numpy as np

KV8_QMAX = {"int8": 127.0, "e4m3": 448.0}


def kv8_plan(seq_len, new_len, table, free_pages, n_free, page, tokens):
    """Returns kv_len, cu_q, slots, positions, n_free, table, free_pages, short, bad (whether
    pages or places ran out; whether an input was out of range)."""
    table, cells = table.copy(), free_pages.copy()
    B, width = table.shape
    room = width * page
    pages = lambda n: -(-n // page)  # noqa: E731
    short = False
    bad = not 0 <= n_free <= len(cells)
    top = min(max(n_free, 0), len(cells))
    ok = [not (s < 0 or s > room or (n > 0 and n > room - s)) for s, n in zip(seq_len, new_len)]
    bad = bad or not all(ok)
    for b in range(B):
        if ok[b] and new_len[b] < 0:
            for i in range(pages(int(seq_len[b]))):
                if top < len(cells):
                    cells[top] = table[b, i]
                    top += 1
                else:
                    short = True
    kv, cu, slots, pos = [], [0], [-1] * tokens, [0] * tokens
    left, open_ = top, True  # once a request lacks pages or places, no later one is served
    wanted = 0
    for b in range(B):
        s, n = int(seq_len[b]), max(0, int(new_len[b]))
        at = cu[-1]
        cu.append(at + n)
        if not ok[b]:
            kv.append(min(max(s, 0), room))
            open_ = open_ and cu[-1] <= tokens
            continue
        if new_len[b] < 0:
            kv.append(0)
            continue
        need = pages(s + n) - pages(s)
        wanted += need
        open_ = open_ and wanted <= top and cu[-1] <= tokens
        if not open_:
            kv.append(s)
            short = short or n > 0
            continue
        for i in range(need):
            left -= 1
            table[b, pages(s) + i] = cells[left]
        kv.append(s + n)
        for i in range(n):
            p = int(table[b, (s + i) // page])
            if 0 <= p <= (2 ** 31 - 1) // page:
                slots[at + i] = p * page + (s + i) % page
                pos[at + i] = s + i
            else:
                bad = True
    a = lambda v: np.array(v, dtype=np.int64)  # noqa: E731
    return dict(kv_len=a(kv), cu_q=np.minimum(a(cu), tokens), slots=a(slots), positions=a(pos), n_free=left, table=table,
                free_pages=cells, short=short, bad=bad)


def kv8_scale(amax: float, fmt: str) -> float:
    """The smallest power of two s, exponent in [-120, 122], with amax <= qmax s."""
    e = -120
    while e < 122 and KV8_QMAX[fmt] * math.ldexp(1.0, e) < amax:
        e += 1
    return math.ldexp(1.0, e)


def kv8_round(x, fmt: str):
    """The nearest number the format holds, ties to even, for |x| <= qmax (float64 array)."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.rint(x)
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))  # |x| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, e - 4)
    return np.rint(x / step) * step


def kv8_store(x, s, fmt):
    """What the bytes of x hold under the scale s: x / s rounded, but no further from zero than the
    format's largest number whose product with s is a finite float32."""
    top = float(np.finfo(np.float32).max) / s
    if fmt == "int8":
        top = math.floor(top)
    elif top < 448.0:
        m, e = math.frexp(top)  # three bits behind the leading one
        top = math.ldexp(math.floor(m * 16.0), e - 4)
    return np.clip(kv8_round(np.asarray(x, dtype=np.float64) / s, fmt), -top, top)


def kv8_write(val, scale, x, slots, page, fmt):
    """val [n][H][page][dh] (the numbers the bytes hold) and scale [n][H] after the rows x
    [T][H][dh] went to `slots`; both are copies."""
    val, scale = val.astype(np.float64).copy(), scale.astype(np.float64).copy()
    T, H, _ = x.shape
    t = 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= val.shape[0] * page:
            t += 1
            continue
        n = 1
        while t + n < T and int(slots[t + n]) == s + n and (s + n) % page:
            n += 1
        p, first = s // page, s % page
        for h in range(H):
            rows = x[t:t + n, h].astype(np.float64)
            if not np.isfinite(rows).all() or (first and np.isnan(scale[p, h])):
                scale[p, h] = np.nan
                val[p, h, first:first + n] = 0
                continue
            new = kv8_scale(float(np.abs(rows).max()), fmt)
            if first:
                new = max(new, scale[p, h])
                if new != scale[p, h]:
                    val[p, h, :first] = kv8_store(val[p, h, :first] * scale[p, h], new, fmt)
            scale[p, h] = new
            val[p, h, first:first + n] = kv8_store(rows, new, fmt)
        t += n
    return val, scale


def kv8_read(val, scale, slots, page):
    """[T][H][dh]: scale * value of every slot, zeros outside the cache."""
    out = np.zeros((len(slots), val.shape[1], val.shape[3]))
    for t, s in enumerate(np.asarray(slots).tolist()):
        if 0 <= s < val.shape[0] * page:
            out[t] = val[s // page, :, s % page] * scale[s // page][:, None]
    return out


def kv8_attention(q, K, V, scale=0.0, window=0, softcap=0.0):
    """One request: q [n][Hq][dh], K and V [kv][Hkv][dh] (its cached rows); the last query is
    at the last key. Returns out [n][Hq][dh], sum_j p_j |v_j| of the same shape (what rounding
    errors of the weights scale with) and the largest sum_c |q_c k_c| * scale of a row [n][Hq]
    (what rounding errors of the scores scale with)."""
    n, Hq, dh = q.shape
    kv, Hkv = K.shape[:2]
    f = scale if scale > 0 else 1.0 / math.sqrt(dh)
    out, mass, size = np.zeros((n, Hq, dh)), np.zeros((n, Hq, dh)), np.zeros((n, Hq))
    for i in range(n):
        pos = kv - n + i
        lo = max(0, pos - window + 1) if window > 0 else 0
        if pos < lo:
            continue
        for h in range(Hq):
            k, v = K[lo:pos + 1, h // (Hq // Hkv)], V[lo:pos + 1, h // (Hq // Hkv)]
            z = (k @ q[i, h]) * f
            size[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * f
            if softcap > 0:
                z = softcap * np.tanh(z / softcap)
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h], mass[i, h] = p @ v, p @ np.abs(v)
    return out, mass, size
