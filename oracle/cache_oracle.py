"""fp64 definitions of the 8-bit key/value cache operators (TEST
INFRASTRUCTURE ONLY, see the package docstring): the page plan, the quantising
append and the attention over the cache, on NumPy arrays and plain loops.

Layouts as in include/vattn.h; e4m3 caches are held here as the float64 values
of their bytes.
"""
from __future__ import annotations

import math

import numpy as np

SCALE_TOKENS = 16
E_MIN = -40


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

def plan(page_tokens, width, pages, new_tokens, kv_lens, table, free_pages, n_free, max_tokens):
    """One step: returns (status, kv_lens, table, free_pages, n_free, q_starts, slots, result); inputs are left alone."""
    streams = len(new_tokens)
    lens, table, free = list(map(int, kv_lens)), table.copy(), free_pages.copy()

    def stop(status):
        return (status, list(map(int, kv_lens)), table, free_pages.copy(), n_free, [0] * (streams + 1),
                [-1] * max_tokens, [status, 0, n_free, max([0, *map(int, kv_lens)])])

    worst = 0
    for n, old in zip(new_tokens, lens):
        if old < 0 or old > width * page_tokens:
            worst = max(worst, 4)
        elif n >= 0 and old + n > width * page_tokens:
            worst = max(worst, 2)
    if worst:
        return stop(worst)
    stack = [int(x) for x in free[:max(n_free, 0)]]
    for s, n in enumerate(new_tokens):
        if n < 0:
            for j in range(-(-lens[s] // page_tokens)):
                if not 0 <= table[s, j] < pages:
                    return stop(4)
                stack.append(int(table[s, j]))
    if not 0 <= n_free <= pages or len(stack) > pages:
        return stop(4)
    if sum(max(0, int(n)) for n in new_tokens) > max_tokens:
        return stop(3)
    free[:len(stack)] = stack
    need = sum(-(-(old + n) // page_tokens) - -(-old // page_tokens) for n, old in zip(new_tokens, lens) if n >= 0)
    if need > len(stack):
        return stop(1)
    filled = [table[s, old // page_tokens] for s, (n, old) in enumerate(zip(new_tokens, lens)) if n > 0 and old % page_tokens]
    if not all(0 <= x < pages for x in stack[len(stack) - need:] + filled):
        return stop(4)                   # a page to be handed out, or gone on filling
    starts, slots = [0], []
    for s, n in enumerate(new_tokens):
        old, n = lens[s], int(n)
        if n < 0:
            lens[s] = 0
            n = 0
        else:
            lens[s] = old + n
        for p in range(old, old + n):
            if p % page_tokens == 0:
                table[s, p // page_tokens] = stack.pop()
            slots.append(int(table[s, p // page_tokens]) * page_tokens + p % page_tokens)
        starts.append(starts[-1] + n)
    slots += [-1] * (max_tokens - len(slots))
    return (0, lens, table, free, len(stack), starts, slots, [0, starts[-1], len(stack), max([0, *lens])])


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def round_e4m3(x):
    """Nearest e4m3 value (ties to even) of float64 x with |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.abs(x))
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.rint(x / step) * step


def scale_exponent(absmax):
    """Smallest e >= E_MIN with absmax <= 448 * 2^e, by trial."""
    e = E_MIN
    while absmax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(k, v, slots, kc, vc, ks, vs):
    """k, v float64 [n, heads, d]; kc, vc the values of the cache's bytes [pages, heads, page_tokens, d]; returns new arrays.
    Lists that come back to a block raise ValueError."""
    kc, vc, ks, vs = kc.copy(), vc.copy(), ks.copy(), vs.copy()
    n, heads, _ = k.shape
    page_tokens = kc.shape[2]
    i, met = 0, set()
    while i < n:
        if slots[i] < 0:
            i += 1
            continue
        if slots[i] // SCALE_TOKENS in met:
            raise ValueError(f"slot {slots[i]}: the list comes back to its block")
        met.add(slots[i] // SCALE_TOKENS)
        j = i + 1
        while j < n and slots[j] == slots[j - 1] + 1 and slots[j] % SCALE_TOKENS:
            j += 1
        page, row = divmod(slots[i], page_tokens)
        blk, held = divmod(row, SCALE_TOKENS)
        r0 = blk * SCALE_TOKENS
        for h in range(heads):
            good = [np.isfinite(k[t, h]).all() and np.isfinite(v[t, h]).all() for t in range(i, j)]
            for x, c, s, is_k in ((k, kc, ks, True), (v, vc, vs, False)):
                e = max([scale_exponent(np.abs(x[t, h]).max()) if g else E_MIN for t, g in zip(range(i, j), good)])
                if held:
                    e = max(e, int(math.log2(s[page, h, blk])))
                    c[page, h, r0:row] = round_e4m3(c[page, h, r0:row] * (s[page, h, blk] / 2.0 ** e))
                s[page, h, blk] = 2.0 ** e
                for t, g in zip(range(i, j), good):
                    c[page, h, row + t - i] = round_e4m3(x[t, h] / 2.0 ** e) if g else (math.nan if is_k else 0.0)
                c[page, h, row + j - i:r0 + SCALE_TOKENS] = 0.0
        i = j
    return kc, vc, ks, vs


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def seen(frame, window, length, n):
    """bool [n, length]: which cached tokens each of a stream's n new tokens sees."""
    m = np.zeros((n, length), dtype=bool)
    for i in range(n):
        p = length - n + i
        for j in range(length):
            if frame == 0:
                m[i, j] = True
            elif p >= 0:
                back = p // frame - j // frame
                m[i, j] = back >= 0 and (window == 0 or back < window)
    return m


def dequantise(c, s):
    """[pages, heads, page_tokens, d] values of bytes and their scales -> values."""
    return c * np.repeat(s, SCALE_TOKENS, axis=2)[..., None]


def stream_rows(c, s, table_row, length):
    """[length, heads, d] cached rows of one stream."""
    pt = c.shape[2]
    out = np.zeros((length, c.shape[1], c.shape[3]))
    for p in range(length):
        page = table_row[p // pt]
        out[p] = c[page, :, p % pt] * s[page, :, p % pt // SCALE_TOKENS][:, None]
    return out


def attend(q, k, v, mask, scale):
    """q [n, q_heads, d], k, v [length, kv_heads, d], mask [n, length] ->
    (o, lse, a): a = sum_j p_j |v_j|, what a relative error of the p_j is taken of."""
    n, qh, d = q.shape
    group = qh // k.shape[1]
    o, a, lse = np.zeros((n, qh, d)), np.zeros((n, qh, d)), np.full((n, qh), -math.inf)
    for h in range(qh):
        x = np.where(mask, scale * (q[:, h] @ k[:, h // group].T), -math.inf)
        for i in range(n):
            if not mask[i].any():
                continue
            row = x[i][mask[i]]
            vv = v[:, h // group][mask[i]]
            m = row.max()
            w = np.exp(row - m)
            z = w.sum()
            o[i, h], a[i, h], lse[i, h] = w @ vv / z, w @ np.abs(vv) / z, m + math.log(z)
    return o, lse, a
