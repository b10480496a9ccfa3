"""Plain fp64 statement of the paged-cache operators (include/stem.h:
stem_cache_extend, stem_rope, stem_tree_attn), used only by tests.  One
sequence, one token, one head at a time, in numpy; no code is shared with the
CUDA path."""

from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ stem_cache_extend
def extend(table, page_size, num_pages, cache_lens, new_lens, held, free, cursor, max_tokens, parents=None,
           mask_words=0):
    """Returns dict(table, held, cursor, cu, kv, slots, positions, mask, status) with
    status a set of {"bad", "pages"}."""
    table = np.array(table, dtype=np.int64)
    S, max_pages = table.shape
    status = set()
    if not 0 <= cursor <= len(free):
        status.add("bad")
        cursor = min(max(cursor, 0), len(free))
    held = list(held)
    slots, positions = np.full(max_tokens, -1, dtype=np.int64), np.zeros(max_tokens, dtype=np.int64)
    mask = np.zeros((max_tokens, mask_words), dtype=np.uint32)
    cu, kv = [0], []
    for s in range(S):
        c, n = int(cache_lens[s]), int(new_lens[s])
        if c < 0 or n < 0 or not 0 <= held[s] <= max_pages:
            status.add("bad")
        c, n, held[s] = max(c, 0), max(n, 0), min(max(held[s], 0), max_pages)
        if n > max_tokens - cu[-1]:
            status.add("bad")
            n = max_tokens - cu[-1]
        need = -(-(c + n) // page_size)
        if need > max_pages:
            status.add("pages")
            need = max_pages
        for e in range(held[s], need):
            if cursor < len(free):
                page, cursor, held[s] = int(free[cursor]), cursor + 1, held[s] + 1
                if not 0 <= page < num_pages:
                    status.add("bad")
                    page = -1
            else:
                status.add("pages")
                page = -1
            table[s, e] = page
        o = cu[-1]
        above = []
        for i in range(n):
            p = c + i
            page = table[s, p // page_size] if p // page_size < max_pages else -1
            if 0 <= page < num_pages:
                slots[o + i] = page * page_size + p % page_size
            elif p // page_size < int(held[s]):
                status.add("bad")
            if parents is None:
                positions[o + i] = p
                continue
            up = int(parents[o + i])
            if up >= i or up < -1:
                status.add("bad")
                up = -1
            above.append((above[up] if up >= 0 else []) + [i])
            positions[o + i] = c + len(above[i]) - 1
            for j in above[i]:
                if j // 32 < mask_words:
                    mask[o + i, j // 32] |= np.uint32(1 << (j % 32))
                else:
                    status.add("bad")
        cu.append(o + n)
        kv.append(c + n)
    return dict(table=table, held=np.array(held), cursor=cursor, cu=np.array(cu), kv=np.array(kv), slots=slots,
                positions=positions, mask=mask, status=status)


# ------------------------------------------------------------------ stem_rope
def rope_frequencies(rotary, base=1e6, scaling="plain", factor=1.0, original_len=1, beta_fast=32.0, beta_slow=1.0,
                     amplitude=0.0):
    """(radians per position of each pair, amplitude)."""
    j = np.arange(rotary // 2, dtype=np.float64)
    b = base * factor ** (rotary / (rotary - 2)) if scaling == "ntk" else base
    w = np.exp(-2.0 * j / rotary * math.log(b))
    amp = amplitude or 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "yarn":
        pair = lambda turns: rotary * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rotary - 1)
        if low == high:
            high += 0.001
        if high > low:
            t = np.clip((j - low) / (high - low), 0, 1)
        else:  # every pair makes fewer turns than beta_slow, or more than beta_fast
            t = np.full(rotary // 2, 1.0 if pair(beta_slow) <= 0 else 0.0)
        w = w * (1 - t) + w / factor * t
        amp = amplitude or 0.1 * math.log(factor) + 1
    return w, amp


def rope_pairs(rotary, layout):
    j = np.arange(rotary // 2)
    return (j, j + rotary // 2) if layout == "half" else (2 * j, 2 * j + 1)


def rope(x, positions, rotary, layout, **freq):
    """x fp64 [T, H, d] -> (rotated, |a| + |b| of the pair each element came from, times the amplitude)."""
    w, amp = rope_frequencies(rotary, **freq)
    a, b = rope_pairs(rotary, layout)
    y, size = x.copy(), np.abs(x)
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * w
    y[..., a] = amp * (x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang))
    y[..., b] = amp * (x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang))
    size[..., a] = size[..., b] = amp * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


# ------------------------------------------------------------------ stem_tree_attn
def sees(i, j, mask_row):
    """Query i sees new token j."""
    if mask_row is None:
        return j <= i
    return j // 32 < len(mask_row) and bool((int(mask_row[j // 32]) >> (j % 32)) & 1)


def tree_attn(q, k_rows, v_rows, cu, kv_lens, mask=None, scale=0.0):
    """q fp64 [T, Hq, d]; k_rows / v_rows: per sequence the fp64 [kv, Hkv, d] keys
    in order.  Returns out, lse, and per (query, head) what error bounds need:
    sum p |v| / sum p, the largest sum |q||k| scale of a seen key, and max |v|."""
    T, hq, d = q.shape
    sigma = scale or 1.0 / math.sqrt(d)
    out, lse = np.zeros((T, hq, d)), np.full((hq, T), -np.inf)
    absav, qk, vmax = np.zeros((T, hq, d)), np.zeros((T, hq)), np.zeros((T, hq))
    for s in range(len(cu) - 1):
        n, kv = cu[s + 1] - cu[s], int(kv_lens[s])
        ctx = kv - n
        for i in range(n):
            t = cu[s] + i
            keys = [u for u in range(kv) if u < ctx or sees(i, u - ctx, None if mask is None else mask[t])]
            if not keys:
                continue
            for h in range(hq):
                g = h // (hq // k_rows[s].shape[1])
                K, V = k_rows[s][keys, g], v_rows[s][keys, g]
                x = K @ q[t, h] * sigma
                m = x.max()
                p = np.exp(x - m)
                z = p.sum()
                out[t, h] = p @ V / z
                lse[h, t] = m + math.log(z)
                absav[t, h] = p @ np.abs(V) / z
                qk[t, h] = (np.abs(K) @ np.abs(q[t, h])).max() * sigma
                vmax[t, h] = np.abs(V).max()
    return out, lse, dict(absav=absav, qk=qk, vmax=vmax)
