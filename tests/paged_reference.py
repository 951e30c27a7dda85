"""Plain host forms of the paged code cache, in Python integers and 64-bit
floats: what the GPU tests compare with."""
import math

import numpy as np


def blocks_of(n, page):
    return -(-n // page)


def reserve(lens, new, free, count, table, page):
    """(lens, count, cu, slots, table) after the reservation."""
    table = [list(row) for row in table]
    width = len(table[0]) if table else 0
    left = min(max(count, 0), len(free))
    stack, wanted = left, 0
    out, cu, slots = [], [0], []
    for r, (h, n) in enumerate(zip(lens, new)):
        h, n = max(h, 0), max(n, 0)
        cu.append(cu[-1] + n)
        fits = h + n <= width * page
        want = range(blocks_of(h, page), blocks_of(h + n, page)) if fits else ()
        wanted += len(want)
        if not fits or (len(want) and wanted > left):
            out.append(h)
            slots += [-1] * n
            continue
        for b in want:
            stack -= 1
            table[r][b] = free[stack]
        out.append(h + n)
        for p in range(h, h + n):
            pg = table[r][p // page]
            slots.append(pg * page + p % page if pg >= 0 else -1)
    return out, stack, cu, slots, table


def trim(lens, keep, table, page, free, count):
    """(lens, count, free) after the trim."""
    free = list(free)
    top = min(max(count, 0), len(free))
    width = len(table[0]) if table else 0
    out = []
    for r, (h, k) in enumerate(zip(lens, keep)):
        h = min(max(h, 0), width * page)
        k = min(max(k, 0), h)
        out.append(k)
        for b in range(blocks_of(k, page), blocks_of(h, page)):
            if top < len(free):
                free[top] = table[r][b]
                top += 1
    return out, top, free


def rows_of(table_row, codes, books, head, tokens, page):
    """(seen [tokens] bool, rows [tokens, dim]) of one request and head."""
    pages, _, _, ns = codes.shape
    n_c, sub = books.shape[1:]
    book = np.concatenate([books[head], np.zeros((256, sub))])  # codes >= n_c: zero rows
    seen = np.zeros(tokens, bool)
    rows = np.zeros((tokens, ns * sub))
    for t in range(tokens):
        b = t // page
        pg = int(table_row[b]) if b < len(table_row) else -1
        if 0 <= pg < pages:
            seen[t] = True
            code = codes[pg, head, t % page].astype(np.int64)
            code = np.where(code < n_c, code, n_c)
            rows[t] = book[code].reshape(-1)
    return seen, rows


def attention(q, cu, lens, table, k_codes, v_codes, k_books, v_books, window=0, scale=0.0, weight_eps=0.0,
              weight_abs=0.0):
    """(out, lse, out bound, lse bound): the definition in 64 bits, and how far
    an fp32 evaluation may be off.

    With u = 2^-24, kappa = scale log2 e, S_t = kappa q . K^_t, A_t = kappa
    sum |q_i K^_ti|, M = max S_t, T seen tokens and D the head size:
      * S_t is off by d_t <= (D + 4) u A_t (D products and sums in any order, a
        rounded factor kappa, a rounded product with it; an input of 16 bits
        times another is exact in fp32);
      * the weight 2^(S_t - m) is off by a relative e_t <= ln2 (d_t + 2 u (M - S_t + 8)) +
        2^-21 + weight_eps: the subtraction, ex2 (2 ulp, at most 2^-22), the
        rescales and merges (each exp2 and product 2^-22; at most a few), the
        rounding to the type of the product (weight_eps = half its epsilon,
        and weight_abs, half its least step, where the weight is below its
        normal range; the maximum a weight is relative to lies at most 8
        powers of two below the true one, so l >= 1);
      * the sums add (T + 200) u.
    out moves by at most max|V^| (2 mean e + 2 T weight_abs + 4 (T + 200) u), the
    mean over the weights; the log of the sum by max e + T weight_abs + (T + 200) u
    plus its own d and a few roundings of its value."""
    u = 2.0 ** -24
    tokens, hq, dim = q.shape
    hkv = k_codes.shape[1]
    page = k_codes.shape[2]
    group = hq // hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(dim)
    out = np.zeros((tokens, hq, dim))
    lse = np.full((tokens, hq), -np.inf)
    tol, tol_lse = np.zeros((tokens, hq, 1)), np.zeros((tokens, hq))
    for r, length in enumerate(lens):
        new = max(0, cu[r + 1] - cu[r])
        held = max(0, min(length, len(table[r]) * page)) if len(table) else 0
        for h in range(hkv):
            ok, keys = rows_of(table[r], k_codes, k_books, h, held, page)
            _, values = rows_of(table[r], v_codes, v_books, h, held, page)
            for i in range(new):
                p = length - new + i
                t = np.arange(held)
                seen = ok & (t <= p)
                if window:
                    seen &= t > p - window
                if not seen.any():
                    continue
                k, v = keys[seen], values[seen]
                for g in range(group):
                    row, head = cu[r] + i, h * group + g
                    s = scale * (k @ q[row, head])
                    top = s.max()
                    w = np.exp(s - top)
                    total = w.sum()
                    out[row, head] = w @ v / total
                    lse[row, head] = top + math.log(total)
                    kappa = scale / math.log(2)
                    d = (dim + 4) * u * kappa * (np.abs(k) @ np.abs(q[row, head]))
                    e = math.log(2) * (d + 2 * u * ((top - s) / math.log(2) + 8)) + 2.0 ** -21 + weight_eps
                    n = len(s)
                    tol[row, head] = 1.1 * np.abs(v).max() * (2 * (w @ e) / total + 2 * n * weight_abs + 4 * (n + 200) * u)
                    tol_lse[row, head] = 1.1 * (e.max() + n * weight_abs + (n + 200) * u) + 4 * u * abs(lse[row, head])
    return out, lse, tol, tol_lse
