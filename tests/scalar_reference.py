"""Plain host forms of the paged cache in 4 bits: the append in rounded fp32 steps, the
attention in 64 bits with the bounds its fp32 evaluation keeps."""
import math

import numpy as np
import torch

HALF_EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
HALF_STEP = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 0.0}  # half the least step


def encode_rows(x, centroids, signs=None):
    """(codes [.., D], scales [..] in x's dtype) of the rows of x (a CPU tensor)."""
    dtype = x.dtype
    y = x.float().numpy().astype(np.float32)
    dim = y.shape[-1]
    with np.errstate(all="ignore"):
        if signs is not None:
            y = y * signs.astype(np.float32)
            at = np.arange(dim)
            stride = 1
            while stride < dim:
                partner = y[..., at ^ stride]
                y = np.where(at & stride == 0, y + partner, partner - y)
                stride *= 2
            y = y * np.float32(1.0 / math.sqrt(dim))
        width = 1 << (dim - 1).bit_length()
        total = np.zeros((*y.shape[:-1], width), np.float32)
        total[..., :dim] = y * y
        while total.shape[-1] > 1:
            total = total[..., 0::2] + total[..., 1::2]
        total = total[..., 0]
        assert total.dtype == np.float32
        scale = torch.from_numpy(np.sqrt(total / np.float32(dim))).to(dtype)
        scale = torch.where(torch.isfinite(scale.float()), scale, torch.zeros((), dtype=dtype))
        # the largest value of the type whose product with every centroid is not above its largest
        top = torch.finfo(dtype).max
        most = max(1.0, *(abs(float(c)) for c in torch.tensor(list(centroids), dtype=torch.float32).to(dtype)))
        cap = torch.tensor(top / most, dtype=torch.float64).to(dtype)
        while float(cap) * most > top:
            bits = torch.int32 if dtype == torch.float32 else torch.int16
            cap = (cap.view(bits) - 1).view(dtype)  # the next below
        scale = torch.minimum(scale, cap)
        s = scale.float().numpy()[..., None]
        z = np.where(s > 0, y * (np.float32(1) / s), np.float32(0))
        best = np.full(z.shape, np.inf, np.float32)
        code = np.zeros(z.shape, np.uint8)
        for j, c in enumerate(np.asarray(centroids, np.float32)):
            d = z - c
            d = d * d
            nearer = d < best
            best, code = np.where(nearer, d, best), np.where(nearer, j, code).astype(np.uint8)
    return code, scale


def pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def rows_of(table_row, codes, scales, cents, head, tokens, page):
    """(seen [tokens] bool, rows [tokens, dim]) of one request and head; cents: 16 values."""
    pages, _, _, ns = codes.shape
    seen = np.zeros(tokens, bool)
    rows = np.zeros((tokens, 2 * ns))
    for t in range(tokens):
        b = t // page
        pg = int(table_row[b]) if b < len(table_row) else -1
        if 0 <= pg < pages:
            seen[t] = True
            byte = codes[pg, head, t % page]
            rows[t, 0::2], rows[t, 1::2] = cents[byte & 15], cents[byte >> 4]
            rows[t] *= scales[pg, head, t % page]
    return seen, rows


def attention(q, cu, lens, table, k_codes, v_codes, k_scales, v_scales, k_cents, v_cents, dtype, window=0, scale=0.0,
              tensor=False):
    """(out, lse, out bound, lse bound).

    The bounds are those of the code cache (paged_reference.attention): with u = 2^-24,
    kappa = scale log2 e, S_t = kappa q . K^_t, A_t = kappa sum |q_i K^_ti|, M = max S_t,
    T seen tokens and D the head size,
      * S_t is off by d_t <= (D + 6) u A_t: D products and sums, a product with the scale
        (after the sum) and a rounded factor kappa and its product;
      * a weight by a relative e_t <= ln 2 (d_t + 2 u (M - S_t + 8)) + 2^-21;
      * the sums add (T + 200) u.
    `tensor`: the tensor kernels round the weights to the rows' type (h = half its epsilon
    relative, or half its least step): e_t gains h and T times half the least step (as for
    codes), out its own rounding, max|V^| h + step."""
    u = 2.0 ** -24
    h = HALF_EPS[dtype] if tensor else 0.0
    step = HALF_STEP[dtype] if tensor else 0.0
    tokens, hq, dim = q.shape
    hkv, page = k_codes.shape[1], k_codes.shape[2]
    group = hq // hkv
    scale = scale if scale > 0 else 1.0 / math.sqrt(dim)
    kappa = scale / math.log(2)

    def book(cents):
        out = np.zeros(16)
        out[:len(cents)] = torch.tensor(cents, dtype=torch.float32).to(dtype).double().numpy()
        return out

    k_book, v_book = book(k_cents), book(v_cents)
    out = np.zeros((tokens, hq, dim))
    lse = np.full((tokens, hq), -np.inf)
    tol, tol_lse = np.zeros((tokens, hq, 1)), np.zeros((tokens, hq))
    for r, length in enumerate(lens):
        new = max(0, cu[r + 1] - cu[r])
        held = max(0, min(length, len(table[r]) * page)) if len(table) else 0
        for hd in range(hkv):
            ok, keys = rows_of(table[r], k_codes, k_scales, k_book, hd, held, page)
            _, values = rows_of(table[r], v_codes, v_scales, v_book, hd, held, page)
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
                    row, head = cu[r] + i, hd * group + g
                    s = scale * (k @ q[row, head])
                    top = s.max()
                    w = np.exp(s - top)
                    total = w.sum()
                    out[row, head] = w @ v / total
                    lse[row, head] = top + math.log(total)
                    n = len(s)
                    d = (dim + 6) * u * kappa * (np.abs(k) @ np.abs(q[row, head]))
                    e = math.log(2) * (d + 2 * u * ((top - s) / math.log(2) + 8)) + 2.0 ** -21 + h
                    most = np.abs(v).max()
                    tol[row, head] = 1.1 * (most * (2 * (w @ e) / total + 2 * n * step + 4 * (n + 200) * u + h) + step)
                    tol_lse[row, head] = 1.1 * (e.max() + n * step + (n + 200) * u) + 4 * u * abs(lse[row, head])
    return out, lse, tol, tol_lse
