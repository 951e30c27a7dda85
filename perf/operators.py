"""Measured cases of the paged code cache: page reservation and trimming,
appending new tokens as product-VQ codes, and attention of new tokens over the
pages.

Every case is one call that a serving loop makes.  ``run`` makes it through
the package where ``own`` is true, and in plain torch where it is false;
``exact`` states the definitions once more, on the host or in 64 bits.
Attention and append run in fp16 and bf16, the types such a loop serves in,
and append in fp32 too.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode step of 64 requests: one new token each, a page now and then
        {"name": "reserve-decode", "op": "reserve", "requests": 64, "page": 16, "held": 32768, "new_low": 1,
         "new_high": 1, "spare": 1.0},
        # admission of a burst of prompts, the pool too small for the last ones
        {"name": "reserve-prompts", "op": "reserve", "requests": 257, "page": 16, "held": 0, "new_low": 1,
         "new_high": 1021, "spare": 0.9},
        # rejected drafts of 64 requests: up to 4 tokens back
        {"name": "trim-drafts", "op": "trim", "requests": 64, "page": 16, "held": 32768, "drop": "few"},
        # a third of 1000 requests finished, all their pages go back
        {"name": "trim-finished", "op": "trim", "requests": 1000, "page": 16, "held": 8192, "drop": "all"},
        # a decode step of 64 tokens, 8 KV heads of 128
        {"name": "append-decode", "op": "append", "tokens": 64, "heads": 8, "dim": 128, "sub": 8, "centroids": 256,
         "page": 16, "dtype": "f16", "smooth": False},
        # a prefill step, keys and values inside a packed projection
        {"name": "append-prefill", "op": "append", "tokens": 8191, "heads": 8, "dim": 128, "sub": 8,
         "centroids": 256, "page": 64, "dtype": "bf16", "smooth": False},
        # heads of 256 in sub-vectors of 4, outlier channels smoothed
        {"name": "append-smooth", "op": "append", "tokens": 4096, "heads": 4, "dim": 256, "sub": 4,
         "centroids": 256, "page": 16, "dtype": "f16", "smooth": True},
        # one request, one token: the least latency
        {"name": "attend-one", "op": "attend", "requests": 1, "held_low": 777, "held_high": 777, "new_low": 1,
         "new_high": 1, "chunk": 0, "hq": 32, "hkv": 8, "dim": 128, "sub": 8, "centroids": 256, "page": 16,
         "dtype": "f16", "window": 0},
        # the decode step of a batch of uneven long requests
        {"name": "attend-decode", "op": "attend", "requests": 32, "held_low": 1000, "held_high": 32768,
         "new_low": 1, "new_high": 1, "chunk": 0, "hq": 32, "hkv": 8, "dim": 128, "sub": 8, "centroids": 256,
         "page": 16, "dtype": "f16", "window": 0},
        # verification of up to four drafts for each of 16 requests, sliding window
        {"name": "attend-drafts", "op": "attend", "requests": 16, "held_low": 5, "held_high": 16000, "new_low": 1,
         "new_high": 5, "chunk": 0, "hq": 32, "hkv": 8, "dim": 128, "sub": 8, "centroids": 256, "page": 64,
         "dtype": "bf16", "window": 8192},
        # a 2048-token chunk of one prompt beside the decode step of 15 others
        {"name": "attend-mixed", "op": "attend", "requests": 16, "held_low": 2000, "held_high": 24000, "new_low": 1,
         "new_high": 1, "chunk": 2048, "hq": 32, "hkv": 8, "dim": 128, "sub": 8, "centroids": 256, "page": 16,
         "dtype": "bf16", "window": 0},
        # two prompts' chunks, heads of 256 in sub-vectors of 4, three query heads to a KV head
        {"name": "attend-wide", "op": "attend", "requests": 2, "held_low": 3000, "held_high": 9000, "new_low": 1500,
         "new_high": 2100, "chunk": 0, "hq": 12, "hkv": 4, "dim": 256, "sub": 4, "centroids": 256, "page": 16,
         "dtype": "f16", "window": 0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["reserve", "trim", "append", "append", "attend", "attend", "attend"])
    if op == "reserve":
        if rng.random() < 0.5:
            return {"op": op, "requests": _log(rng, 1, 512), "page": rng.choice([16, 32, 64]),
                    "held": _log(rng, 16, 32768), "new_low": 1, "new_high": rng.choice([1, 1, 5]), "spare": 1.0}
        requests = _log(rng, 1, 257)
        return {"op": op, "requests": requests, "page": rng.choice([16, 32, 64]), "held": rng.choice([0, 0, 1000]),
                "new_low": 1, "new_high": min(16384, 130000 // requests), "spare": rng.choice([1.0, 0.9, 0.5])}
    if op == "trim":
        return {"op": op, "requests": _log(rng, 1, 1000), "page": rng.choice([16, 32, 64]),
                "held": _log(rng, 16, 8192), "drop": rng.choice(["few", "all"])}
    shapes = [(8, 128, 8), (8, 128, 4), (4, 256, 4), (8, 64, 8), (2, 256, 8), (3, 64, 4)]
    if op == "append":
        heads, dim, sub = rng.choice(shapes)
        tokens = min(_log(rng, 1, 8191), 2_000_000 // (heads * dim // sub * 2))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "sub": sub,
                "centroids": rng.choice([256, 256, 256, 200, 64]), "page": rng.choice([16, 32, 64]),
                "dtype": rng.choice(["f16", "bf16", "f16", "bf16", "f32"]), "smooth": rng.random() < 0.3}
    hkv, dim, sub = rng.choice(shapes)
    group = rng.choice([1, 2, 3, 4, 4, 8])
    case = {"op": op, "requests": 1, "held_low": 1, "held_high": 1, "new_low": 1, "new_high": 1, "chunk": 0,
            "hq": hkv * group, "hkv": hkv, "dim": dim, "sub": sub, "centroids": rng.choice([256, 256, 256, 200]),
            "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["f16", "bf16"]),
            "window": rng.choice([0, 0, 0, _log(rng, 100, 8192)])}
    kind = rng.choice(["decode", "drafts", "mixed", "chunks"])
    if kind == "decode":
        case["requests"] = _log(rng, 1, 64)
        case["held_high"] = min(32768, _log(rng, 100, 600_000 // case["requests"]))
    elif kind == "drafts":
        case["requests"] = _log(rng, 1, 32)
        case["held_high"] = min(16000, _log(rng, 100, 300_000 // case["requests"]))
        case["new_high"] = rng.choice([3, 5, 8, 17])
    elif kind == "mixed":
        case["requests"] = _log(rng, 2, 16)
        case["held_high"] = _log(rng, 100, 12000)
        case["chunk"] = _log(rng, 33, min(2048, 2048 * 4 * 8 * 128 // (hkv * group * dim)))
    else:
        case["requests"] = rng.choice([1, 2, 3])
        case["held_high"] = _log(rng, 1, 9000)
        case["new_low"] = 17
        case["new_high"] = max(17, _log(rng, 17, min(2100, 4200 * 32 * 128 // (case["requests"] * hkv * group * dim))))
    return case


# ---------------------------------------------------------------- what a program has in hand


def _lengths(case):
    """Lengths of the case's requests, the same for every seed (so that the
    work of a case does not depend on it): held before the step, and new."""
    rng = np.random.default_rng([case["requests"], case.get("held", case.get("held_high", 0)), case["page"]])
    r = case["requests"]
    if case["op"] in ("reserve", "trim"):
        held = rng.integers(0, case["held"] + 1, r)
    else:
        held = rng.integers(case["held_low"], case["held_high"] + 1, r)
    if case["op"] == "trim":
        if case["drop"] == "few":
            return held, held - np.minimum(held, rng.integers(0, 5, r))
        return held, np.where(rng.random(r) < 1 / 3, 0, held)
    new = rng.integers(case["new_low"], case["new_high"] + 1, r)
    if case.get("chunk"):
        new[r // 2] = case["chunk"]
    return held, new


def _pages(total, page):
    return -(-total // page)


def _table(held_pages, width, pool):
    """Block table whose first held_pages[r] entries are pages of the pool, in
    no order, and the rest -1; and the pages left over."""
    table = np.full((len(held_pages), width), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(held_pages):
        table[r, :n] = pool[at:at + n]
        at += n
    return table, pool[at:]


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op in ("reserve", "trim"):
        held, second = _lengths(case)
        order = rng.permutation(len(held))  # another order of the requests for each seed
        held, second = held[order], second[order]
        page = case["page"]
        if op == "reserve":
            want = _pages(held + second, page) - _pages(held, page)
            spare = int(math.ceil(case["spare"] * want.sum())) + (7 if case["spare"] >= 1 else 0)
            width = int(_pages(held + second, page).max())
        else:
            spare, width = 5, max(1, int(_pages(held, page).max()))
        pages = int(_pages(held, page).sum()) + spare
        table, left = _table(_pages(held, page), width, rng.permutation(pages))
        free = np.full(pages, -1, dtype=np.int32)
        free[:len(left)] = left
        state.update(lens=_int32(held), second=_int32(second), table=_int32(table), free=_int32(free),
                     count=_int32([len(left)]), total=int(second.sum()))
        return state
    dtype = DTYPES[case["dtype"]]
    hkv, dim, sub, nc, page = (case[k] for k in ("heads" if op == "append" else "hkv", "dim", "sub", "centroids", "page"))
    books = [torch.randn((hkv, nc, sub), generator=gen, device="cuda").to(dtype) for _ in range(2)]
    state.update(kcb=books[0], vcb=books[1])
    if op == "append":
        tokens = case["tokens"]
        packed = torch.randn((tokens, 3 * hkv, dim), generator=gen, device="cuda")
        smooth = None
        if case["smooth"]:
            smooth = torch.exp(0.5 * torch.randn((hkv, dim), generator=gen, device="cuda"))
            packed[:, hkv:2 * hkv] *= smooth
        packed = packed.to(dtype)
        pages = _pages(tokens, page) + 3
        shape = (pages, hkv, page, dim // sub)
        slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens].clone()
        slots[::61] = -1  # tokens of refused requests
        state.update(k=packed[:, hkv:2 * hkv], v=packed[:, 2 * hkv:], smooth=smooth, slots=slots,
                     kc=torch.zeros(shape, dtype=torch.uint8, device="cuda"),
                     vc=torch.zeros(shape, dtype=torch.uint8, device="cuda"))
        return state
    held, new = _lengths(case)
    order = rng.permutation(len(held))
    held, new = held[order], new[order]
    lens = held + new
    blocks = _pages(lens, page)
    pages = int(blocks.sum()) + 3
    table, _ = _table(blocks, int(blocks.max()), rng.permutation(pages))
    shape = (pages, hkv, page, dim // sub)
    tokens = int(new.sum())
    packed = torch.randn((tokens, case["hq"] + 2 * hkv, dim), generator=gen, device="cuda").to(dtype)
    state.update(
        q=packed[:, :case["hq"]], table=_int32(table), lens=_int32(lens),
        cu=_int32(np.concatenate([[0], np.cumsum(new)])), max_new=int(new.max()),
        kc=torch.randint(0, nc, shape, generator=gen, device="cuda", dtype=torch.uint8),
        vc=torch.randint(0, nc, shape, generator=gen, device="cuda", dtype=torch.uint8),
        lens_list=[int(n) for n in lens], new_list=[int(n) for n in new])
    return state


# ---------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _own_reserve(s):
    import product_vq_kv_gb300 as vq

    lens, count, cu, slots = vq.vq_paged_reserve(s["lens"], s["second"], s["free"], s["count"], s["table"],
                                                 s["case"]["page"], s["total"])
    return lens, count, cu, slots, s["table"]


def _own_trim(s):
    import product_vq_kv_gb300 as vq

    lens, count = vq.vq_paged_trim(s["lens"], s["second"], s["table"], s["case"]["page"], s["free"], s["count"])
    return lens, count, s["free"]


def _own_append(s):
    import product_vq_kv_gb300 as vq

    vq.vq_paged_append(s["k"], s["v"], s["slots"], s["kcb"], s["vcb"], s["kc"], s["vc"], k_smooth=s["smooth"])
    return s["kc"], s["vc"]


def _own_attend(s):
    import product_vq_kv_gb300 as vq

    return vq.vq_paged_attention(s["q"], s["cu"], s["lens"], s["table"], s["kc"], s["vc"], s["kcb"], s["vcb"],
                                 max_new=s["max_new"], window=s["case"]["window"], return_lse=True)


def _plain_reserve(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    held, new, count = s["lens"].long(), s["second"].long(), s["count"].long()
    width = table.shape[1]
    old, upto = (held + page - 1) // page, (held + new + page - 1) // page
    need = torch.where(upto <= width, upto - old, 0)
    upto_sum = need.cumsum(0)
    granted = (held + new <= width * page) & ((need == 0) | (upto_sum <= count))
    taken = torch.where(granted, need, 0)
    before = upto_sum - need
    block = torch.arange(width, device=table.device)[None, :]
    fresh = granted[:, None] & (block >= old[:, None]) & (block < upto[:, None])
    nth = count - 1 - before[:, None] - (block - old[:, None])
    table = torch.where(fresh, free[nth.clamp(0, free.numel() - 1)], table)
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    token = torch.arange(s["total"], device=table.device)
    r = (token[:, None] >= cu[None, 1:]).sum(1)
    at = held[r] + token - cu[r]
    slots = torch.where(granted[r], table[r, (at // page).clamp(max=width - 1)].long() * page + at % page, -1)
    return (held + torch.where(granted, new, 0)).int(), (count - taken.sum()).int(), cu.int(), slots, table


def _plain_trim(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    held, count = s["lens"].long(), s["count"].long()
    keep = torch.minimum(s["second"].long().clamp(min=0), held)
    first, upto = (keep + page - 1) // page, (held + page - 1) // page
    back = upto - first
    before = back.cumsum(0) - back
    block = torch.arange(table.shape[1], device=table.device)[None, :]
    given = (block >= first[:, None]) & (block < upto[:, None])
    at = torch.where(given, count + before[:, None] + block - first[:, None], free.numel())
    room = torch.cat([free, free[:1]])  # one place past the end takes what is not given back
    room[at.reshape(-1)] = table.reshape(-1)
    return keep.int(), (count + back.sum()).int(), room[:-1]


def _nearest(x, books):
    """Index of the nearest centroid of every row x [T, H, S, sub] of head h in
    books [H, n, sub], by the fp32 sum of squares, the lowest of equals."""
    x, books = x.float(), books.float()
    t, h, s, sub = x.shape
    n = books.shape[1]
    out = torch.empty((t, h, s), dtype=torch.uint8, device=x.device)
    number = torch.arange(n, device=x.device)
    step = max(1, (1 << 26) // (h * s * n))
    for a in range(0, t, step):
        dist = 0.0
        for i in range(sub):
            d = x[a:a + step, :, :, None, i] - books[None, :, None, :, i]
            dist = dist + d * d
        dist = torch.where(dist == dist, dist, math.inf)
        best = dist.amin(-1, keepdim=True)
        out[a:a + step] = torch.where((dist == best) & (dist < math.inf), number, n).amin(-1).remainder(n).to(torch.uint8)
    return out


def _plain_append(s):
    case = s["case"]
    page, sub, heads = case["page"], case["sub"], case["heads"]
    slots = s["slots"]
    done = []
    for x, books, codes, smooth in ((s["k"], s["kcb"], s["kc"], s["smooth"]), (s["v"], s["vcb"], s["vc"], None)):
        if smooth is not None:
            x = x.float() / smooth
        code = _nearest(x.reshape(case["tokens"], heads, -1, sub), books)
        room = torch.cat([codes, codes[:1]])  # one page past the end takes what has no slot
        at = torch.where(slots >= 0, slots, codes.shape[0] * page)
        room[at // page, :, at % page] = code
        done.append(room[:-1])
    return tuple(done)


def _plain_attend(s):
    case, q = s["case"], s["q"]
    hq, hkv, dim, page, window = (case[k] for k in ("hq", "hkv", "dim", "page", "window"))
    out = torch.empty((q.shape[0], hq, dim), dtype=q.dtype, device=q.device)
    lse = torch.empty((q.shape[0], hq), dtype=torch.float32, device=q.device)
    head = torch.arange(hkv, device=q.device)[:, None, None]
    row = 0
    for r, (length, new) in enumerate(zip(s["lens_list"], s["new_list"])):
        low = max(0, length - new - window + 1) if window else 0
        pages = s["table"][r, low // page:-(-length // page)].long()
        low = low // page * page

        def rebuilt(codes, books):
            code = codes[pages].transpose(0, 1).reshape(hkv, -1, codes.shape[3])[:, :length - low].long()
            return books.float()[head, code].reshape(hkv, length - low, dim)

        keys, values = rebuilt(s["kc"], s["kcb"]), rebuilt(s["vc"], s["vcb"])
        at = torch.arange(low, length, device=q.device)
        step = max(1, (1 << 28) // (hq * (length - low)))
        for a in range(0, new, step):
            n = min(step, new - a)
            rows = q[row + a:row + a + n].float().reshape(n, hkv, hq // hkv, dim).permute(1, 2, 0, 3).reshape(hkv, -1, dim)
            score = torch.matmul(rows, keys.transpose(1, 2)) * (1.0 / math.sqrt(dim))
            pos = torch.arange(length - new + a, length - new + a + n, device=q.device)
            seen = at[None, :] <= pos[:, None]
            if window:
                seen &= at[None, :] > pos[:, None] - window
            score = score.reshape(hkv, hq // hkv, n, -1).masked_fill(~seen, -math.inf).reshape(hkv, -1, length - low)
            top = score.amax(-1, keepdim=True)
            weight = torch.exp(score - top)
            total = weight.sum(-1, keepdim=True)
            o = torch.matmul(weight, values) / total
            out[row + a:row + a + n] = o.reshape(hkv, hq // hkv, n, dim).permute(2, 0, 1, 3).reshape(n, hq, dim).to(q.dtype)
            lse[row + a:row + a + n] = (top + torch.log(total)).reshape(hq, n).t()
        row += new
    return out, lse


_own = {"reserve": _own_reserve, "trim": _own_trim, "append": _own_append, "attend": _own_attend}
_plain = {"reserve": _plain_reserve, "trim": _plain_trim, "append": _plain_append, "attend": _plain_attend}


# ---------------------------------------------------------------- the least work of one pass


def work(case):
    op = case["op"]
    if op in ("reserve", "trim"):
        held, second = _lengths(case)
        page = case["page"]
        if op == "trim":
            pages = int((_pages(held, page) - _pages(second, page)).sum())
            return {"bytes": 12 * len(held) + 8 * pages + 8, "flops": 0}
        pages = int((_pages(held + second, page) - _pages(held, page)).sum())
        return {"bytes": 16 * len(held) + 8 * pages + 8 * int(second.sum()) + 8, "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "append":
        rows = 2 * case["tokens"] * case["heads"] * (case["dim"] // case["sub"])
        return {"bytes": rows * (case["sub"] * size + 1) + 8 * case["tokens"]
                + 2 * case["heads"] * case["centroids"] * case["sub"] * size,
                "flops": 2 * rows * case["sub"] * case["centroids"]}
    held, new = _lengths(case)
    seen = tokens = 0
    for h, n in zip(held.tolist(), new.tolist()):
        low = max(0, h - case["window"] + 1) if case["window"] else 0
        tokens += h + n - low
        pos = np.arange(h, h + n)
        seen += int(np.minimum(pos + 1, case["window"] or h + n + 1).sum())
    codes = 2 * tokens * case["hkv"] * (case["dim"] // case["sub"])
    books = 2 * case["hkv"] * case["centroids"] * case["sub"] * size
    rows = int(new.sum()) * case["hq"]
    return {"bytes": codes + books + rows * (2 * case["dim"] * size + 4), "flops": 4 * seen * case["hq"] * case["dim"]}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"reserve": _exact_reserve, "trim": _exact_trim, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_reserve(s):
    page = s["case"]["page"]
    held, new, free = (s[k].cpu().tolist() for k in ("lens", "second", "free"))
    table = s["table"].cpu().numpy().copy()
    left = int(s["count"].item())
    wanted, out, cu, slots = 0, [], [0], []
    stack = left
    for r, (h, n) in enumerate(zip(held, new)):
        cu.append(cu[-1] + n)
        fits = h + n <= table.shape[1] * page
        blocks = list(range(-(-h // page), -(-(h + n) // page))) if fits else []
        wanted += len(blocks)
        if not fits or (blocks and wanted > left):
            out.append(h)
            slots += [-1] * n
            continue
        for b in blocks:
            stack -= 1
            table[r, b] = free[stack]
        out.append(h + n)
        slots += [int(table[r, p // page]) * page + p % page for p in range(h, h + n)]
    return (np.array(out, np.int32), np.array([stack], np.int32), np.array(cu, np.int32),
            np.array(slots, np.int64), table)


def _exact_trim(s):
    page = s["case"]["page"]
    held, keep = (s[k].cpu().tolist() for k in ("lens", "second"))
    table, free = s["table"].cpu().tolist(), s["free"].cpu().tolist()
    top = int(s["count"].item())
    for r, (h, k) in enumerate(zip(held, keep)):
        for b in range(-(-k // page), -(-h // page)):
            free[top] = table[r][b]
            top += 1
    return np.array(keep, np.int32), np.array([top], np.int32), np.array(free, np.int32)


def _exact_append(s):
    """The rule is stated in fp32 steps: each is one operation in 64 bits,
    rounded to 32 (exact, as 53 bits are more than twice 24 and two)."""
    case = s["case"]
    done = []
    slots = s["slots"].cpu().numpy()
    for x, books, codes, smooth in (("k", "kcb", "kc", s["smooth"]), ("v", "vcb", "vc", None)):
        x, books, codes = s[x].double(), s[books].double(), s[codes].cpu().numpy().copy()
        if smooth is not None:
            x = (x / smooth.double()).float().double()
        x = x.reshape(case["tokens"], case["heads"], -1, case["sub"])
        for h in range(case["heads"]):
            rows = x[:, h].reshape(-1, case["sub"])
            best = torch.full((rows.shape[0],), math.inf, dtype=torch.float64, device=rows.device)
            index = torch.zeros(rows.shape[0], dtype=torch.int64, device=rows.device)
            for c in range(case["centroids"]):
                total = None
                for i in range(case["sub"]):
                    d = (rows[:, i] - books[h, c, i]).float().double()
                    d = (d * d).float().double()
                    total = d if total is None else (total + d).float().double()
                nearer = total < best
                best, index = torch.where(nearer, total, best), torch.where(nearer, c, index)
            index = index.reshape(case["tokens"], -1).cpu().numpy().astype(np.uint8)
            at = slots >= 0
            codes[slots[at] // case["page"], h, slots[at] % case["page"]] = index[at]
        done.append(codes)
    return tuple(done)


def _exact_attend(s):
    case = s["case"]
    hq, hkv, dim, page, window = (case[k] for k in ("hq", "hkv", "dim", "page", "window"))
    group = hq // hkv
    q = s["q"]
    out = torch.zeros((q.shape[0], hq, dim), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device=q.device)
    row = 0
    for r, (length, new) in enumerate(zip(s["lens_list"], s["new_list"])):
        where = torch.arange(length, device=q.device)
        page_of = s["table"][r].long()[where // page]
        for h in range(hkv):
            rows_k = s["kc"][page_of, h, where % page].long()
            rows_v = s["vc"][page_of, h, where % page].long()
            keys = s["kcb"][h].double()[rows_k].reshape(length, dim)
            values = s["vcb"][h].double()[rows_v].reshape(length, dim)
            for g in range(group):
                for a in range(0, new, 1024):
                    e = min(new, a + 1024)
                    z = q[row + a:row + e, h * group + g].double() @ keys.t() / math.sqrt(dim)
                    pos = length - new + torch.arange(a, e, device=q.device)[:, None]
                    hidden = where[None, :] > pos
                    if window:
                        hidden = hidden | (where[None, :] <= pos - window)
                    z[hidden] = -math.inf
                    l = torch.logsumexp(z, 1)
                    lse[row + a:row + e, h * group + g] = l
                    out[row + a:row + e, h * group + g] = torch.exp(z - l[:, None]) @ values
        row += new
    return out, lse
