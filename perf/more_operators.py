"""Measured cases of the paged cache held in 4 bits and of shared pages:
appending new tokens as scalar codes of 4 bits, attention of new tokens over
them, forking requests whose pages are shared, compacting the pool, and the
copies of pages that both ask for.

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
        # a decode step of 64 tokens, 8 KV heads of 128, keys rotated
        {"name": "append-decode", "op": "append", "tokens": 64, "heads": 8, "dim": 128, "centroids": 16, "page": 16,
         "dtype": "f16", "rotate": True},
        # a prefill step, keys and values inside a packed projection
        {"name": "append-prefill", "op": "append", "tokens": 8191, "heads": 8, "dim": 128, "centroids": 16,
         "page": 64, "dtype": "bf16", "rotate": True},
        # one request, one token: the least latency
        {"name": "attend-one", "op": "attend", "requests": 1, "held_low": 777, "held_high": 777, "new_low": 1,
         "new_high": 1, "chunk": 0, "hq": 32, "hkv": 8, "dim": 128, "centroids": 16, "page": 16, "dtype": "f16",
         "window": 0},
        # the decode step of a batch of uneven long requests
        {"name": "attend-decode", "op": "attend", "requests": 32, "held_low": 1000, "held_high": 32768, "new_low": 1,
         "new_high": 1, "chunk": 0, "hq": 32, "hkv": 8, "dim": 128, "centroids": 16, "page": 16, "dtype": "f16",
         "window": 0},
        # verification of up to four drafts for each of 16 requests, heads of 256, sliding window
        {"name": "attend-drafts", "op": "attend", "requests": 16, "held_low": 5, "held_high": 16000, "new_low": 1,
         "new_high": 5, "chunk": 0, "hq": 12, "hkv": 4, "dim": 256, "centroids": 16, "page": 64, "dtype": "bf16",
         "window": 8192},
        # a 2048-token chunk of one prompt beside the decode step of 15 others
        {"name": "attend-mixed", "op": "attend", "requests": 16, "held_low": 2000, "held_high": 24000, "new_low": 1,
         "new_high": 1, "chunk": 2048, "hq": 32, "hkv": 8, "dim": 128, "centroids": 16, "page": 16, "dtype": "bf16",
         "window": 0},
        # a step of beam search: 64 requests of four beams each
        {"name": "fork-beams", "op": "fork", "groups": 64, "beams": 4, "held": 2000, "page": 16, "kind": "beams"},
        # 100 prompts just read, each split into 8 samples; the seats of finished requests are emptied
        {"name": "fork-samples", "op": "fork", "groups": 100, "beams": 8, "held": 8192, "page": 16, "kind": "samples"},
        # a pool of 4099 pages half of them free, scattered
        {"name": "compact-small", "op": "compact", "requests": 64, "held": 1000, "page": 16, "free": 0.5},
        # a pool of 200,000 pages, a fifth of them free
        {"name": "compact-large", "op": "compact", "requests": 1000, "held": 5000, "page": 16, "free": 0.2},
        # the last pages of a beam step's forks, codes and scales of one layer
        {"name": "copy-forks", "op": "copy", "rows": 256, "live": 0.4, "layers": 1, "heads": 8, "dim": 128, "page": 16,
         "dtype": "f16"},
        # the moves of a compaction, eight layers at once
        {"name": "copy-moves", "op": "copy", "rows": 2047, "live": 1.0, "layers": 8, "heads": 8, "dim": 128,
         "page": 16, "dtype": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


SHAPES = [(8, 128), (8, 128), (4, 256), (8, 64), (2, 256), (3, 64), (5, 128)]


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "fork", "compact", "copy"])
    if op == "append":
        heads, dim = rng.choice(SHAPES)
        return {"op": op, "tokens": min(_log(rng, 1, 8191), 8_000_000 // (heads * dim)), "heads": heads, "dim": dim,
                "centroids": rng.choice([16, 16, 16, 15, 8]), "page": rng.choice([16, 32, 64]),
                "dtype": rng.choice(["f16", "bf16", "f16", "bf16", "f32"]), "rotate": rng.random() < 0.6}
    if op == "fork":
        kind = rng.choice(["beams", "samples"])
        groups, beams = _log(rng, 1, 100), rng.choice([2, 3, 4, 5, 8])
        return {"op": op, "groups": groups, "beams": beams, "held": _log(rng, 17, 8192),
                "page": rng.choice([16, 32, 64]), "kind": kind}
    if op == "compact":
        return {"op": op, "requests": _log(rng, 1, 1000), "held": _log(rng, 16, 5000), "page": rng.choice([16, 32, 64]),
                "free": rng.choice([0.05, 0.2, 0.5, 0.9])}
    if op == "copy":
        heads, dim = rng.choice(SHAPES)
        layers = rng.choice([1, 1, 2, 8])
        page = rng.choice([16, 32, 64])
        most = 2047 * 8 * 8 * 128 * 16 // (layers * heads * dim * page)
        return {"op": op, "rows": _log(rng, 1, min(2047, most)), "live": rng.choice([0.3, 0.7, 1.0]), "layers": layers,
                "heads": heads, "dim": dim, "page": page, "dtype": rng.choice(["f16", "bf16", "f32"])}
    hkv, dim = rng.choice(SHAPES)
    group = rng.choice([1, 2, 3, 4, 4, 8])
    case = {"op": op, "requests": 1, "held_low": 1, "held_high": 1, "new_low": 1, "new_high": 1, "chunk": 0,
            "hq": hkv * group, "hkv": hkv, "dim": dim, "centroids": rng.choice([16, 16, 16, 15]),
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
    """Lengths of an attention's requests, the same for every seed (so that
    the work of a case does not depend on it): held before the step, and new."""
    rng = np.random.default_rng([case["requests"], case["held_high"], case["page"]])
    held = rng.integers(case["held_low"], case["held_high"] + 1, case["requests"])
    new = rng.integers(case["new_low"], case["new_high"] + 1, case["requests"])
    if case["chunk"]:
        new[case["requests"] // 2] = case["chunk"]
    return held, new


def _fork_lengths(case):
    """Of a fork, by group: tokens that all beams share, and each beam's own."""
    rng = np.random.default_rng([case["groups"], case["beams"], case["held"]])
    shared = rng.integers(case["held"] // 2, case["held"] + 1, case["groups"])
    apart = rng.integers(1, case["held"] // 8 + 2, (case["groups"], case["beams"]))
    return shared, apart


def _compact_lengths(case):
    rng = np.random.default_rng([case["requests"], case["held"], case["page"]])
    return rng.integers(0, case["held"] + 1, case["requests"])


def _pages(total, page):
    return -(-total // page)


def _table(held_pages, width, pool):
    """Block table whose first held_pages[r] entries are pages of the pool, in
    no order, and the rest -1."""
    table = np.full((len(held_pages), width), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(held_pages):
        table[r, :n] = pool[at:at + n]
        at += n
    return table


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _centroids(n, rng):
    """Quantiles of a normal distribution, each a little off: ascending."""
    at = (np.arange(n) + 0.5 + rng.uniform(-0.1, 0.1, n)) / n
    return (math.sqrt(2) * torch.erfinv(torch.from_numpy(2 * at - 1))).float().cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"append": _prepare_append, "attend": _prepare_attend, "fork": _prepare_fork,
            "compact": _prepare_compact, "copy": _prepare_copy}[case["op"]](case, rng, gen)


def _prepare_append(case, rng, gen):
    dtype, heads, dim, page, tokens = (case[k] for k in ("dtype", "heads", "dim", "page", "tokens"))
    dtype = DTYPES[dtype]
    packed = torch.randn((tokens, 3 * heads, dim), generator=gen, device="cuda")
    packed[:, heads:2 * heads] *= torch.exp(0.5 * torch.randn((heads, dim), generator=gen, device="cuda"))  # outlier channels
    packed *= torch.exp(0.5 * torch.randn((tokens, 3 * heads, 1), generator=gen, device="cuda"))
    packed = packed.to(dtype)
    pages = _pages(tokens, page) + 3
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens].clone()
    slots[::61] = -1  # tokens of refused requests
    signs = None
    if case["rotate"]:
        signs = torch.randint(0, 2, (dim,), generator=gen, device="cuda").float() * 2 - 1
    codes, scales = (pages, heads, page, dim // 2), (pages, heads, page)
    return {"case": case, "k": packed[:, heads:2 * heads], "v": packed[:, 2 * heads:], "slots": slots, "signs": signs,
            "kcent": _centroids(case["centroids"], rng), "vcent": _centroids(case["centroids"], rng),
            "kc": torch.zeros(codes, dtype=torch.uint8, device="cuda"),
            "vc": torch.zeros(codes, dtype=torch.uint8, device="cuda"),
            "ks": torch.zeros(scales, dtype=dtype, device="cuda"), "vs": torch.zeros(scales, dtype=dtype, device="cuda")}


def _prepare_attend(case, rng, gen):
    dtype, hkv, dim, page, nc = (case[k] for k in ("dtype", "hkv", "dim", "page", "centroids"))
    dtype = DTYPES[dtype]
    held, new = _lengths(case)
    order = rng.permutation(len(held))  # another order of the requests for each seed
    held, new = held[order], new[order]
    lens = held + new
    blocks = _pages(lens, page)
    pages = int(blocks.sum()) + 3
    table = _table(blocks, int(blocks.max()), rng.permutation(pages))
    tokens = int(new.sum())
    packed = torch.randn((tokens, case["hq"] + 2 * hkv, dim), generator=gen, device="cuda").to(dtype)

    def codes():
        c = torch.randint(0, 256, (pages, hkv, page, dim // 2), generator=gen, device="cuda", dtype=torch.uint8)
        return c if nc == 16 else (c % 16 % nc) | (c // 16 % nc) << 4

    def scales():
        return torch.exp(0.5 * torch.randn((pages, hkv, page), generator=gen, device="cuda")).to(dtype)

    return {"case": case, "q": packed[:, :case["hq"]], "table": _int32(table), "lens": _int32(lens),
            "cu": _int32(np.concatenate([[0], np.cumsum(new)])), "max_new": int(new.max()), "kc": codes(),
            "vc": codes(), "ks": scales(), "vs": scales(), "kcent": _centroids(nc, rng), "vcent": _centroids(nc, rng),
            "lens_list": [int(n) for n in lens], "new_list": [int(n) for n in new]}


def _prepare_fork(case, rng, gen):
    """A beam step: beams of a request share the pages of its first tokens and
    hold the rest alone; each beam goes on from any beam of its request.
    Samples: a request's first seat holds a prompt, the others are empty or end."""
    groups, beams, page = case["groups"], case["beams"], case["page"]
    shared, apart = _fork_lengths(case)
    order = rng.permutation(groups)
    shared, apart = shared[order], apart[order]
    seats = groups * beams
    lens = np.zeros(seats, np.int64)
    width = int(_pages(shared + apart.max(1), page).max())
    pages = int((_pages(shared, page) + beams * (_pages(apart.max(1), page) + 1)).sum()) + seats + 5
    pool = rng.permutation(pages)
    table = np.full((seats, width), -1, np.int32)
    at = 0
    for g in range(groups):
        whole = int(shared[g]) // page
        for b in range(beams if case["kind"] == "beams" else 1):
            n = int(shared[g] + apart[g, b])
            s = g * beams + b
            lens[s] = n
            if b == 0:
                table[s, :whole] = pool[at:at + whole]
                at += whole
            else:
                table[s, :whole] = table[g * beams, :whole]
            own_pages = _pages(n, page) - whole
            table[s, whole:whole + own_pages] = pool[at:at + own_pages]
            at += own_pages
    first = np.arange(seats) // beams * beams
    if case["kind"] == "beams":
        parents = first + rng.integers(0, beams, seats)
        keep = None
    else:
        parents = np.where(rng.random(groups)[np.arange(seats) // beams] < 0.1, -1, first)
        keep = lens[first]
    free = np.full(pages, -1, np.int32)
    free[:pages - at] = pool[at:]
    return {"case": case, "lens": _int32(lens), "parents": _int32(parents), "table": _int32(table),
            "keep": None if keep is None else _int32(keep), "free": _int32(free), "count": _int32([pages - at])}


def _prepare_compact(case, rng, gen):
    page = case["page"]
    lens = _compact_lengths(case)[rng.permutation(case["requests"])]
    held = int(_pages(lens, page).sum())
    pages = max(1, int(round(held / (1 - case["free"])))) + 1
    pool = rng.permutation(pages)
    free = np.full(pages, -1, np.int32)
    free[:pages - held] = pool[held:]
    table = _table(_pages(lens, page), max(1, int(_pages(lens, page).max())), pool)
    return {"case": case, "lens": _int32(lens), "table": _int32(table), "free": _int32(free),
            "count": _int32([pages - held])}


def _prepare_copy(case, rng, gen):
    rows, layers, heads, dim, page = (case[k] for k in ("rows", "layers", "heads", "dim", "page"))
    dtype = DTYPES[case["dtype"]]
    pages = 2 * rows + 3
    order = rng.permutation(pages)
    pairs = np.stack([order[:rows], order[rows:2 * rows]], 1)
    pairs[int(math.ceil(case["live"] * rows)):] = -1
    if case["live"] < 0.5:
        pairs = pairs[rng.permutation(rows)]  # a fork's copies lie among the seats that need none
    codes = torch.randint(0, 256, (layers, pages, 2, heads, page, dim // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randn((layers, pages, 2, heads, page), generator=gen, device="cuda").to(dtype)
    return {"case": case, "pairs": _int32(pairs), "codes": codes, "scales": scales}


# ---------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _own_append(s):
    import product_vq_kv_gb300 as vq

    vq.vq_paged_scalar_append(s["k"], s["v"], s["slots"], s["kcent"], s["vcent"], s["kc"], s["vc"], s["ks"], s["vs"],
                              k_signs=s["signs"])
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _own_attend(s):
    import product_vq_kv_gb300 as vq

    return vq.vq_paged_scalar_attention(s["q"], s["cu"], s["lens"], s["table"], s["kc"], s["vc"], s["ks"], s["vs"],
                                        s["kcent"], s["vcent"], max_new=s["max_new"], window=s["case"]["window"],
                                        return_lse=True)


def _own_fork(s):
    import product_vq_kv_gb300 as vq

    lens, table, count, copies = vq.vq_paged_fork(s["lens"], s["parents"], s["table"], s["case"]["page"], s["free"],
                                                  s["count"], keep_lens=s["keep"])
    return lens, table, count, copies, s["free"]


def _own_compact(s):
    import product_vq_kv_gb300 as vq

    return vq.vq_paged_compact(s["lens"], s["table"], s["case"]["page"], s["free"], s["count"])


def _own_copy(s):
    import product_vq_kv_gb300 as vq

    vq.vq_paged_copy(s["pairs"], [s["codes"], s["scales"]], layered=True)
    return s["codes"], s["scales"]


def _rotated(x, signs):
    """The randomised Hadamard rotation of the last axis, in rounded fp32 steps."""
    y = x.float() * signs
    n = y.shape[-1]
    step = 1
    while step < n:
        z = y.reshape(*y.shape[:-1], n // (2 * step), 2, step)
        a, b = z[..., 0, :], z[..., 1, :]
        y = torch.stack([a + b, a - b], -2).reshape(y.shape)
        step *= 2
    return y * float(np.float32(1.0 / math.sqrt(n)))


def _plain_append(s):
    case = s["case"]
    page, slots = case["page"], s["slots"]
    done = []
    for x, cent, codes, scales, signs in ((s["k"], s["kcent"], s["kc"], s["ks"], s["signs"]),
                                          (s["v"], s["vcent"], s["vc"], s["vs"], None)):
        y = _rotated(x, signs) if signs is not None else x.float()
        total = y * y  # summed in pairs of neighbours
        while total.shape[-1] > 1:
            total = total[..., 0::2] + total[..., 1::2]
        scale = torch.sqrt((total / case["dim"]).double()).float().to(x.dtype)  # (rounded once in either type)
        scale = torch.where(torch.isfinite(scale), scale, 0)
        z = torch.where(scale > 0, y * torch.reciprocal(scale.double()).float(), 0)
        best = torch.full_like(z, math.inf)
        code = torch.zeros(z.shape, dtype=torch.uint8, device=z.device)
        for j in range(case["centroids"]):
            d = z - cent[j]
            d = d * d
            code = torch.where(d < best, j, code)
            best = torch.minimum(d, best)
        packed = code[..., 0::2] | code[..., 1::2] << 4
        room, room_s = torch.cat([codes, codes[:1]]), torch.cat([scales, scales[:1]])  # a page for what has no slot
        at = torch.where(slots >= 0, slots, codes.shape[0] * page)
        room[at // page, :, at % page] = packed
        room_s[at // page, :, at % page] = scale[..., 0]
        done.append((room[:-1], room_s[:-1]))
    return done[0][0], done[1][0], done[0][1], done[1][1]


def _plain_attend(s):
    case, q = s["case"], s["q"]
    hq, hkv, dim, page, window = (case[k] for k in ("hq", "hkv", "dim", "page", "window"))
    out = torch.empty((q.shape[0], hq, dim), dtype=q.dtype, device=q.device)
    lse = torch.empty((q.shape[0], hq), dtype=torch.float32, device=q.device)
    row = 0
    for r, (length, new) in enumerate(zip(s["lens_list"], s["new_list"])):
        low = max(0, length - new - window + 1) if window else 0
        pages = s["table"][r, low // page:-(-length // page)].long()
        low = low // page * page

        def rebuilt(codes, scales, cent):
            code = codes[pages].transpose(0, 1).reshape(hkv, -1, dim // 2)[:, :length - low].int()
            scale = scales[pages].transpose(0, 1).reshape(hkv, -1, 1)[:, :length - low].float()
            values = cent.to(q.dtype).float()  # centroids in the rows' type
            return torch.stack([values[code & 15], values[code >> 4]], -1).reshape(hkv, length - low, dim) * scale

        keys, values = rebuilt(s["kc"], s["ks"], s["kcent"]), rebuilt(s["vc"], s["vs"], s["vcent"])
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


def _plain_fork(s):
    page, table, free, parents = s["case"]["page"], s["table"], s["free"], s["parents"].long()
    seats, width = table.shape
    pages, dev = free.numel(), table.device
    held = s["lens"].long()
    have = parents >= 0
    kept = torch.where(have, held[parents.clamp(min=0)], 0)
    if s["keep"] is not None:
        kept = torch.minimum(kept, s["keep"].long().clamp(min=0))
    block = torch.arange(width, device=dev)[None, :]
    upto = (kept + page - 1) // page
    new = torch.where(block < upto[:, None], table[parents.clamp(min=0)], -1)
    whole = block < (kept // page)[:, None]

    def mark(where, entries):
        flags = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
        flags[torch.where(where, entries, pages).reshape(-1).long()] = True
        return flags[:-1]

    held_before = mark(block < ((held + page - 1) // page)[:, None], table)
    held_whole, held_after = mark(whole, new), mark(block < upto[:, None], new)
    freed = held_before & ~held_after
    # the free list takes the freed pages, in order
    count = s["count"].long()
    at = torch.where(freed, count + freed.cumsum(0) - 1, pages)
    room = torch.cat([free, free[:1]])
    room[at] = torch.arange(pages, dtype=torch.int32, device=dev)
    free.copy_(room[:-1])
    count = count + freed.sum()
    # last pages not full, held by someone else too: all but the first such seat get a copy
    part = kept % page != 0
    seat = torch.arange(seats, device=dev)
    tail = new.gather(1, (upto - 1).clamp(min=0)[:, None])[:, 0].long()
    tail = torch.where(part, tail, pages)
    first = torch.full((pages + 1,), seats, dtype=torch.long, device=dev).scatter_reduce(0, tail, seat, "amin")
    other = part & (held_whole[tail.clamp(max=pages - 1)] | (first[tail] < seat))
    nth = other.long().cumsum(0) - 1
    granted = other & (nth < count)
    to = free[(count - 1 - nth).clamp(0, pages - 1)]
    copies = torch.where(granted[:, None], torch.stack([tail.int(), to], 1), -1)
    last = block == (upto - 1)[:, None]
    new = torch.where(last & granted[:, None], to[:, None], torch.where(last & (other & ~granted)[:, None], -1, new))
    kept = torch.where(other & ~granted, kept // page * page, kept)
    return kept.int(), new, (count - granted.sum()).int(), copies, free


def _plain_compact(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    pages, dev = free.numel(), free.device
    number = torch.arange(pages, device=dev)
    held = torch.ones(pages + 1, dtype=torch.bool, device=dev)
    held[torch.where(number < s["count"], free.long(), pages)] = False
    held = held[:-1]
    used = held.sum()
    hole, mover = ~held & (number < used), held & (number >= used)
    nth_hole, nth_mover = hole.cumsum(0) - 1, mover.cumsum(0) - 1
    holes = torch.full((pages + 1,), -1, dtype=torch.long, device=dev)
    holes[torch.where(hole, nth_hole, pages)] = number
    target = torch.where(mover, holes[nth_mover.clamp(min=0)], torch.where(held, number, -1))
    moves = torch.full((pages // 2 + 1, 2), -1, dtype=torch.int32, device=dev)
    moves[torch.where(mover, nth_mover, pages // 2)] = torch.stack([number, target], 1).int()
    block = torch.arange(table.shape[1], device=dev)[None, :]
    mine = block < ((s["lens"].long() + page - 1) // page)[:, None]
    new = torch.where(mine, target[table.clamp(min=0).long()].int(), table)
    left = torch.where(number < pages - used, pages - 1 - number, -1).int()
    return new, left, (pages - used).int().reshape(1), moves[:-1], target.int()


def _plain_copy(s):
    live = s["pairs"][:, 0] >= 0
    pairs = s["pairs"][live].long()
    for pool in (s["codes"], s["scales"]):
        pool[:, pairs[:, 1]] = pool[:, pairs[:, 0]]
    return s["codes"], s["scales"]


_own = {"append": _own_append, "attend": _own_attend, "fork": _own_fork, "compact": _own_compact, "copy": _own_copy}
_plain = {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact,
          "copy": _plain_copy}


# ---------------------------------------------------------------- the least work of one pass


def work(case):
    op = case["op"]
    if op == "fork":
        shared, apart = _fork_lengths(case)
        page, seats = case["page"], case["groups"] * case["beams"]
        n = shared[:, None] + apart
        if case["kind"] == "samples":
            n = np.repeat(n[:, :1], case["beams"], 1)
            before = int(_pages(n[:, 0], page).sum())
        else:
            before = int(_pages(n, page).sum())
        width = int(_pages(shared + apart.max(1), page).max())
        return {"bytes": 4 * (before + seats * width + 3 * seats + 2 * seats), "flops": 0}
    if op == "compact":
        lens = _compact_lengths(case)
        entries = int(_pages(lens, case["page"]).sum())
        pages = max(1, int(round(entries / (1 - case["free"])))) + 1
        width = max(1, int(_pages(lens, case["page"]).max()))
        # the table read and written, the free list read and written, the map and the moves written
        return {"bytes": 4 * (2 * len(lens) * width + len(lens) + (pages - entries) + pages + pages + pages), "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "copy":
        live = int(math.ceil(case["live"] * case["rows"]))
        page_bytes = 2 * case["heads"] * case["page"] * (case["dim"] // 2 + size)
        return {"bytes": 2 * live * case["layers"] * page_bytes + 8 * case["rows"], "flops": 0}
    if op == "append":
        rows = 2 * case["tokens"] * case["heads"]
        turns = int(math.log2(case["dim"])) if case["rotate"] else 0
        return {"bytes": rows * (case["dim"] * size + case["dim"] // 2 + size) + 8 * case["tokens"],
                "flops": rows // 2 * case["dim"] * turns + rows * case["dim"] * 3}
    held, new = _lengths(case)
    seen = tokens = 0
    for h, n in zip(held.tolist(), new.tolist()):
        low = max(0, h - case["window"] + 1) if case["window"] else 0
        tokens += h + n - low
        pos = np.arange(h, h + n)
        seen += int(np.minimum(pos + 1, case["window"] or h + n + 1).sum())
    codes = 2 * tokens * case["hkv"] * (case["dim"] // 2 + size)
    rows = int(new.sum()) * case["hq"]
    return {"bytes": codes + rows * (2 * case["dim"] * size + 4), "flops": 4 * seen * case["hq"] * case["dim"]}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "fork": _exact_fork, "compact": _exact_compact,
            "copy": _exact_copy}[case["op"]](s)


def _fl(x):
    """One fp32 rounding of a 64-bit result (exact for one operation on fp32
    values: 53 bits are more than twice 24 and two)."""
    return x.float().double()


def _exact_append(s):
    """The rule is stated in fp32 steps: each is one operation in 64 bits, rounded to 32."""
    case = s["case"]
    dim, page = case["dim"], case["page"]
    slots = s["slots"].cpu().numpy()
    at = slots >= 0
    out = []
    for x, cent, codes, scales, signs in (("k", "kcent", "kc", "ks", s["signs"]), ("v", "vcent", "vc", "vs", None)):
        dtype = s[x].dtype
        y = s[x].double()
        if signs is not None:
            y = _fl(y * signs.double())
            index = torch.arange(dim, device=y.device)
            stride = 1
            while stride < dim:
                partner = y[..., index ^ stride]
                y = _fl(torch.where(index & stride == 0, y + partner, partner - y))
                stride *= 2
            y = _fl(y * float(np.float32(1.0 / math.sqrt(dim))))
        total = _fl(y * y)
        n = dim
        while n > 1:
            n //= 2
            pairs = total.reshape(*total.shape[:-1], n, 2)
            total = _fl(pairs[..., 0] + pairs[..., 1])
        scale = _fl(torch.sqrt(_fl(total / dim))).to(dtype).double()
        scale = torch.where(torch.isfinite(scale), scale, 0.0)
        z = torch.where(scale > 0, _fl(y * _fl(1.0 / scale)), 0.0)
        dist = torch.stack([_fl(_fl(z - c) ** 2) for c in s[cent].double()])
        lowest = dist.min(0).values
        code = (dist == lowest).to(torch.uint8).argmax(0).cpu().numpy().astype(np.uint8)  # the first of equals
        new_codes, new_scales = s[codes].cpu().numpy().copy(), s[scales].double().cpu().numpy()
        packed = code[..., 0::2] | code[..., 1::2] << 4
        new_codes[slots[at] // page, :, slots[at] % page] = packed[at]
        new_scales[slots[at] // page, :, slots[at] % page] = scale[..., 0].cpu().numpy()[at]
        out.append((new_codes, new_scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _exact_attend(s):
    case = s["case"]
    hq, hkv, dim, page, window = (case[k] for k in ("hq", "hkv", "dim", "page", "window"))
    group = hq // hkv
    q = s["q"]
    out = torch.zeros((q.shape[0], hq, dim), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device=q.device)
    cents = [s[c].to(q.dtype).double() for c in ("kcent", "vcent")]
    row = 0
    for r, (length, new) in enumerate(zip(s["lens_list"], s["new_list"])):
        where = torch.arange(length, device=q.device)
        page_of = s["table"][r].long()[where // page]
        for h in range(hkv):
            rebuilt = []
            for codes, scales, cent in ((s["kc"], s["ks"], cents[0]), (s["vc"], s["vs"], cents[1])):
                byte = codes[page_of, h, where % page].long()
                rows = torch.empty((length, dim), dtype=torch.float64, device=q.device)
                rows[:, 0::2], rows[:, 1::2] = cent[byte % 16], cent[byte // 16]
                rebuilt.append(rows * scales[page_of, h, where % page].double()[:, None])
            keys, values = rebuilt
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


def _exact_fork(s):
    page = s["case"]["page"]
    lens, parents, table, free = (s[k].cpu().tolist() for k in ("lens", "parents", "table", "free"))
    top = int(s["count"].item())
    keep = s["keep"].cpu().tolist() if s["keep"] is not None else None
    width = len(table[0])
    kept, rows = [], []
    for d, p in enumerate(parents):
        n = lens[p] if p >= 0 else 0
        if keep is not None:
            n = min(n, max(0, keep[d]))
        kept.append(n)
        rows.append(table[p][:-(-n // page)] if n else [])
    before = {pg for n, row in zip(lens, table) for pg in row[:-(-n // page)]}
    after = {pg for row in rows for pg in row}
    for pg in sorted(before - after):
        free[top] = pg
        top += 1
    whole = {pg for n, row in zip(kept, rows) for pg in row[:n // page]}
    copies, owned = [], set()
    for d, (n, row) in enumerate(zip(kept, rows)):
        copies.append([-1, -1])
        if n % page == 0:
            continue
        tail = row[-1]
        if tail not in whole and tail not in owned:
            owned.add(tail)
        elif top > 0:
            top -= 1
            copies[d] = [tail, free[top]]
            row[-1] = free[top]
        else:
            row.pop()
            kept[d] = n // page * page
    new = [row + [-1] * (width - len(row)) for row in rows]
    return (np.array(kept, np.int32), np.array(new, np.int32), np.array([top], np.int32), np.array(copies, np.int32),
            np.array(free, np.int32))


def _exact_compact(s):
    page = s["case"]["page"]
    lens, table, free = (s[k].cpu().tolist() for k in ("lens", "table", "free"))
    pages = len(free)
    idle = set(free[:int(s["count"].item())])
    used = pages - len(idle)
    target = [-1 if p in idle else p for p in range(pages)]
    holes = (p for p in range(used) if p in idle)
    moves = []
    for p in range(used, pages):
        if p not in idle:
            target[p] = next(holes)
            moves.append([p, target[p]])
    moves += [[-1, -1]] * (pages // 2 - len(moves))
    new = [[target[pg] if b < -(-n // page) else pg for b, pg in enumerate(row)] for n, row in zip(lens, table)]
    left = list(range(pages - 1, used - 1, -1)) + [-1] * used
    return (np.array(new, np.int32), np.array(left, np.int32), np.array([pages - used], np.int32),
            np.array(moves, np.int32).reshape(-1, 2), np.array(target, np.int32))


def _exact_copy(s):
    pairs = s["pairs"].cpu().tolist()
    pools = [s["codes"].clone(), s["scales"].clone()]
    for pool in pools:
        for a, b in pairs:
            if a >= 0:
                pool[:, b].copy_(pool[:, a])
    return pools[0].cpu().numpy(), pools[1].double().cpu().numpy()
