"""The paged cache in 4 bits on the GPU: the append exactly, attention within the bounds
derived in ``scalar_reference``, each against a plain host form; and a whole step."""
import math

import numpy as np
import pytest
import torch

import scalar_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
CENTS = [-2.73, -2.07, -1.62, -1.26, -0.94, -0.66, -0.39, -0.13, 0.13, 0.39, 0.66, 0.94, 1.26, 1.62, 2.07, 2.73]


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def f32(a):
    return torch.tensor(a, dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------ append


def check_append(vq, k, v, slots, k_cents, v_cents, signs, pages, page, shared=False, pad=0):
    """One append into pools of a pattern; rows without a slot keep it.  `shared`: keys and
    values in one pool; `pad`: bytes (elements) behind each page."""
    tokens, heads, dim = k.shape
    dtype = k.dtype
    ns, rows = dim // 2, heads * page
    sets = 2 if shared else 1
    pool = torch.full((pages, sets * rows * ns + pad), 0xA5, dtype=torch.uint8, device="cuda")
    spool = torch.full((pages, sets * rows + pad), 7.0, dtype=dtype, device="cuda")
    pools = [pool, pool if shared else pool.clone()]
    spools = [spool, spool if shared else spool.clone()]
    codes = [p.as_strided((pages, heads, page, ns), (p.shape[1], page * ns, ns, 1), (i if shared else 0) * rows * ns)
             for i, p in enumerate(pools)]
    scales = [p.as_strided((pages, heads, page), (p.shape[1], page, 1), (i if shared else 0) * rows) for i, p in enumerate(spools)]
    vq.vq_paged_scalar_append(k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"), f32(k_cents), f32(v_cents), *codes,
                              *scales, k_signs=None if signs is None else f32(signs.tolist()))
    for x, cents, sg, c, s in ((k, k_cents, signs, codes[0], scales[0]), (v, v_cents, None, codes[1], scales[1])):
        want, want_s = ref.encode_rows(x.cpu(), cents, sg)
        full = np.full((pages, heads, page, ns), 0xA5, np.uint8)
        full_s = torch.full((pages, heads, page), 7.0, dtype=dtype)
        for t, slot in enumerate(slots):
            if 0 <= slot < pages * page:
                full[slot // page, :, slot % page] = ref.pack(want[t])
                full_s[slot // page, :, slot % page] = want_s[t]
        assert np.array_equal(c.cpu().numpy(), full)
        assert torch.equal(s.cpu().view(torch.uint8), full_s.view(torch.uint8))
    if pad:
        for p in pools:
            assert (p[:, -pad:] == 0xA5).all()
        for p in spools:
            assert (p[:, -pad:] == 7.0).all()


def rows(seed, tokens, heads, dim, dtype):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((tokens, heads, dim)) * np.exp(rng.standard_normal((tokens, heads, 1)))
    x[:, :, rng.integers(0, dim)] *= 8  # an outlier channel
    return torch.from_numpy(x).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("dim", [2, 4, 8, 16, 30, 32, 48, 64, 80, 96, 128, 192, 256, 320, 512])
@pytest.mark.parametrize("rotate", [False, True])
def test_append(vq, dtype, dim, rotate):
    if rotate and dim & (dim - 1):
        pytest.skip("a rotation is of a power of two")
    rng = np.random.default_rng(dim)
    tokens, heads, page = 37, 3, 16
    k, v = rows(dim, tokens, heads, dim, dtype), rows(dim + 1, tokens, heads, dim, dtype)
    slots = rng.permutation(4 * page)[:tokens].tolist()
    slots[3], slots[11], slots[12] = -1, 4 * page, -(1 << 40)
    signs = rng.choice([-1.0, 1.0], dim) if rotate else None
    check_append(vq, k, v, slots, CENTS, sorted(rng.standard_normal(16).tolist()), signs, 4, page)


@pytest.mark.parametrize("n_c", [1, 2, 7, 15, 16])
@pytest.mark.parametrize("kind", ["sorted", "any order", "equal", "wide", "far"])
def test_append_centroids(vq, n_c, kind):
    rng = np.random.default_rng(n_c)
    c = rng.standard_normal(n_c)
    c = {"sorted": np.sort(c), "any order": c, "equal": np.round(c), "wide": c * 10.0 ** rng.integers(-30, 30, n_c),
         "far": 1e6 + c}[kind].tolist()
    k, v = rows(1, 21, 2, 128, F16), rows(2, 21, 2, 128, BF16).half()
    check_append(vq, k, v, list(range(21)), c, list(reversed(c)), rng.choice([-1.0, 1.0], 128), 2, 16)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_append_special_rows(vq, dtype, dim):
    """Rows of zeros, NaN, infinities, the largest and the least numbers, and one element alone."""
    top = torch.finfo(dtype).max
    low = torch.finfo(dtype).smallest_normal
    x = torch.zeros((12, 2, dim))
    x[1, 0, 3] = math.nan
    x[2, 0, 5] = math.inf
    x[2, 1, 5] = -math.inf
    x[3] = top
    x[4, 0] = low
    x[4, 1] = low / 4
    x[5, :, 7] = 1.0
    x[6, :, dim - 1] = -low / 8
    x[7] = torch.randn(2, dim, generator=torch.Generator().manual_seed(0)) * 1e-3
    x[8, 0, 0], x[8, 0, 1] = top, -top
    x[9] = -0.0
    x[10, 0] = 1e-20 if dtype != F16 else 1e-7
    x[11] = torch.randn(2, dim, generator=torch.Generator().manual_seed(1))
    x = x.to(dtype).cuda()
    signs = np.random.default_rng(3).choice([-1.0, 1.0], dim) if dim & (dim - 1) == 0 else None
    for sg in [None] if signs is None else [None, signs]:
        check_append(vq, x, x.flip(0).contiguous(), list(range(12)), CENTS, CENTS, sg, 1, 16)


@pytest.mark.parametrize("dtype, dim", [(F16, 128), (BF16, 64), (F32, 256), (F16, 80)])
def test_append_layouts(vq, dtype, dim):
    """Rows inside a packed projection, off 16-byte alignment, in one pool for keys and
    values, in padded pages."""
    tokens, heads = 50, 2
    packed = rows(9, tokens, 3 * heads + 1, dim, dtype)
    flat = rows(10, tokens, heads, dim, dtype).reshape(-1)
    off = torch.empty(flat.numel() + 1, dtype=dtype, device="cuda")[1:].copy_(flat).view(tokens, heads, dim)
    slots = np.random.default_rng(1).permutation(64)[:tokens].tolist()
    for k, v in ((packed[:, heads:2 * heads], packed[:, 2 * heads:3 * heads]), (off, packed[:, 1:1 + heads])):
        for shared, pad in ((False, 0), (True, 0), (False, 3), (True, 16)):
            check_append(vq, k, v, slots, CENTS, CENTS, None, 4, 16, shared, pad)


@pytest.mark.parametrize("tokens, heads, page", [(1, 1, 1), (3, 1, 1), (1, 64, 32), (2000, 5, 8), (700, 3, 1024)])
def test_append_sizes(vq, tokens, heads, page):
    k, v = rows(4, tokens, heads, 64, F16), rows(5, tokens, heads, 64, F16)
    pages = -(-tokens // page) + 1
    slots = np.random.default_rng(2).permutation(pages * page)[:tokens].tolist()
    check_append(vq, k, v, slots, CENTS, CENTS, np.random.default_rng(2).choice([-1.0, 1.0], 64), pages, page)


def test_append_nothing(vq):
    k = torch.empty((0, 2, 64), dtype=F16, device="cuda")
    codes, scales = torch.zeros((3, 2, 16, 32), dtype=torch.uint8, device="cuda"), torch.zeros((3, 2, 16), dtype=F16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    vq.vq_paged_scalar_append(k, k, none, f32(CENTS), f32(CENTS), codes, codes.clone(), scales, scales.clone())
    assert not codes.any()
    k = torch.ones((2, 2, 64), dtype=F16, device="cuda")
    vq.vq_paged_scalar_append(k, k, none.new_zeros(2), f32(CENTS), f32(CENTS), codes[:0], codes[:0], scales[:0], scales[:0])


def test_append_matches_the_hadamard_quantizer(vq):
    """Rows whose rotation has a root mean square of one exactly: the codes are
    vq_hadamard_quantize's."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((9, 2, 64), dtype=F16, device="cuda")
    x[:, :, 5] = 8.0  # its rotation is +-1 everywhere
    x[4:, :, 5] = 0.0
    x[4:, :, 9] = -8.0
    signs = torch.randint(0, 2, (64,), generator=gen, device="cuda").float() * 2 - 1
    codes = [torch.zeros((1, 2, 16, 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((1, 2, 16), dtype=F16, device="cuda") for _ in range(2)]
    vq.vq_paged_scalar_append(x, x, torch.arange(9, device="cuda"), f32(CENTS), f32(CENTS), *codes, *scales, k_signs=signs)
    want = vq.vq_hadamard_quantize(x.view(-1, 64), signs, f32(CENTS)).view(9, 2, 64)
    got = codes[0][0, :, :9].transpose(0, 1)
    assert torch.equal(got & 15, want[..., 0::2]) and torch.equal(got >> 4, want[..., 1::2])
    assert (scales[0][0, :, :9] == 1).all()


# ------------------------------------------------------------------ attention


def cache(rng, pages, hkv, page, dim, dtype, spread=0.5):
    codes = [rng.integers(0, 256, (pages, hkv, page, dim // 2)).astype(np.uint8) for _ in range(2)]
    # (products with the centroids finite in every type, as the append leaves them)
    scales = [torch.from_numpy(np.minimum(np.exp(spread * rng.standard_normal((pages, hkv, page))), 15000.0)).to(dtype)
              for _ in range(2)]
    return codes, scales


def tensor_takes(dtype, dim, page):
    return dtype is not F32 and dim in (64, 128, 256) and page >= 16


def check_attention(vq, lens, new, hq, hkv, dim, page, dtype, window=0, n_c=16, seed=0, holes=0, extra=0, max_new=0, scale=0.0,
                    hide=None, slots=None, spread=0.5):
    rng = np.random.default_rng([seed, dim, page])
    width = max([1] + [-(-n // page) for n in lens]) + 1
    need = [max(0, -(-n // page)) for n in lens]
    pages = sum(need) + 2
    order = rng.permutation(pages).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + rng.choice([-1, pages, 1 << 30], width - n).tolist())
        at += n
    for _ in range(holes):
        r = int(rng.integers(len(lens)))
        table[r][int(rng.integers(width))] = int(rng.choice([-1, pages, -(1 << 31)]))
    (kc, vc), (ks, vs) = cache(rng, pages, hkv, page, dim, dtype, spread)
    cents = [sorted(rng.standard_normal(n_c).tolist()) for _ in range(2)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    tokens = cu[-1] + extra
    q = torch.from_numpy(rng.standard_normal((tokens, hq, dim))).to(dtype)
    held = list(lens)
    if slots is not None:  # refused requests hold nothing
        held = [0 if cu[r] < len(slots) and cu[r + 1] > cu[r] and slots[cu[r]] < 0 else n for r, n in enumerate(lens)]
    want, want_lse, tol, tol_lse = ref.attention(q.double().numpy(), cu, held, table, kc, vc, ks.double().numpy(),
                                                 vs.double().numpy(), *cents, dtype, window, scale, tensor_takes(dtype, dim, page))
    # what nobody may see: scales behind the last token of a request and in pages of nobody
    bad = torch.ones((pages, page), dtype=torch.bool)
    for n, row in zip(lens, table):
        for t in range(max(0, min(n, width * page))):
            if 0 <= row[t // page] < pages:
                bad[row[t // page], t % page] = False
    for s, value in ((ks, math.nan), (vs, math.inf)):
        s.copy_(torch.where(bad[:, None, :], torch.tensor(value, dtype=dtype), s))
    d_table = i32(table) if table else torch.empty((0, width), dtype=torch.int32, device="cuda")
    args = (q.cuda(), i32(cu), i32(list(lens)), d_table, torch.from_numpy(kc).cuda(),
            torch.from_numpy(vc).cuda(), ks.cuda(), vs.cuda(), f32(cents[0]), f32(cents[1]))
    kw = dict(max_new=max_new, window=window, scale=scale, return_lse=True)
    if slots is not None:
        kw["slots"] = torch.tensor(slots, dtype=torch.int64, device="cuda")
    out, lse = vq.vq_paged_scalar_attention(*args, **kw)
    got = out.double().cpu().numpy()
    tol = tol + ref.HALF_EPS[dtype] * (np.abs(want) + tol) + ref.HALF_STEP[dtype]
    bad = np.abs(got - want) > tol
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], np.abs(got - want).max(), tol.max())
    got_lse = lse.double().cpu().numpy()
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), none)
    assert (np.abs(got_lse - want_lse)[~none] <= tol_lse[~none]).all()
    assert not got[none].any()
    again = vq.vq_paged_scalar_attention(*args, **kw)
    assert torch.equal(out.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(lse.view(torch.uint8), again[1].view(torch.uint8))
    return args, out


SHAPES = [(F16, 128, 16), (BF16, 128, 64), (F16, 64, 32), (BF16, 64, 16), (F16, 256, 16), (BF16, 256, 32), (F32, 128, 16),
          (F16, 128, 8), (BF16, 96, 16), (F16, 512, 16), (F32, 2, 1), (F16, 30, 4)]


@pytest.mark.parametrize("dtype, dim, page", SHAPES)
@pytest.mark.parametrize("group", [1, 3, 4, 8, 11])
def test_attention_decode(vq, dtype, dim, page, group):
    check_attention(vq, [1, 17, 300, 128, 129, 64], [1] * 6, 2 * group, 2, dim, page, dtype, seed=group, max_new=1)


@pytest.mark.parametrize("dtype, dim, page", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 37, 200])
def test_attention_mixed(vq, dtype, dim, page, window):
    """One token, drafts and runs in one call; pages missing; rows behind the last request."""
    check_attention(vq, [5, 260, 130, 0, 33, 150], [1, 4, 60, 0, 33, 2], 6, 2, dim, page, dtype, window, seed=1, holes=3, extra=3)


@pytest.mark.parametrize("dtype, dim, page", SHAPES[:6])
@pytest.mark.parametrize("known", [0, 1])
def test_attention_chunks(vq, dtype, dim, page, known):
    new = [150, 1, 300, 40]
    check_attention(vq, [400, 350, 300, 90], new, 4, 2, dim, page, dtype, seed=2, max_new=max(new) * known)


@pytest.mark.parametrize("dtype, dim, page", [(F16, 128, 16), (BF16, 256, 16), (F32, 64, 16), (F16, 64, 16)])
def test_attention_lengths(vq, dtype, dim, page):
    """Lengths around the tiles; more new tokens than the length; no tokens; a negative length."""
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 3, -4]
    new = [1, 1, 2, 1, 16, 3, 63, 1, 2, 1, 5, 1, 7, 2]
    check_attention(vq, lens, new, 4, 1, dim, page, dtype, seed=3)


@pytest.mark.parametrize("dtype, dim", [(F16, 128), (BF16, 64), (F16, 256), (F32, 64)])
def test_attention_few_centroids(vq, dtype, dim):
    check_attention(vq, [200, 90], [1, 40], 4, 2, dim, 16, dtype, n_c=5, seed=4)


@pytest.mark.parametrize("dtype, dim", [(F16, 128), (BF16, 128), (F16, 64), (BF16, 256)])
@pytest.mark.parametrize("spread", [2.0, 4.0])
def test_attention_uneven_scales(vq, dtype, dim, spread):
    """Scales over several powers of ten: the weights of the largest keys take all."""
    check_attention(vq, [300, 140, 90], [1, 30, 2], 4, 2, dim, 16, dtype, seed=5, spread=spread)


@pytest.mark.parametrize("dtype, dim, page", [(F16, 128, 16), (BF16, 256, 16), (F32, 64, 16)])
def test_attention_refused(vq, dtype, dim, page):
    new = [3, 40, 1, 1]
    slots = [0, 1, 2] + [-1] * 40 + [9] + [-1]
    check_attention(vq, [50, 90, 20, 64], new, 4, 2, dim, page, dtype, seed=6, slots=slots)


def test_attention_scale(vq):
    for dtype in (F16, F32):
        check_attention(vq, [100, 70], [1, 30], 4, 2, 128, 16, dtype, scale=0.02, seed=7)


def test_attention_nothing(vq):
    cents = f32(CENTS)
    codes, scales = torch.zeros((2, 2, 16, 32), dtype=torch.uint8, device="cuda"), torch.zeros((2, 2, 16), dtype=F16, device="cuda")
    q = torch.empty((0, 4, 64), dtype=F16, device="cuda")
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    out = vq.vq_paged_scalar_attention(q, i32([0]), i32([]), none, codes, codes, scales, scales, cents, cents)
    assert out.shape == (0, 4, 64)
    q = torch.ones((3, 4, 64), dtype=F16, device="cuda")
    out, lse = vq.vq_paged_scalar_attention(q, i32([0]), i32([]), none, codes, codes, scales, scales, cents, cents, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    out = vq.vq_paged_scalar_attention(q, i32([0, 3]), i32([3]), i32([[1]]), codes[:0], codes[:0], scales[:0], scales[:0], cents, cents)
    assert not out.any()


@pytest.mark.parametrize("dtype, dim", [(F16, 128), (BF16, 256), (F32, 64)])
def test_attention_special_queries(vq, dtype, dim):
    """NaN and infinities in a row of q stay in that row, and do not depend on its neighbours."""
    args, out = check_attention(vq, [300, 200], [3, 150], 4, 2, dim, 16, dtype, seed=8)
    q = args[0].clone()
    q[1, 2, 0] = math.nan
    q[80, 0] = math.inf
    q[81, 3, 1] = -math.inf
    got = vq.vq_paged_scalar_attention(q, *args[1:])
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[80, 0] = hit[81, 3] = True
    assert torch.equal(got[~hit], out[~hit])
    assert torch.isnan(got[1, 2]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new", [1, 60])
def test_attention_strides(vq, dtype, new):
    """Queries inside a packed projection; keys and values in one pool; pools off 16-byte
    alignment take the general kernel."""
    args, out = check_attention(vq, [300, 64], [new, 1], 4, 2, 128, 16, dtype, seed=9)
    q, cu, lens, table, kc, vc, ks, vs, kcent, vcent = args
    packed = torch.randn((q.shape[0], 9, 128), device="cuda").to(dtype)
    packed[:, 3:7] = q
    pool = torch.stack([kc, vc], 1)
    spool = torch.stack([ks, vs], 1)
    got = vq.vq_paged_scalar_attention(packed[:, 3:7], cu, lens, table, pool[:, 0], pool[:, 1], spool[:, 0], spool[:, 1], kcent, vcent)
    assert torch.equal(got, out)
    flat = torch.empty(kc.numel() + 8, dtype=torch.uint8, device="cuda")
    moved = flat[8:].view(kc.shape).copy_(kc)
    got = vq.vq_paged_scalar_attention(q, cu, lens, table, moved, vc, ks, vs, kcent, vcent)
    bound = 4 * 8 * ref.HALF_EPS[dtype]  # both within a few roundings of values below 8
    assert (got.float() - out.float()).abs().max() <= bound
    wide = torch.empty((kc.shape[0], 33), dtype=dtype, device="cuda")
    got = vq.vq_paged_scalar_attention(q, cu, lens, table, kc, vc, wide[:, :32].view(-1, 2, 16).copy_(ks),
                                       torch.empty_like(wide)[:, :32].view(-1, 2, 16).copy_(vs), kcent, vcent)
    assert (got.float() - out.float()).abs().max() <= bound


@pytest.mark.parametrize("dtype, dim", [(F16, 128), (BF16, 64), (F16, 256), (F32, 128)])
def test_step(vq, dtype, dim):
    """Appends of prompts and tokens with rotated keys, then attention with rotated queries:
    as the definition on rows that were encoded on the host; a fork and a compaction between."""
    rng = np.random.default_rng(11)
    hq, hkv, page, seats, width = 4, 2, 16, 4, 8
    pages = seats * width + 3
    signs = rng.choice([-1.0, 1.0], dim)
    d_signs = f32(signs.tolist())
    pool = torch.zeros((pages, 2, hkv, page, dim // 2), dtype=torch.uint8, device="cuda")
    spool = torch.zeros((pages, 2, hkv, page), dtype=dtype, device="cuda")
    table, free = torch.full((seats, width), -1, dtype=torch.int32, device="cuda"), torch.arange(pages, dtype=torch.int32, device="cuda")
    lens, count = i32([0] * seats), i32([pages])
    cents = f32(CENTS)
    lines = [[] for _ in range(seats)]
    for n, new in enumerate(([40, 3, 0, 17], [1, 1, 0, 1], [1, 5, 2, 1], [1, 1, 1, 1], [20, 1, 1, 1])):
        if n == 2:  # seat 2 is empty: it goes on from seat 0's, seat 3 from a part of it
            p, keep = [0, 1, 0, 0], [99, 99, 41, 21]
            lens, table, count, copies = vq.vq_paged_fork(lens, i32(p), table, page, free, count, keep_lens=i32(keep))
            vq.vq_paged_copy(copies, [pool, spool])
            lines = [list(lines[a][:k]) for a, k in zip(p, keep)]
        if n == 3:
            table, free, count, moves, _ = vq.vq_paged_compact(lens, table, page, free, count)
            vq.vq_paged_copy(moves, [pool, spool])
        tokens = sum(new)
        x = torch.from_numpy(rng.standard_normal((tokens, hq + 2 * hkv, dim))).to(dtype).cuda()
        lens, count, cu, slots = vq.vq_paged_reserve(lens, i32(new), free, count, table, page, tokens)
        k, v = x[:, hq:hq + hkv], x[:, hq + hkv:]
        vq.vq_paged_scalar_append(k, v, slots, cents, cents, pool[:, 0], pool[:, 1], spool[:, 0], spool[:, 1], k_signs=d_signs)
        q = vq.vq_hadamard_rotate(x[:, :hq].reshape(-1, dim).contiguous(), d_signs).to(dtype).view(tokens, hq, dim)
        out = vq.vq_paged_scalar_attention(q, cu, lens, table, pool[:, 0], pool[:, 1], spool[:, 0], spool[:, 1], cents, cents,
                                           max_new=max(new), slots=slots)
        kcode, kscale = ref.encode_rows(k.cpu(), CENTS, signs)
        vcode, vscale = ref.encode_rows(v.cpu(), CENTS)
        book = torch.tensor(CENTS).to(dtype).double().numpy()
        krows = book[kcode] * kscale.double().numpy()[..., None]
        vrows = book[vcode] * vscale.double().numpy()[..., None]
        row = 0
        for r, m in enumerate(new):
            for i in range(m):
                lines[r].append((krows[row], vrows[row]))
                kk, vv = (np.stack([a[j] for a in lines[r]]) for j in (0, 1))  # [tokens, hkv, dim]
                for h in range(hq):
                    s = kk[:, h // 2] @ q[row, h].double().cpu().numpy() / math.sqrt(dim)
                    w = np.exp(s - s.max())
                    want = w @ vv[:, h // 2] / w.sum()
                    # a wrong token would be off by about 1; roundings of values below 8: 2^-8 each in bf16
                    assert np.abs(out[row, h].double().cpu().numpy() - want).max() < 8 * 4 * 2.0 ** -8
                row += 1
        assert lens.tolist() == [len(a) for a in lines]


def test_example_serving_loop_in_4_bits(vq):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")
    spec = importlib.util.spec_from_file_location("paged_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    for requests in ("5", "8"):
        report = module.main(["--scalar", "--steps", "20", "--requests", requests, "--prompt", "300", "--answer", "30"])
        assert report["tokens"] > 500
