"""The paged code cache on the GPU: reservation and trimming of pages and the
append exactly, attention within a bound derived in ``paged_reference``, each
against a plain host form; and the whole step captured in a CUDA graph."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
HALF_STEP = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 0.0}


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    oracle.build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


def i32(a, device="cuda"):
    return torch.tensor(a, dtype=torch.int32, device=device)


# ------------------------------------------------------------------ pages


def pool(rng, lens, page, width, spare):
    """A block table holding the pages of `lens`, and the free list."""
    need = [min(ref.blocks_of(max(n, 0), page), width) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    free = order[at:] + [-1] * at
    return table, free, pages - at


RESERVE = [
    # lens, new, page, width, spare
    ([0], [1], 16, 1, 1),
    ([16], [1], 16, 1, 4),                      # the table is full
    ([15], [1], 16, 1, 0),                      # no page needed
    ([0], [1], 16, 4, 0),                       # no page there
    ([0, 0, 0], [0, 0, 0], 16, 2, 3),
    ([5, 31, 32, 0, 100], [3, 1, 1, 0, 64], 32, 6, 3),
    ([0, 0, 3, 0], [40, 40, 1, 8], 8, 5, 5),    # the second and fourth are refused, the third needs none
    ([0, 0, 0], [100, 8, 8], 8, 4, 9),          # the first does not fit the table
    ([-3, 7], [5, -2], 4, 3, 4),                # negative lengths count as none
    ([0, 9], [1000, 3], 1, 1100, 1005),         # a page a token
    ([3] * 70, [1] * 70, 4, 3, 40),
]


@pytest.mark.parametrize("case", range(len(RESERVE) + 3))
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(vq, case, in_place):
    rng = np.random.default_rng(100 + case)
    if case < len(RESERVE):
        lens, new, page, width, spare = RESERVE[case]
    else:  # more requests than threads, several blocks of the cluster
        n = [1025, 2500, 8192][case - len(RESERVE)]
        page = 16
        lens = rng.integers(0, 60, n).tolist()
        new = rng.integers(0, 40, n).tolist()
        width, spare = 6, n
    table, free, count = pool(rng, lens, page, width, spare)
    want = ref.reserve(lens, new, free, count, table, page)
    total = sum(max(n, 0) for n in new)
    for extra in (0, 5):
        d_lens, d_new, d_free, d_count, d_table = i32(lens), i32(new), i32(free), i32([count]), i32(table)
        kw = dict(lens_out=d_lens, free_count_out=d_count) if in_place else {}
        got = vq.vq_paged_reserve(d_lens, d_new, d_free, d_count, d_table, page, total + extra, **kw)
        assert got[0].tolist() == want[0]
        assert got[1].tolist() == [want[1]]
        assert got[2].tolist() == want[2]
        assert got[3].tolist() == want[3] + [-1] * extra
        assert d_table.tolist() == want[4]
        if not in_place:
            assert d_lens.tolist() == lens and d_count.tolist() == [count]


def test_reserve_no_requests(vq):
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    got = vq.vq_paged_reserve(i32([]), i32([]), i32([0, 1]), i32([2]), table, 16, 3)
    assert got[1].tolist() == [2] and got[2].tolist() == [0] and got[3].tolist() == [-1] * 3


def test_reserve_fewer_slots_than_tokens(vq):
    table = i32([[-1, -1]])
    got = vq.vq_paged_reserve(i32([0]), i32([5]), i32([7, 3]), i32([2]), table, 4, 2)
    assert got[0].tolist() == [5] and got[3].tolist() == [12, 13]
    assert table.tolist() == [[3, 7]]


def test_reserve_count_out_of_range(vq):
    """A count outside the list is taken into it."""
    for count, left in ((-4, 0), (9, 2)):
        table = i32([[-1, -1]])
        got = vq.vq_paged_reserve(i32([0]), i32([4]), i32([1, 0]), i32([count]), table, 4, 4)
        assert got[0].tolist() == ([4] if left else [0])
        assert got[1].tolist() == [max(0, left - 1)]


@pytest.mark.parametrize("case", range(6))
@pytest.mark.parametrize("in_place", [False, True])
def test_trim(vq, case, in_place):
    rng = np.random.default_rng(200 + case)
    n = [1, 3, 64, 65, 1025, 8192][case]
    page = [16, 4, 1, 32, 16, 8][case]
    width = 7
    lens = rng.integers(-1, width * page + 1, n).tolist()
    keep = [int(rng.choice([0, h, max(0, h - 3), h + 5, -2])) for h in lens]
    table, free, count = pool(rng, lens, page, width, 2)
    want = ref.trim(lens, keep, table, page, free, count)
    d_lens, d_free, d_count, d_table = i32(lens), i32(free), i32([count]), i32(table)
    kw = dict(lens_out=d_lens, free_count_out=d_count) if in_place else {}
    got = vq.vq_paged_trim(d_lens, i32(keep), d_table, page, d_free, d_count, **kw)
    assert got[0].tolist() == want[0]
    assert got[1].tolist() == [want[1]]
    assert d_free.tolist() == want[2]
    assert d_table.tolist() == table


def test_trim_full_list(vq):
    """Pages beyond the list's room are dropped, not written past it."""
    free = i32([5, 6, 7])
    got = vq.vq_paged_trim(i32([4, 4]), i32([0, 0]), i32([[0, 1], [2, 3]]), 2, free[:2], i32([1]))
    assert got[1].tolist() == [2]
    assert free.tolist() == [5, 0, 7]


def test_reserve_and_trim_give_every_page_back(vq):
    rng = np.random.default_rng(5)
    page, pages, width, n = 16, 300, 20, 17
    lens, count = i32([0] * n), i32([pages])
    free = i32(rng.permutation(pages).tolist())
    table = i32([[-1] * width] * n)
    for step in range(40):
        new = i32(rng.integers(0, 30, n).tolist())
        vq.vq_paged_reserve(lens, new, free, count, table, page, 30 * n, lens_out=lens, free_count_out=count)
        held = [t for r, h in enumerate(lens.tolist()) for t in table[r].tolist()[:ref.blocks_of(h, page)]]
        left = free.tolist()[:count.item()]
        assert sorted(held + left) == list(range(pages))
        keep = torch.where(torch.from_numpy(rng.random(n) < 0.3).cuda(), torch.zeros_like(lens), lens - 2)
        vq.vq_paged_trim(lens, keep.int(), table, page, free, count, lens_out=lens, free_count_out=count)
    vq.vq_paged_trim(lens, i32([0] * n), table, page, free, count, lens_out=lens, free_count_out=count)
    assert count.item() == pages and sorted(free.tolist()) == list(range(pages))


# ------------------------------------------------------------------ append


def values(rng, shape, dtype):
    """A CUDA tensor of `dtype`, and its values as the oracle takes them."""
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DTYPES[dtype])
    return t.cuda(), t


def oracle_codes(x, books, smooth=None):
    """The oracle's codes of x [T, H, D] against books [H, n, sub]: [T, H, ns]."""
    t, h, d = x.shape
    sub = books.shape[2]
    rows = x.transpose(0, 1).contiguous().reshape(h, -1, sub)
    if books.dtype == torch.bfloat16:  # bf16 values are fp32 values
        rows, books = rows.float(), books.float()
    rows, books = rows.numpy(), books.numpy()
    if smooth is None:
        idx = oracle.encode(rows, books, n_threads=8)
    else:
        idx = oracle.encode_smooth(rows, smooth.numpy(), books, d, n_threads=8)
    return idx.reshape(h, t, d // sub).transpose(1, 0, 2).astype(np.uint8)


APPEND = [
    # tokens, heads, dim, sub, n_c, page, dtype, smooth
    (1, 1, 8, 8, 256, 16, "f16", False),
    (1, 8, 128, 8, 256, 16, "f16", True),
    (64, 8, 128, 8, 256, 16, "bf16", False),
    (129, 3, 64, 4, 200, 32, "f16", False),
    (37, 2, 256, 4, 64, 1, "f32", True),
    (1000, 2, 128, 8, 256, 64, "f32", False),
    (333, 5, 128, 8, 256, 16, "bf16", True),
    (2049, 4, 256, 4, 256, 16, "f16", True),
    (50, 2, 96, 8, 256, 16, "f16", False),       # 12 sub-vectors a head
    (50, 2, 24, 3, 256, 8, "f16", True),         # general shapes
    (50, 2, 64, 16, 100, 4, "bf16", False),
    (33, 3, 64, 8, 63, 16, "f16", True),
    (33, 3, 64, 8, 1, 16, "f16", False),
    (20, 1, 32, 32, 17, 2, "f32", False),
]


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("layout", ["plain", "packed", "odd"])
def test_append(vq, case, layout):
    tokens, heads, dim, sub, n_c, page, dtype, smooth = case
    rng = np.random.default_rng([tokens, heads, dim, sub, n_c])
    kcb, kcb_h = values(rng, (heads, n_c, sub), dtype)
    vcb, vcb_h = values(rng, (heads, n_c, sub), dtype)
    factors = torch.from_numpy(np.exp(0.5 * rng.standard_normal((heads, dim))).astype(np.float32)) if smooth else None
    k_h = torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).to(DTYPES[dtype])
    v_h = torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).to(DTYPES[dtype])
    # exact copies of centroids, so that distances are zero and ties are met
    k_h[tokens // 2, 0, :sub] = kcb_h[0, n_c - 1]
    if layout == "plain":
        k, v = k_h.cuda(), v_h.cuda()
    else:
        # inside a packed projection; "odd": rows off the vector loads' alignment
        off = 0 if layout == "packed" else 1
        width = 3 * heads * dim + 2 * off
        packed = torch.zeros((tokens, width), dtype=DTYPES[dtype], device="cuda")
        k = packed[:, heads * dim + off:2 * heads * dim + off].unflatten(1, (heads, dim))
        v = packed[:, 2 * heads * dim + off:3 * heads * dim + off].unflatten(1, (heads, dim))
        k.copy_(k_h)
        v.copy_(v_h)
    ns = dim // sub
    pages = ref.blocks_of(tokens, page) + 2
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int64))
    slots[::7] = torch.tensor([-1, pages * page, 1 << 40, -(1 << 40)])[torch.arange(len(slots[::7])) % 4]
    pool_codes = torch.full((pages, 2, heads, page, ns), 7, dtype=torch.uint8, device="cuda")
    kc, vc = pool_codes[:, 0], pool_codes[:, 1]  # interleaved: the stride is not a page's size
    vq.vq_paged_append(k, v, slots.cuda(), kcb, vcb, kc, vc,
                       k_smooth=factors.cuda() if smooth else None)
    assert vq.vq_kernel_status() == 0
    for got, x, books, f in ((kc, k_h, kcb_h, factors), (vc, v_h, vcb_h, None)):
        want = np.full((pages, heads, page, ns), 7, np.uint8)
        codes = oracle_codes(x, books, f)
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < pages * page:
                want[slot // page, :, slot % page] = codes[t]
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_special_values(vq):
    """NaN and infinities in the rows, and a codebook of equal centroids."""
    heads, dim, sub, n_c, page, tokens = 2, 64, 8, 256, 16, 40
    rng = np.random.default_rng(9)
    kcb, kcb_h = values(rng, (heads, n_c, sub), "f16")
    kcb_h[1] = kcb_h[1, :1]
    kcb = kcb_h.cuda()
    x = torch.from_numpy(rng.standard_normal((tokens, heads, dim)).astype(np.float32)).half()
    x[3, 0, 5] = math.nan
    x[4, 1, 0] = math.inf
    x[5] = -math.inf
    x[6] = 65504.0
    kc = torch.zeros((3, heads, page, dim // sub), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    xd = x.cuda()
    vq.vq_paged_append(xd, xd, torch.arange(tokens, device="cuda"), kcb, kcb, kc, vc)
    want = oracle_codes(x, kcb_h)
    for got in (kc, vc):
        rows = got.permute(0, 2, 1, 3).reshape(-1, heads, dim // sub)[:tokens]
        assert np.array_equal(rows.cpu().numpy(), want)


def test_append_nothing(vq):
    kc = torch.zeros((1, 2, 16, 8), dtype=torch.uint8, device="cuda")
    cb = torch.zeros((2, 256, 8), dtype=torch.float16, device="cuda")
    x = torch.zeros((0, 2, 64), dtype=torch.float16, device="cuda")
    vq.vq_paged_append(x, x, torch.zeros(0, dtype=torch.int64, device="cuda"), cb, cb, kc, kc.clone())


# ------------------------------------------------------------------ attention


class Cache:
    """A pool of pages with the codes of some requests, on device and host."""

    def __init__(self, seed, lens, hq, hkv, dim, sub, n_c, page, dtype, gain=1.0, max_code=None):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.dtype = rng, page, dtype
        self.lens = list(lens)
        self.hq, self.hkv, self.dim, self.sub = hq, hkv, dim, sub
        width = max([ref.blocks_of(max(n, 0), page) for n in lens] + [1]) + 1
        table, _, _ = pool(rng, lens, page, width, 3)
        self.pages = sum(ref.blocks_of(max(n, 0), page) for n in lens) + 3
        self.table = table
        ns = dim // sub
        top = n_c if max_code is None else max_code
        self.kc = rng.integers(0, top, (self.pages, hkv, page, ns), dtype=np.uint8)
        self.vc = rng.integers(0, top, (self.pages, hkv, page, ns), dtype=np.uint8)
        self.kcb, self.kcb_h = values(rng, (hkv, n_c, sub), dtype)
        self.vcb, self.vcb_h = values(rng, (hkv, n_c, sub), dtype)
        self.gain = gain

    def queries(self, tokens):
        t = torch.from_numpy((self.gain * self.rng.standard_normal((tokens, self.hq, self.dim))).astype(np.float32))
        return t.to(DTYPES[self.dtype])

    def device(self):
        pool_codes = torch.stack([torch.from_numpy(self.kc), torch.from_numpy(self.vc)], 1).cuda()
        return i32(self.lens), i32(self.table), pool_codes[:, 0], pool_codes[:, 1]


def check_attention(vq, c, new, window=0, scale=0.0, max_new=None, pad=0, q=None, rows=None, **kw):
    """One call against the reference; returns (out, lse) on the host."""
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    tokens = cu[-1] + pad
    q_h = c.queries(tokens) if q is None else q
    lens, table, kc, vc = c.device()
    packed = torch.zeros((tokens, c.hq + 2, c.dim), dtype=q_h.dtype, device="cuda")
    packed[:, :c.hq] = q_h.cuda()
    out, lse = vq.vq_paged_attention(packed[:, :c.hq], i32(cu), lens, table, kc, vc, c.kcb, c.vcb,
                                     max_new=max(new + [0]) if max_new is None else max_new,
                                     window=window, scale=scale, return_lse=True, **kw)
    assert vq.vq_kernel_status() == 0
    eps = HALF_EPS[c.dtype]
    want, want_lse, tol, tol_lse = ref.attention(
        q_h.double().numpy(), cu, c.lens, c.table, c.kc, c.vc, c.kcb_h.double().numpy(),
        c.vcb_h.double().numpy(), window, scale, 0.0 if c.dtype == "f32" else eps, HALF_STEP[c.dtype])
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = tol + eps * (np.abs(want) + tol) + HALF_STEP[c.dtype]
    sel = slice(None) if rows is None else rows
    off = np.abs(got - want)[sel] - tol[sel]
    assert (off <= 0).all(), f"out beyond its bound by {off.max():.3g} at {np.unravel_index(off.argmax(), off.shape)}"
    fine = np.isfinite(want_lse)[sel]
    assert np.array_equal(np.isneginf(got_lse)[sel], ~fine)
    with np.errstate(invalid="ignore"):
        off = (np.where(np.isfinite(want_lse), np.abs(got_lse - want_lse), 0) - tol_lse)[sel]
    assert (off <= 0).all(), f"lse beyond its bound by {off.max():.3g}"
    assert (got[sel][~fine] == 0).all()
    return got, got_lse


SHAPES = [
    # hq, hkv, dim, sub, n_c, page, dtype
    (8, 2, 128, 8, 256, 16, "f16"),
    (8, 2, 128, 8, 256, 64, "bf16"),
    (3, 1, 256, 4, 256, 16, "f16"),
    (6, 2, 256, 8, 200, 32, "bf16"),
    (4, 4, 64, 8, 256, 16, "f16"),
    (14, 2, 64, 4, 100, 128, "bf16"),
    (8, 1, 128, 4, 256, 16, "bf16"),
    (17, 1, 128, 8, 256, 16, "f16"),
    (40, 1, 64, 8, 256, 1024, "f16"),
    # shapes of the general kernel
    (8, 2, 128, 8, 256, 16, "f32"),
    (4, 2, 128, 8, 256, 4, "f16"),
    (2, 1, 96, 8, 256, 16, "bf16"),
    (2, 1, 128, 16, 256, 16, "f16"),
    (11, 1, 30, 3, 50, 1, "f32"),
    (2, 2, 512, 8, 256, 16, "f16"),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_attention_decode(vq, shape):
    """One new token per request; lengths around units and pages, none at all,
    and one long enough to be split over many blocks."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 1300]
    c = Cache(1, lens, hq, hkv, dim, sub, n_c, page, dtype)
    check_attention(vq, c, [1] * len(lens))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 100])
def test_attention_mixed(vq, shape, window):
    """Requests with no, one, a few and many new tokens side by side, one of
    them longer than its own cache (its first rows see nothing), and padding."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    lens = [40, 0, 300, 7, 130, 129, 33, 200]
    new = [1, 0, 5, 7, 67, 0, 40, 200]
    c = Cache(2, lens, hq, hkv, dim, sub, n_c, page, dtype)
    check_attention(vq, c, new, window=window, pad=3)


@pytest.mark.parametrize("shape", SHAPES[:3] + SHAPES[9:10])
@pytest.mark.parametrize("max_new", [0, 1, 1000])
def test_attention_hint_never_changes_the_result(vq, shape, max_new):
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(3, [90, 140, 513], hq, hkv, dim, sub, n_c, page, dtype)
    check_attention(vq, c, [90, 1, 3], max_new=max_new)


@pytest.mark.parametrize("shape", SHAPES[:7] + SHAPES[9:11])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_peaked(vq, shape, new):
    """Scores of hundreds, so that the maximum moves far and weights vanish."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(4, [700, 200], hq, hkv, dim, sub, n_c, page, dtype, gain=30.0)
    check_attention(vq, c, [new, new])


@pytest.mark.parametrize("shape", SHAPES[:7] + SHAPES[9:11])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_hides_missing_pages(vq, shape, new):
    """Entries that name no page hide their tokens, wherever they are."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(5, [400, 300, 64, 140], hq, hkv, dim, sub, n_c, page, dtype)
    for b in range(len(c.table[0])):
        if b % 3 == 1:
            c.table[0][b] = [-1, c.pages, 2 ** 31 - 1, -2 ** 31][b % 4]
    c.table[2] = [-1] * len(c.table[2])  # all of them
    c.table[3][0] = c.pages + 5
    check_attention(vq, c, [new] * 4)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], SHAPES[5], SHAPES[9]])
def test_attention_lengths_beyond_the_table(vq, shape):
    """Tokens past the table's last block are not seen; negative lengths hold none."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(6, [100, 64, 30], hq, hkv, dim, sub, n_c, page, dtype)
    width = len(c.table[0])
    c.lens = [width * page + 3, 64, -5]
    for row in c.table:
        row[-1] = 0
    check_attention(vq, c, [9, 30, 4])


@pytest.mark.parametrize("shape", SHAPES[:7] + SHAPES[9:10])
@pytest.mark.parametrize("new", [1, 70])
def test_attention_codes_beyond_the_codebook(vq, shape, new):
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(7, [150, 90], hq, hkv, dim, sub, 100, page, dtype, max_code=256)
    check_attention(vq, c, [new, new])


@pytest.mark.parametrize("shape", SHAPES[:7] + SHAPES[9:10])
@pytest.mark.parametrize("new", [3, 70])
def test_attention_rows_stay_apart(vq, shape, new):
    """A row of NaN or infinities touches no other row, and becomes NaN itself."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(8, [200, 90], hq, hkv, dim, sub, n_c, page, dtype)
    q = c.queries(2 * new)
    clean = np.ones((2 * new, hq), bool)
    q[1, 0, 3] = math.nan
    q[new + 2, hq - 1, :] = math.inf
    clean[1, 0] = clean[new + 2, hq - 1] = False
    q_ref = torch.where(torch.from_numpy(clean)[:, :, None], q, torch.zeros_like(q))
    lens, table, kc, vc = c.device()
    cu = i32([0, new, 2 * new])
    args = (cu, lens, table, kc, vc, c.kcb, c.vcb)
    out, lse = vq.vq_paged_attention(q.cuda(), *args, max_new=new, return_lse=True)
    same, same_lse = vq.vq_paged_attention(q_ref.cuda(), *args, max_new=new, return_lse=True)
    mask = torch.from_numpy(clean).cuda()
    assert torch.equal(out[mask], same[mask]) and torch.equal(lse[mask], same_lse[mask])
    assert torch.isnan(out[~mask]).all() and torch.isnan(lse[~mask]).all()


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2], SHAPES[4]])
@pytest.mark.parametrize("new", [1, 18])
def test_attention_many_requests(vq, shape, new):
    """More short requests than blocks: every block takes several in a row."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(13, [new + i % 23 for i in range(450)], hq, hkv, dim, sub, n_c, page, dtype)
    check_attention(vq, c, [new] * 450)


@pytest.mark.parametrize("new", [1, 9])
def test_attention_more_requests_than_are_staged(vq, new):
    """Lengths read from memory instead of shared memory."""
    c = Cache(14, [new + i % 5 for i in range(700)], 4, 2, 64, 8, 256, 16, "bf16")
    check_attention(vq, c, [new] * 700)


@pytest.mark.parametrize("new", [1, 3])
def test_attention_more_heads_than_a_tile(vq, new):
    """160 query heads to a KV head: head groups of 8 and of 128."""
    c = Cache(16, [150, 9, 40], 160, 1, 64, 8, 256, 16, "f16")
    check_attention(vq, c, [new, 1, 0])


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2], SHAPES[9]])
def test_attention_descending_offsets_end(vq, shape):
    """Offsets that descend are a caller's mistake: the call ends, writes inside its
    outputs, and the next call is right."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(17, [300, 200, 100, 90], hq, hkv, dim, sub, n_c, page, dtype)
    lens, table, kc, vc = c.device()
    for cu in ([0, 70, 20, 90, 100], [100, 0, 0, 0, 0], [0, -5, 2000, 3, 1 << 30], [50, 60, 10, 0, 100]):
        guard = torch.full((102, hq, dim), 7.0, dtype=DTYPES[dtype], device="cuda")
        vq.vq_paged_attention(c.queries(100).cuda(), i32(cu), lens, table, kc, vc, c.kcb, c.vcb, out=guard[1:101])
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[101] == 7).all()
    assert vq.vq_kernel_status() == 0
    check_attention(vq, c, [30, 1, 60, 9])


@pytest.mark.parametrize("new", [2, 40])
def test_offsets_past_32_bits(vq, new):
    """Pages more than 2^32 bytes apart, query tokens more than 2^31 elements in
    all: the same bits as from a compact pool, and the append writes there too."""
    c = Cache(15, [300, 77], 4, 2, 128, 8, 256, 16, "f16")
    lens, table, kc, vc = c.device()
    stride = (5 << 30) // c.pages // 16 * 16
    far = [torch.empty(stride * c.pages, dtype=torch.uint8, device="cuda").as_strided(kc.shape, (stride, 256, 16, 1))
           for _ in range(2)]
    assert stride * (c.pages - 1) > 1 << 32
    for a, b in zip(far, (kc, vc)):
        a.copy_(b)
    cu = i32([0, new, 2 * new])
    q = c.queries(2 * new).cuda()
    step = (1 << 31) // (2 * new - 1) + 8
    step -= step % 8
    wide = torch.empty(step * (2 * new - 1) + 4 * 128, dtype=torch.float16, device="cuda").as_strided(q.shape, (step, 128, 1))
    wide.copy_(q)
    want = vq.vq_paged_attention(q, cu, lens, table, kc, vc, c.kcb, c.vcb, max_new=new)
    got = vq.vq_paged_attention(wide, cu, lens, table, *far, c.kcb, c.vcb, max_new=new)
    assert torch.equal(want, got)
    k = wide[:, :2]
    slots = torch.arange(2 * new, device="cuda") + (c.pages * 16 - 2 * new)
    near = [kc.contiguous(), vc.contiguous()]
    vq.vq_paged_append(q[:, :2], q[:, 2:], slots, c.kcb, c.vcb, *near)
    vq.vq_paged_append(k, wide[:, 2:], slots, c.kcb, c.vcb, *far)
    assert all(torch.equal(a, b) for a, b in zip(near, far))


def test_attention_scale_and_repeat(vq):
    """An explicit scale; two calls give the same bits; a dirty workspace does not matter."""
    c = Cache(10, [3000, 20, 700], 8, 2, 128, 8, 256, 16, "bf16")
    check_attention(vq, c, [1, 2, 60], scale=0.3)
    lens, table, kc, vc = c.device()
    q = c.queries(63).cuda()
    ws = torch.full((vq.vq_paged_attention_workspace_bytes(3, 63, 60, 8, 2, 128, 8, 256, 16),), 255,
                    dtype=torch.uint8, device="cuda")
    a = vq.vq_paged_attention(q, i32([0, 1, 3, 63]), lens, table, kc, vc, c.kcb, c.vcb, max_new=60, workspace=ws)
    b = vq.vq_paged_attention(q, i32([0, 1, 3, 63]), lens, table, kc, vc, c.kcb, c.vcb, max_new=60)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_attention_no_pages(vq):
    """A pool without pages, and requests without blocks: zeros."""
    cb = torch.ones((2, 256, 8), dtype=torch.float16, device="cuda")
    codes = torch.zeros((0, 2, 16, 16), dtype=torch.uint8, device="cuda")
    q = torch.ones((3, 4, 128), dtype=torch.float16, device="cuda")
    for requests in (0, 2):
        table = torch.zeros((requests, 0), dtype=torch.int32, device="cuda")
        out, lse = vq.vq_paged_attention(q, i32([0, 1, 2][:requests + 1]), i32([0, 9][:requests]), table, codes,
                                         codes, cb, cb, return_lse=True)
        assert (out == 0).all() and torch.isneginf(lse).all()


def test_attention_misaligned_pages_and_rows(vq):
    """Pages and query rows off the vector loads' alignment."""
    c = Cache(11, [300, 45], 4, 2, 128, 8, 256, 16, "f16")
    lens, table, _, _ = c.device()
    inner = 2 * 16 * 16
    raw = torch.zeros((2, c.pages * (inner + 3) + 1), dtype=torch.uint8, device="cuda")
    views = [raw[i, 1:].as_strided((c.pages, 2, 16, 16), (inner + 3, 256, 16, 1)) for i in range(2)]
    views[0].copy_(torch.from_numpy(c.kc))
    views[1].copy_(torch.from_numpy(c.vc))
    for new in ([1, 1], [80, 45]):
        cu = [0, new[0], sum(new)]
        q_h = c.queries(sum(new))
        wide = torch.zeros((sum(new), 4 * 128 + 3), dtype=torch.float16, device="cuda")
        q = wide[:, 1:513].unflatten(1, (4, 128))
        q.copy_(q_h)
        out = vq.vq_paged_attention(q, i32(cu), lens, table, *views, c.kcb, c.vcb, max_new=max(new))
        want, _, tol, _ = ref.attention(q_h.double().numpy(), cu, c.lens, c.table, c.kc, c.vc, c.kcb_h.double().numpy(),
                                        c.vcb_h.double().numpy(), weight_eps=2.0 ** -11, weight_abs=2.0 ** -25)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25).all()


def test_attention_matches_the_dense_decode(vq):
    """Equal lengths, one token each: the result of vq_attention_decode on the
    same codes, both within their rounding of the same sums."""
    b, hq, hkv, t, dim = 3, 8, 2, 640, 128
    c = Cache(12, [t] * b, hq, hkv, dim, 8, 256, 16, "f16")
    lens, table, kc, vc = c.device()
    q = c.queries(b).cuda()
    dense = []
    for codes in (kc, vc):
        dense.append(torch.stack([codes[table[r, :t // 16].long()].transpose(0, 1).reshape(hkv, t, -1) for r in range(b)]))
    want = vq.vq_attention_decode(q, dense[0].contiguous(), c.kcb, dense[1].contiguous(), c.vcb)
    got = vq.vq_paged_attention(q, i32([0, 1, 2, 3]), lens, table, kc, vc, c.kcb, c.vcb, max_new=1)
    _, _, tol, _ = ref.attention(q.double().cpu().numpy(), [0, 1, 2, 3], c.lens, c.table, c.kc, c.vc,
                                 c.kcb_h.double().numpy(), c.vcb_h.double().numpy(), weight_eps=2.0 ** -11,
                                 weight_abs=2.0 ** -25)
    w = want.double().cpu().numpy()
    assert (np.abs(got.double().cpu().numpy() - w) <= 2 * tol + 2.0 ** -10 * (np.abs(w) + tol)).all()


# ------------------------------------------------------------------ the step


def step(vq, s, stream=None):
    """One serving step over the state `s`, in place."""
    kw = {} if stream is None else {"stream": stream}
    vq.vq_paged_reserve(s["lens"], s["new"], s["free"], s["count"], s["table"], 16, s["k"].shape[0],
                        lens_out=s["lens"], free_count_out=s["count"], cu_new=s["cu"], slots=s["slots"], **kw)
    vq.vq_paged_append(s["k"], s["v"], s["slots"], s["kcb"], s["vcb"], s["kc"], s["vc"], **kw)
    vq.vq_paged_attention(s["q"], s["cu"], s["lens"], s["table"], s["kc"], s["vc"], s["kcb"], s["vcb"],
                          out=s["out"], lse=s["lse"], workspace=s["ws"], max_new=s["max_new"], **kw)


def state(vq, max_new):
    gen = torch.Generator(device="cuda").manual_seed(1)
    r, pages, rows, hq, hkv, dim = 5, 200, 40, 8, 2, 128
    kcb, vcb = (torch.randn((hkv, 256, 8), generator=gen, device="cuda").half() for _ in range(2))
    return {"lens": i32([0] * r), "new": i32([0] * r), "free": i32(list(range(pages))), "count": i32([pages]),
            "table": i32([[-1] * 30] * r), "cu": i32([0] * (r + 1)),
            "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"),
            "k": torch.zeros((rows, hkv, dim), dtype=torch.float16, device="cuda"),
            "v": torch.zeros((rows, hkv, dim), dtype=torch.float16, device="cuda"),
            "q": torch.zeros((rows, hq, dim), dtype=torch.float16, device="cuda"),
            "kcb": kcb, "vcb": vcb, "kc": torch.zeros((pages, hkv, 16, 16), dtype=torch.uint8, device="cuda"),
            "vc": torch.zeros((pages, hkv, 16, 16), dtype=torch.uint8, device="cuda"),
            "out": torch.zeros((rows, hq, dim), dtype=torch.float16, device="cuda"),
            "lse": torch.zeros((rows, hq), device="cuda"), "max_new": max_new,
            "ws": torch.empty(vq.vq_paged_attention_workspace_bytes(r, rows, max_new, hq, hkv, dim, 8, 256, 16),
                              dtype=torch.uint8, device="cuda")}


def test_step_in_a_graph_equals_the_eager_step(vq):
    """Steps of changing lengths replayed from one captured graph, against the
    same steps made eagerly on a side stream: the same bits."""
    rng = np.random.default_rng(3)
    a, b = state(vq, 0), state(vq, 0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(vq, b, side)  # first use outside the capture; no new tokens
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(vq, b)
    for n in range(6):
        new = rng.integers(0, 9, 5).tolist() if n else [30, 0, 1, 9, 0]
        gen = torch.Generator(device="cuda").manual_seed(n)
        for s in (a, b):
            s["new"].copy_(i32(new))
        for name in ("k", "v", "q"):
            x = torch.randn(a[name].shape, generator=gen, device="cuda").half()
            a[name].copy_(x)
            b[name].copy_(x)
        torch.cuda.synchronize()
        step(vq, a, side)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("lens", "count", "table", "cu", "slots", "kc", "vc", "out", "lse"):
            assert torch.equal(a[name], b[name]), name
        assert (a["out"][sum(new):] == 0).all()
    assert a["lens"].sum().item() > 50


def test_step_on_another_stream_than_the_tensors(vq):
    """Tensors made on the default stream, the step on a side stream that waits
    for it: the state of the same step on the default stream."""
    a, b = state(vq, 9), state(vq, 9)
    gen = torch.Generator(device="cuda").manual_seed(7)
    for s in (a, b):
        s["new"].copy_(i32([9, 3, 1, 0, 7]))
    for name in ("k", "v", "q"):
        x = torch.randn(a[name].shape, generator=gen, device="cuda").half()
        a[name].copy_(x)
        b[name].copy_(x)
    step(vq, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(vq, b, side)
    torch.cuda.current_stream().wait_stream(side)
    for name in ("lens", "count", "table", "cu", "slots", "kc", "vc", "out", "lse"):
        assert torch.equal(a[name], b[name]), name


def test_example_serving_loop(vq):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")
    spec = importlib.util.spec_from_file_location("paged_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    report = module.main(["--steps", "30", "--requests", "5", "--prompt", "300", "--answer", "30"])
    assert report["finished"] > 3 and report["tokens"] > 500
