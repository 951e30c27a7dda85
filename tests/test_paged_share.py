"""Shared pages on the GPU: fork, compact and copy against plain host forms, exactly;
and a run of them between appends and attention of the code cache."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import share_reference as share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def table_of(a, width):
    return i32(a).reshape(len(a), width)


def check_fork(vq, lens, parents, keep, table, page, free, count, in_place=False, **kw):
    width = len(table[0]) if table else 0
    want = share.fork(lens, parents, keep, table, page, free, count)
    d_lens, d_free, d_count = i32(lens), i32(free), i32([count])
    if in_place:
        kw.update(lens_out=d_lens, free_count_out=d_count)
    d_table = table_of(table, width)
    got = vq.vq_paged_fork(d_lens, i32(parents), d_table, page, d_free, d_count,
                           keep_lens=None if keep is None else i32(keep), **kw)
    assert got[0].tolist() == want[0]
    assert got[1].tolist() == want[1]
    assert got[2].tolist() == [want[2]]
    assert got[3].tolist() == want[3]
    assert d_free.tolist() == want[4]
    assert d_table.tolist() == table
    return want


FORKS = [
    # lens, parents, keep, table, page, free list, count
    ([5], [0], None, [[3, 1]], 4, [0, 2, -1, -1], 2),                      # stays as it is
    ([5, 0], [0, 0], None, [[3, 1], [-1, -1]], 4, [0, 2, -1, -1], 2),      # a fork: whole page shared, the part copied
    ([8, 0], [0, 0], None, [[3, 1], [-1, -1]], 4, [0, 2, -1, -1], 2),      # whole pages alone: no copy
    ([5, 3], [1, 0], None, [[3, 1], [0, -1]], 4, [2, -1, -1, -1], 1),      # seats change places
    ([5, 3], [-1, 7], None, [[3, 1], [0, -1]], 4, [2, -1, -1, -1], 1),     # both are emptied
    ([8, 8], [0, 0], [8, 6], [[3, 1], [0, 2]], 4, [-1] * 4, 0),            # cut inside a page that another holds whole
    ([6, 0, 0], [0, 0, 0], [6, 5, 3], [[3, 1], [-1, -1], [-1, -1]], 4, [0, 2, -1, -1], 2),
    ([6, 0, 0, 0], [0, 0, 0, 0], None, [[3, 1]] + [[-1, -1]] * 3, 4, [0, 2, -1, -1], 1),  # pages for one copy of three
    ([6, 0], [0, 0], [0, 0], [[3, 1], [-1, -1]], 4, [0, 2, -1, -1], 2),    # cut to nothing
    ([6, -4], [0, 1], [-3, 9], [[3, 1], [0, 2]], 4, [-1] * 4, 0),          # negative counts are none
    ([100, 2], [0, 0], None, [[3, 1], [0, 2]], 4, [-1] * 4, 0),            # a length past the table
    ([7, 0], [0, 0], None, [[3, 9], [-1, -1]], 4, [0, 2, -1, -1], 2),      # an entry that is no page
    ([7, 0], [0, 0], None, [[-1, 1], [-1, -1]], 4, [0, 2, -1, -1], 2),
    ([7, 0], [0, 0], None, [[3, 1], [-1, -1]], 4, [0, 2, -1, -1], 9),      # counts outside the list
    ([7, 0], [0, 0], None, [[3, 1], [-1, -1]], 4, [0, 2, -1, -1], -2),
    ([3, 2], [0, 1], None, [[0, 1, 2], [2, 1, 0]], 1, [-1] * 3, 0),        # a page a token, held twice
    ([3, 3], [1, 1], None, [[0, 0], [0, 0]], 2, [1], 0),                   # one page in every place
]


@pytest.mark.parametrize("case", range(len(FORKS)))
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(vq, case, in_place):
    check_fork(vq, *FORKS[case], in_place=in_place)


def random_pool(rng, seats, width, page, spare, shared):
    """Seats over a pool: a share of the rows begin with another's whole pages."""
    lens = rng.integers(0, width * page + 1, seats)
    table = np.full((seats, width), -1, np.int64)
    pages = int(seats * width + spare)
    order = rng.permutation(pages)
    at = 0
    for r in range(seats):
        n = share.blocks_of(int(lens[r]), page)
        first = 0
        if r and rng.random() < shared:
            other = int(rng.integers(r))
            first = min(int(lens[other]) // page, n)
            table[r, :first] = table[other, :first]
        table[r, first:n] = order[at:at + n - first]
        at += n - first
    free = np.full(pages, -1)
    free[:pages - at] = order[at:]
    return lens.tolist(), table.tolist(), free.tolist(), pages - at


# the second past one block of the cluster's pages, the third past a segment of a row,
# the last past a block's threads
@pytest.mark.parametrize("seats, width, page, spare", [(7, 5, 4, 3), (150, 130, 16, 900), (30, 300, 1, 0), (1500, 3, 8, 2),
                                                       (8192, 1, 64, 0), (4, 40000, 2, 5)])
@pytest.mark.parametrize("seed", range(2))
def test_fork_random(vq, seats, width, page, spare, seed):
    rng = np.random.default_rng([seats, seed])
    lens, table, free, count = random_pool(rng, seats, width, page, spare, 0.7)
    parents = rng.integers(-1, seats, seats)
    some = rng.random(seats) < 0.5
    parents[some] = np.arange(seats)[some]
    keep = (rng.integers(0, width * page + 2, seats)).tolist() if seed else None
    after = check_fork(vq, lens, parents.tolist(), keep, table, page, free, count, in_place=seed == 1)
    # and again on what came out
    check_fork(vq, after[0], rng.integers(-1, seats, seats).tolist(), None, after[1], page, after[4], after[2])


def test_fork_nothing(vq):
    got = vq.vq_paged_fork(i32([]), i32([]), torch.empty((0, 3), dtype=torch.int32, device="cuda"), 16, i32([0, 1]), i32([2]))
    assert got[2].tolist() == [2] and got[3].shape == (0, 2)
    got = vq.vq_paged_fork(i32([0, 0]), i32([1, 1]), torch.empty((2, 0), dtype=torch.int32, device="cuda"), 16, i32([0]), i32([1]))
    assert got[0].tolist() == [0, 0] and got[2].tolist() == [1]
    got = vq.vq_paged_fork(i32([5]), i32([0]), i32([[-1]]), 16, i32([]), i32([0]))
    assert got[0].tolist() == [5] and got[1].tolist() == [[-1]] and got[3].tolist() == [[-1, -1]]


def test_fork_refuses_its_own_table(vq):
    table = i32([[0, 1], [-1, -1]])
    with pytest.raises(vq.VQError):
        vq.vq_paged_fork(i32([5, 0]), i32([0, 0]), table, 4, i32([2, 3, -1, -1]), i32([2]), table_out=table)
    with pytest.raises(vq.VQError):
        vq.vq_paged_fork(i32([5]), i32([0]), i32([[0, 1]]), 4, i32([2, 3, -1, -1]), i32([2]),
                         workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ compact


def check_compact(vq, lens, table, page, free, count, in_place=False):
    want = share.compact(lens, table, page, free, count)
    d_table, d_free, d_count = table_of(table, len(table[0]) if table else 0), i32(free), i32([count])
    kw = dict(table_out=d_table, free_pages_out=d_free, free_count_out=d_count) if in_place else {}
    got = vq.vq_paged_compact(i32(lens), d_table, page, d_free, d_count, **kw)
    assert got[0].tolist() == want[0]
    assert got[1].tolist() == want[1]
    assert got[2].tolist() == [want[2]]
    assert got[3].tolist() == want[3]
    assert got[4].tolist() == want[4]
    return want


COMPACTS = [
    # lens, table, page, free list, count
    ([5], [[3, 1]], 4, [0, 2, -1, -1], 2),
    ([5], [[0, 1]], 4, [3, 2, -1, -1], 2),                 # nothing to move
    ([0], [[7, 7]], 4, [1, 0, 2, 3], 4),                   # every page is free
    ([8, 8], [[3, 1], [0, 2]], 4, [-1] * 4, 0),            # none is
    ([9, 8], [[3, 1, -1], [3, 4, 2]], 4, [0, -1, -1, -1, -1], 1),  # a shared page; entries past the length stay
    ([5], [[3, 9]], 4, [0, 2, 5, 2, -4, 0], 6),            # a list with repeats and numbers that are no page
    ([5], [[3, 1]], 4, [0, 2, -1, -1], 77),                # counts outside the list
    ([5], [[3, 1]], 4, [0, 2, -1, -1], -1),
    ([5], [[0, -1]], 4, [0], 1),                           # a page that is on the list and in the table
]


@pytest.mark.parametrize("case", range(len(COMPACTS)))
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(vq, case, in_place):
    check_compact(vq, *COMPACTS[case], in_place=in_place)


@pytest.mark.parametrize("seats, width, page, spare", [(7, 5, 4, 3), (64, 64, 16, 1), (64, 64, 16, 0), (100, 130, 16, 4000),
                                                       (3, 40000, 2, 123457)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_random(vq, seats, width, page, spare, in_place):
    rng = np.random.default_rng(seats + spare)
    lens, table, free, count = random_pool(rng, seats, width, page, spare, 0.3)
    after = check_compact(vq, lens, table, page, free, count, in_place)
    check_compact(vq, lens, after[0], page, after[1], after[2])  # a second time nothing moves


def test_compact_nothing(vq):
    got = vq.vq_paged_compact(i32([]), torch.empty((0, 2), dtype=torch.int32, device="cuda"), 16, i32([1, 0, -1]), i32([2]))
    assert got[1].tolist() == [2, 1, -1] and got[3].tolist() == [[2, 0]] and got[4].tolist() == [-1, -1, 0]
    got = vq.vq_paged_compact(i32([0]), i32([[4]]), 16, i32([]), i32([0]))
    assert got[0].tolist() == [[4]] and got[2].tolist() == [0]


# ------------------------------------------------------------------ copy


@pytest.mark.parametrize("inner, dtype", [((2, 8, 16, 64), torch.uint8), ((3, 16), torch.bfloat16), ((5,), torch.uint8),
                                          ((7, 3), torch.float32), ((4097,), torch.uint8), ((1,), torch.int64), ((9000,), torch.int16)])
@pytest.mark.parametrize("layers", [0, 1, 3])
@pytest.mark.parametrize("rows", [1, 40, 5000])
def test_copy(vq, inner, dtype, layers, rows):
    if rows * int(np.prod(inner)) > 60_000_000:
        rows = 700
    rng = np.random.default_rng(rows)
    pages = 2 * rows + 4
    gen = torch.Generator(device="cuda").manual_seed(rows)
    shape = (pages, *inner) if layers == 0 else (layers, pages, *inner)
    size = torch.empty(0, dtype=dtype).element_size()
    pool = torch.randint(0, 256, (*shape[:-1], shape[-1] * size), generator=gen, device="cuda", dtype=torch.uint8).view(dtype)
    order = rng.permutation(pages)
    pairs = np.stack([order[:rows], order[rows:2 * rows]], 1)
    pairs[::3] = -1
    pairs[1::7, 0] = pages          # no page
    pairs[2::11, 1] = -5
    pairs[4::13, 1] = pairs[4::13, 0]
    want = pool.clone()
    valid = (pairs >= 0).all(1) & (pairs < pages).all(1)
    src, dst = (torch.from_numpy(pairs[valid, i]).cuda() for i in (0, 1))
    at = (slice(None), dst) if layers else (dst,)
    want[at] = pool[(slice(None), src) if layers else (src,)]
    vq.vq_paged_copy(i32(pairs.tolist()).reshape(-1, 2), [pool], layered=layers > 0)
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))


def test_copy_pools_and_strides(vq):
    """Several pools at once; pages inside wider ones, off any alignment; layers inside a page."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randint(0, 256, (50, 4, 333), generator=gen, device="cuda", dtype=torch.uint8)
    flat = torch.randint(0, 256, (1 + 50 * 100,), generator=gen, device="cuda", dtype=torch.uint8)
    pools = [base[:, 1], flat[1:].view(50, 100)[:, :77], torch.randn(50, 3, 8, generator=gen, device="cuda"),
             torch.randn(50, 6, generator=gen, device="cuda").half()]
    pairs = [[3, 4], [-1, -1], [49, 0], [7, 48]]
    kept = [base.clone(), flat.clone()]
    want = [p.clone() for p in pools]
    for w in want:
        for a, b in pairs:
            if a >= 0:
                w[b] = w[a]
    vq.vq_paged_copy(i32(pairs), pools)
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    for now, was in zip((base, flat), kept):  # nothing beside the pages
        pools[0].zero_(), pools[1].zero_()
        was[:, 1].zero_() if was.dim() == 3 else was[1:].view(50, 100)[:, :77].zero_()
        assert torch.equal(now, was)
    inside = torch.randn(20, 5, 16, generator=gen, device="cuda")  # [page][layer][..]
    want = inside.clone()
    want[6] = want[2]
    vq.vq_paged_copy(i32([[2, 6]]), [inside.transpose(0, 1)], layered=True)
    assert torch.equal(inside, want)
    vq.vq_paged_copy(torch.empty((0, 2), dtype=torch.int32, device="cuda"), [inside])
    vq.vq_paged_copy(i32([[0, 1]]), [torch.empty((3, 0), device="cuda")])


def test_copy_refusals(vq):
    pool = torch.zeros((4, 8), device="cuda")
    pairs = i32([[0, 1]])
    with pytest.raises(TypeError):
        vq.vq_paged_copy(pairs, pool)
    with pytest.raises(ValueError, match="1 to 8"):
        vq.vq_paged_copy(pairs, [])
    with pytest.raises(ValueError, match="one number of pages"):
        vq.vq_paged_copy(pairs, [pool, pool[:3]])
    with pytest.raises(ValueError, match="contiguous"):
        vq.vq_paged_copy(pairs, [torch.zeros((4, 8, 8), device="cuda").transpose(1, 2)])
    with pytest.raises(vq.VQError):
        vq.vq_paged_copy(pairs, [torch.zeros(8, device="cuda").expand(4, 8)])
    with pytest.raises(ValueError, match="layers"):
        vq.vq_paged_copy(pairs, [torch.zeros(4, device="cuda")], layered=True)


def test_copy_past_32_bits(vq):
    """Pages beyond 2^32 bytes of a pool."""
    pages = 70000
    pool = torch.empty((pages, 65536 + 16), dtype=torch.uint8, device="cuda")
    pool[pages - 1] = torch.arange(65552, device="cuda").to(torch.uint8)
    pool[pages - 3] = 0
    vq.vq_paged_copy(i32([[pages - 1, pages - 3]]), [pool])
    assert torch.equal(pool[pages - 3], pool[pages - 1])


# ------------------------------------------------------------------ together


def test_step_captured(vq):
    """Fork, copy, reserve and append of a beam step captured as one graph, replayed with
    other parents: every seat attends to what its own line of parents has written."""
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(3)
    seats, heads, dim, sub, page, width = 6, 2, 64, 8, 4, 9
    ns, pages = dim // sub, 60
    books = [torch.randn((heads, 256, sub), generator=gen, device="cuda").half() for _ in range(2)]
    pool = torch.zeros((pages, 2, heads, page, ns), dtype=torch.uint8, device="cuda")
    kc, vc = pool[:, 0], pool[:, 1]
    lens, count = i32([0] * seats), i32([pages])
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    table = torch.full((seats, width), -1, dtype=torch.int32, device="cuda")
    parents, new = i32(list(range(seats))), i32([1] * seats)
    x = torch.zeros((seats, 3 * heads, dim), dtype=torch.float16, device="cuda")
    other = torch.empty_like(table)

    def step():
        _, _, _, copies = vq.vq_paged_fork(lens, parents, table, page, free, count, lens_out=lens, table_out=other,
                                           free_count_out=count)
        table.copy_(other)
        vq.vq_paged_copy(copies, [pool])
        _, _, cu, slots = vq.vq_paged_reserve(lens, new, free, count, table, page, seats, lens_out=lens, free_count_out=count)
        vq.vq_paged_append(x[:, heads:2 * heads], x[:, 2 * heads:], slots, *books, kc, vc)
        return vq.vq_paged_attention(x[:, :heads], cu, lens, table, kc, vc, *books, max_new=1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        saved = [t.clone() for t in (lens, count, free, table, pool)]
        step()
        for t, s in zip((lens, count, free, table, pool), saved):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    lines = [[] for _ in range(seats)]  # what each seat has seen: rows of keys and values
    for n in range(30):
        p = list(range(seats)) if n % 3 == 0 else rng.integers(0, seats, seats).tolist()
        if n % 11 == 10:
            p[2] = -1
        parents.copy_(i32(p))
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda").half())
        graph.replay()
        rows = x[:, heads:].cpu()
        lines = [(list(lines[a]) if a >= 0 else []) + [rows[d]] for d, a in enumerate(p)]
        assert lens.tolist() == [len(a) for a in lines]
        held = {e for a, row in zip(lines, table.tolist()) for e in row[:share.blocks_of(len(a), page)]}
        idle = free.tolist()[:count.item()]
        assert sorted(held | set(idle)) == list(range(pages)) and not held & set(idle) and len(idle) == len(set(idle))
        for d, line in enumerate(lines):
            seen = torch.stack(line)  # [tokens, 2 heads, dim]
            keys, values = (seen[:, i * heads:(i + 1) * heads].transpose(0, 1).reshape(heads, -1, sub).contiguous().cuda() for i in (0, 1))
            k = vq.vq_dequantize_grouped(vq.vq_encode_grouped_u8(keys, books[0]), books[0]).reshape(heads, -1, dim).double()
            v = vq.vq_dequantize_grouped(vq.vq_encode_grouped_u8(values, books[1]), books[1]).reshape(heads, -1, dim).double()
            w = torch.softmax((k * x[d, :heads, None].double()).sum(-1) / dim ** 0.5, -1)
            want = (w[..., None] * v).sum(1)
            # values below 8, fp16 output: a wrong page would be off by about 1
            assert (out[d].double() - want).abs().max() < 0.02
        if max(len(a) for a in lines) >= width * page - 1:
            lines = [[] for _ in range(seats)]
            lens.zero_()
            count.fill_(pages)
            free.copy_(torch.arange(pages, dtype=torch.int32, device="cuda"))


def test_compact_keeps_what_is_held(vq):
    """Compaction and its moves, then attention: the same bits as before."""
    rng = np.random.default_rng(9)
    gen = torch.Generator(device="cuda").manual_seed(9)
    lens, table, free, count = random_pool(rng, 9, 12, 16, 70, 0.4)
    pages = len(free)
    pool = torch.randint(0, 256, (pages, 2, 2, 16, 16), generator=gen, device="cuda", dtype=torch.uint8)
    books = [torch.randn((2, 256, 8), generator=gen, device="cuda").half() for _ in range(2)]
    q = torch.randn((9, 4, 128), generator=gen, device="cuda").half()
    cu, d_lens, d_table = i32(range(10)), i32(lens), i32(table)

    def attend(t):
        return vq.vq_paged_attention(q, cu, d_lens, t, pool[:, 0], pool[:, 1], *books, max_new=1, return_lse=True)

    want = attend(d_table)
    new, left, idle, moves, _ = vq.vq_paged_compact(d_lens, d_table, 16, i32(free), i32([count]))
    vq.vq_paged_copy(moves, [pool])
    got = attend(new)
    used = pages - idle.item()
    assert int(new.max()) < used and left.tolist()[:pages - used] == list(range(pages - 1, used - 1, -1))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))


def test_on_another_stream(vq):
    """Work on a stream that is not the current one, outputs made on it."""
    rng = np.random.default_rng(4)
    lens, table, free, count = random_pool(rng, 40, 20, 8, 100, 0.5)
    parents = rng.integers(0, 40, 40).tolist()
    want = share.fork(lens, parents, None, table, 8, free, count)
    side = torch.cuda.Stream()
    args = i32(lens), i32(parents), i32(table)
    d_free, d_count = i32(free), i32([count])
    side.wait_stream(torch.cuda.current_stream())
    got = vq.vq_paged_fork(*args, 8, d_free, d_count, stream=side)
    back = vq.vq_paged_compact(got[0], got[1], 8, d_free, got[2], stream=side)
    side.synchronize()
    assert [got[0].tolist(), got[1].tolist(), got[2].tolist(), got[3].tolist()] == [want[0], want[1], [want[2]], want[3]]
    again = share.compact(want[0], want[1], 8, want[4], want[2])
    assert [t.tolist() for t in back] == [again[0], again[1], [again[2]], again[3], again[4]]
