"""Long caches: every block of the chunk kernel works through tens of key blocks in a row,
so that its steady loop (accumulating, the one-pass weights with the maximum so far,
rescaling, the ring of stages and masks going round) carries the result, and every warp of
the few-row kernel through tens of groups."""
import math

import pytest
import torch

from test_checked_build import both, libs  # noqa: F401  (a fixture)
from test_paged import DTYPES, HALF_EPS, HALF_STEP, i32

pytestmark = pytest.mark.gpu

KEYS = {64: 128, 128: 128, 256: 64}  # of a key block


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


def make(seed, dim, sub, dtype, hq, hkv, page, lens, news, gain=1.0, late=False, holes=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ns, n_c = dim // sub, 256
    width = -(-max(lens) // page) + 1
    pages = sum(-(-n // page) for n in lens) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.randint(0, n_c, (pages, hkv, page, ns), generator=gen, device="cuda", dtype=torch.uint8)
              for _ in range(2))
    kcb, vcb = (torch.randn((hkv, n_c, sub), generator=gen, device="cuda") for _ in range(2))
    at = 0
    for r, n in enumerate(lens):
        held = -(-n // page)
        table[r, :held] = order[at:at + held]
        at += held
        if late:  # keys grow along the sequence: the maxima come late, step by step
            top = 16 + 240 * torch.arange(held * page, device="cuda") // (held * page)
            draw = torch.rand((held, page, hkv, ns), generator=gen, device="cuda")
            kc[table[r, :held].long()] = (top.reshape(held, page, 1, 1) * draw).to(torch.uint8).transpose(1, 2)
        if holes:
            table[r, held // 3] = -1
            table[r, held // 2:held // 2 + 5] = pages + 9
    if late:
        kcb *= torch.linspace(0.05, 2.0, n_c, device="cuda")[None, :, None]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = (gain * torch.randn((cu[-1], hq, dim), generator=gen, device="cuda")).to(DTYPES[dtype])
    return dict(q=q, cu=cu, lens=lens, table=table, kc=kc, vc=vc, kcb=kcb.to(DTYPES[dtype]), vcb=vcb.to(DTYPES[dtype]),
                dtype=dtype)


def run(vq, c, window=0):
    return vq.vq_paged_attention(c["q"], i32(c["cu"]), i32(c["lens"]), c["table"], c["kc"], c["vc"], c["kcb"], c["vcb"],
                                 max_new=max(b - a for a, b in zip(c["cu"], c["cu"][1:])), window=window, return_lse=True)


def check(c, out, lse, window=0, pieces=1):
    """Against the definition in 64 bits, with the bounds that paged_reference derives
    (e: relative error of a weight, d: error of a score), one request and head at a time.
    Weights in two pieces are off by half a step of the type twice over, and in fp16,
    where the maximum's weight is 2^7 or more, by 2^-32 of it."""
    u, eps, tiny = 2.0 ** -24, HALF_EPS[c["dtype"]], HALF_STEP[c["dtype"]]
    weight_eps = eps ** pieces
    weight_abs = 2.0 ** -32 if pieces == 2 and c["dtype"] == "f16" else tiny
    tokens, hq, dim = c["q"].shape
    pages, hkv, page, ns = c["kc"].shape
    scale = 1 / math.sqrt(dim)
    kappa = scale / math.log(2)
    for r, length in enumerate(c["lens"]):
        a, b = c["cu"][r], c["cu"][r + 1]
        t = torch.arange(length, device="cuda")
        entry = c["table"][r].long()[t // page]
        ok = (entry >= 0) & (entry < pages)
        entry = entry.clamp(0, pages - 1)
        pos = length - (b - a) + torch.arange(b - a, device="cuda")
        seen = ok[None, :] & (t[None, :] <= pos[:, None])
        if window:
            seen &= t[None, :] > pos[:, None] - window
        some = seen.any(1)
        assert (out[a:b][~some] == 0).all() and torch.isneginf(lse[a:b][~some]).all()
        if not some.any():
            continue
        n = seen.sum(1, keepdim=True).double()
        for h in range(hkv):
            keys, values = (book[h].double()[codes[entry, h, t % page].long()].reshape(length, dim)
                            for book, codes in ((c["kcb"], c["kc"]), (c["vcb"], c["vc"])))
            for g in range(hq // hkv):
                head = h * (hq // hkv) + g
                rows = c["q"][a:b, head].double()
                s = (scale * (rows @ keys.t())).masked_fill(~seen, -math.inf)
                top = s.amax(1, keepdim=True)
                w = torch.exp(s - top)
                total = w.sum(1, keepdim=True)
                want = w @ values / total
                want_lse = (top + torch.log(total))[:, 0]
                d = (dim + 4) * u * kappa * (rows.abs() @ keys.abs().t())
                e = math.log(2) * (d + 2 * u * ((top - s) / math.log(2) + 8)) + 2.0 ** -21 + weight_eps
                e = e.masked_fill(~seen, 0)
                big = values[seen.any(0)].abs().max()
                tol = 1.1 * big * (2 * (w * e).sum(1, keepdim=True) / total + 2 * n * weight_abs + 4 * (n + 200) * u)
                tol_lse = 1.1 * (e.amax(1) + n[:, 0] * weight_abs + (n[:, 0] + 200) * u) + 4 * u * want_lse.abs()
                off = (out[a:b, head].double() - want).abs() - (tol + eps * (want.abs() + tol) + tiny)
                assert (off[some] <= 0).all(), f"request {r} head {head}: beyond the bound by {off[some].max():.3g}"
                assert ((lse[a:b, head].double() - want_lse).abs() <= tol_lse)[some].all()


CASES = [  # dim, sub, dtype, hq, hkv, page, lens, news
    (128, 8, "bf16", 32, 8, 16, [5000], [771]),
    (128, 4, "f16", 16, 4, 64, [6000, 4100], [811, 600]),
    (64, 8, "f16", 32, 8, 16, [5000], [907]),
    (64, 4, "bf16", 24, 8, 128, [4000, 5100], [300, 555]),
    (256, 4, "f16", 12, 4, 16, [5000], [1000]),
    (256, 8, "bf16", 16, 4, 32, [4000, 3333], [601, 450]),
]


def key_blocks(case, sms):
    """Key blocks in a row of the average block of the launch."""
    dim, sub, dtype, hq, hkv, page, lens, news = case
    tile = (2 if dim < 256 else 1) * (128 * hkv // hq)
    units = sum(-(-n // tile) * hkv * -(-(length - n // 2) // 128) for length, n in zip(lens, news))
    return units * 128 // KEYS[dim] / sms


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("kind", ["plain", "window", "late", "holes"])
def test_long_chunks(vq, case, kind):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert key_blocks(case, sms) > 10
    dim, sub, dtype, hq, hkv, page, lens, news = case
    window = 2600 if kind == "window" else 0
    c = make(dim + sub, dim, sub, dtype, hq, hkv, page, lens, news, gain=6.0 if kind == "late" else 1.0, late=kind == "late",
             holes=kind == "holes")
    out, lse = run(vq, c, window)
    assert vq.vq_kernel_status() == 0
    check(c, out, lse, window)


FEW = [  # dim, sub, dtype, hq, hkv, page
    (128, 8, "f16", 16, 4, 16), (128, 4, "bf16", 16, 4, 64), (64, 8, "bf16", 12, 4, 32), (64, 4, "f16", 8, 8, 16),
    (256, 4, "f16", 12, 4, 16), (256, 8, "bf16", 16, 4, 128)]


def few_case(case, new, kind):
    dim, sub, dtype, hq, hkv, page = case
    lens = [new + 500 * r + 37 * (r % 5) for r in range(34)]
    assert sum(-(-n // 128) for n in lens) * hkv > 10 * 304  # units a block: 30 groups of tokens a warp
    return make(dim + sub + new, dim, sub, dtype, hq, hkv, page, lens, [new] * len(lens),
                gain=6.0 if kind == "late" else 1.0, late=kind == "late", holes=kind == "holes")


@pytest.mark.parametrize("case", FEW)
@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("kind", ["plain", "window", "late", "holes"])
def test_long_decode(vq, case, new, kind):
    """A few rows over caches of up to 17000 tokens, every warp through tens of groups."""
    window = 4000 if kind == "window" else 0
    c = few_case(case, new, kind)
    out, lse = run(vq, c, window)
    assert vq.vq_kernel_status() == 0
    check(c, out, lse, window, pieces=2)


@pytest.mark.parametrize("case", [FEW[0], FEW[2], FEW[4]])
def test_long_decode_through_the_checked_build(libs, case):  # noqa: F811
    import product_vq_kv_gb300 as m

    c = few_case(case, 3, "holes")
    want, got = both(libs, lambda: run(m, c, 4000))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))


@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[4]])
def test_long_chunks_through_the_checked_build(libs, case):  # noqa: F811
    import product_vq_kv_gb300 as m

    dim, sub, dtype, hq, hkv, page, lens, news = case
    c = make(dim, dim, sub, dtype, hq, hkv, page, lens, news, gain=6.0, late=True, holes=True)
    want, got = both(libs, lambda: run(m, c, 3000))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    check(c, *got, 3000)
