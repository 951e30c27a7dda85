"""The cache in 4 bits with value scales of any size and sign, against the definition in 64
bits.  Bounds go by what a row sums, not by the largest value that it sees."""
import math

import pytest
import torch

import scalar_reference as ref
from test_paged_scalar_long import make, run, vq  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
FORMS = [(64, F16, 16), (64, BF16, 16), (128, F16, 16), (128, BF16, 32), (256, F16, 16), (256, BF16, 16), (96, F16, 16), (128, F32, 8)]


def check(c, out, lse, chunk=False):
    """(out, lse) against 64 bits; returns the most that an element of `out` is off, in bounds of
    its row.

    With u = 2^-24, S_t a score times log2 e, M the row's largest, w_t = 2^(S_t - M), W their sum,
    V_t a value, s_t its scale, n seen tokens, D the head size:
      * S_t is off by d_t <= (D + 6) u kappa sum_i |q_i K_ti|, what is raised to a power lies within
        |S_t - M| + 110 of 0 (a reference lags by at most 39 and is at most 60 off for the values'
        scales) and is rounded twice, the power is off by 2^-21, and up to 16 rises of the
        reference by 2^-22 each: a weight by a relative e_t.
      * weights enter the product rounded to the type in one piece (chunks, half an epsilon) or in
        two (its square): h more.  Their reference is such that the row's largest w_t |s_t| lies at
        2^3 or above in fp16 (2^6 with two pieces), where the least step is 2^-24: half of that
        is `floor` of it.  bf16 has fp32's range: none.
      * a weight of less than 2^-60 of the row's largest may count as none: powers below 2^-126 have
        fewer bits or are 0, and a reference lies up to 60 above the largest score.
      * sums of n products are off by 4 (n + 200) u of the sum of magnitudes."""
    u = 2.0 ** -24
    dtype = c["dtype"]
    eps, tiny = ref.HALF_EPS[dtype], ref.HALF_STEP[dtype]
    dim = c["q"].shape[-1]
    tensor = dtype is not F32 and dim in (64, 128, 256)
    h = 0.0 if not tensor else eps if chunk else eps ** 2
    floor = 0.0 if not tensor or dtype is BF16 else 2.0 ** -28 if chunk else 2.0 ** -31
    hq = c["q"].shape[1]
    pages, hkv, page, _ = c["kc"].shape
    scale, cents = 1 / math.sqrt(dim), c["cents"].to(dtype).double()
    kappa = scale / math.log(2)
    worst = 0.0
    for r, length in enumerate(c["lens"]):
        a, b = c["cu"][r], c["cu"][r + 1]
        t = torch.arange(length, device="cuda")
        entry = c["table"][r].long()[t // page]
        pos = length - (b - a) + torch.arange(b - a, device="cuda")
        seen = t[None, :] <= pos[:, None]
        n = seen.sum(1, keepdim=True).double()
        for hd in range(hkv):
            rows, sizes = [], []
            for codes, scales in ((c["kc"], c["ks"]), (c["vc"], c["vs"])):
                byte = codes[entry, hd, t % page].long()
                x = torch.stack([cents[byte & 15], cents[byte >> 4]], -1).reshape(length, dim)
                sizes.append(scales[entry, hd, t % page].double())
                rows.append(x * sizes[-1][:, None])
            keys, values = rows
            for g in range(hq // hkv):
                head = hd * (hq // hkv) + g
                q = c["q"][a:b, head].double()
                s = (scale * (q @ keys.t())).masked_fill(~seen, -math.inf)
                top = s.amax(1, keepdim=True)
                w = torch.exp(s - top)
                total = w.sum(1, keepdim=True)
                want, sums = w @ values / total, w @ values.abs() / total
                want_lse = (top + torch.log(total))[:, 0]
                d = (dim + 6) * u * kappa * (q.abs() @ keys.abs().t())
                e = math.log(2) * (d + 2 * u * ((top - s) / math.log(2) + 110)) + 2.0 ** -21 + 2.0 ** -18
                e = e.masked_fill(~seen, 0)
                most = (w * sizes[1].abs()).amax(1, keepdim=True)
                tol = 1.1 * ((w * (e + h)) @ values.abs() / total + want.abs() * (w * e).sum(1, keepdim=True) / total +
                             n * floor * most * cents.abs().max() / total + 4 * (n + 200) * u * sums +
                             (w * (w < 2.0 ** -60)) @ values.abs() / total)
                tol = tol + eps * (want.abs() + tol) + tiny
                tol_lse = 1.1 * (e.amax(1) + (n[:, 0] + 200) * u) + 4 * u * want_lse.abs()
                off = (out[a:b, head].double() - want).abs() / tol
                assert (off <= 1).all(), f"request {r} head {head}: {off.max():.3g} bounds off"
                worst = max(worst, off.max().item())
                assert ((lse[a:b, head].double() - want_lse).abs() <= tol_lse).all()
    return worst


@pytest.mark.parametrize("dim, dtype, page", FORMS)
@pytest.mark.parametrize("new", [1, 3, 200])
@pytest.mark.parametrize("size", [14, 20, 27])
def test_large_values_without_weight(vq, dim, dtype, page, new, size):  # noqa: F811
    """Tokens whose values are 2^size times the others' and whose weight is 2^-60 or less take
    nothing from what a row sums, in the blocks that hold them and in those behind."""
    c = make(dim + size, dim, dtype, 8, 2, page, [1500], [new])
    c["q"] = c["q"].abs()
    c["vs"].fill_(2.0 ** (13 - size))
    for at in (70, 700, 701):  # keys that point away from every query
        entry = c["table"][0, at // page].long(), slice(None), at % page
        c["kc"][entry], c["ks"][entry], c["vs"][entry] = 0, 3.0, 2.0 ** 13
    out, lse = run(vq, c)
    chunk = new * 4 > 32
    check(c, out, lse, chunk)
    # (the bounds tell: rows of zeros, and rows a tenth off, are beyond them)
    for wrong in (torch.zeros_like(out), out * 0.9):
        with pytest.raises(AssertionError, match="bounds off"):
            check(c, wrong, lse, chunk)


@pytest.mark.parametrize("dim, dtype, page", FORMS)
@pytest.mark.parametrize("new", [1, 3, 200])
def test_values_of_both_signs(vq, dim, dtype, page, new):  # noqa: F811
    """Value scales below zero: a caller's cache may hold them."""
    c = make(dim, dim, dtype, 8, 2, page, [1500, 77], [new, 1])
    flip = torch.rand(c["vs"].shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.5
    c["vs"] = torch.where(flip, -c["vs"], c["vs"])
    check(c, *run(vq, c), new * 4 > 32)
    c["vs"] = -c["vs"].abs()
    c["ks"] = torch.where(flip, -c["ks"], c["ks"])
    check(c, *run(vq, c), new * 4 > 32)


@pytest.mark.parametrize("dim, page", [(64, 16), (128, 16), (256, 32), (96, 16)])
@pytest.mark.parametrize("new", [1, 3, 200])
@pytest.mark.parametrize("power", [-90, 90, 118])
def test_values_of_bf16_range(vq, dim, page, new, power):  # noqa: F811
    """Values near both ends of bf16's range, under scores that rise along the sequence (so that
    references lag) and that fall."""
    if power > 90 and (new == 200 or dim == 96):
        pytest.skip("sums of hundreds of such values pass fp32's largest")
    for rising in (True, False):
        c = make(dim + new, dim, BF16, 8, 2, page, [900], [new])
        held = -(-900 // page)
        grow = torch.exp(torch.linspace(-3, 1.7, held * page, device="cuda").reshape(held, 1, page))
        here = c["table"][0, :held].long()
        c["ks"][here] = (c["ks"][here] * (grow if rising else 1 / grow * math.exp(-1.3))).to(BF16)
        c["vs"] = (c["vs"].float() * 2.0 ** power).to(BF16)
        check(c, *run(vq, c), new * 4 > 32)


@pytest.mark.parametrize("dim, dtype, page", FORMS)
@pytest.mark.parametrize("new", [1, 3, 200])
def test_scores_that_leap_over_values_of_zero(vq, dim, dtype, page, new):  # noqa: F811
    """Tokens of no value whose scores pass all others' by up to 2^200 at once: they take the
    weight, and nothing becomes infinite."""
    c = make(dim + 3, dim, dtype, 8, 2, page, [1500], [new])
    c["q"] = c["q"].abs()
    for at, size in ((300, 0.5), (431, 1.0), (700, 2.0), (701, 2.0), (1100, 3.5)):  # keys that point along every query
        entry = c["table"][0, at // page].long(), slice(None), at % page
        c["kc"][entry], c["ks"][entry], c["vs"][entry] = 255, size, 0.0
    out, lse = run(vq, c)
    assert torch.isfinite(out).all()
    check(c, out, lse, new * 4 > 32)


@pytest.mark.parametrize("dim, dtype, page", FORMS)
@pytest.mark.parametrize("new", [3, 300])
def test_rows_beside_rows_of_nan(vq, dim, dtype, page, new):  # noqa: F811
    """Uneven scales of both signs: a row has the same bits whatever path the rows beside it take."""
    c = make(dim + 4, dim, dtype, 8, 2, page, [2000], [new], spread=2.0)
    flip = torch.rand(c["vs"].shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.5
    c["vs"] = torch.where(flip, -c["vs"], c["vs"])
    out, lse = run(vq, c)
    check(c, out, lse, new * 4 > 32)
    hit = torch.zeros(c["q"].shape[:2], dtype=torch.bool, device="cuda")
    hit[::7, 1] = hit[1::9, 6] = hit[2::31] = True
    for value in (math.nan, math.inf, 300.0):
        q = c["q"].clone()
        q[hit] = q[hit] * value
        got, got_lse = run(vq, {**c, "q": q})
        assert torch.equal(got[~hit], out[~hit]) and torch.equal(got_lse[~hit], lse[~hit])
