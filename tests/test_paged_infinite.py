"""Scores of -inf in the paged attention: they weigh nothing beside others, and a row of
nothing else is NaN, as 0 / 0 is, while a row that sees no token at all stays zero."""
import math

import numpy as np
import pytest
import torch

from test_paged import DTYPES, HALF_EPS, SHAPES, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("window", [0, 40])
def test_rows_of_scores_of_minus_infinity(vq, shape, new, window):
    """Keys that are all positive and a query with -inf in it: every score is -inf."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    c = Cache(31, [900, 60, 9, 200], hq, hkv, dim, sub, n_c, page, dtype)
    c.kcb = c.kcb.abs().clamp(min=0.25)
    for b in range(len(c.table[3])):
        c.table[3][b] = -1  # the last request has no pages: its rows see nothing
    lens, table, kc, vc = c.device()
    tokens = 4 * new
    cu = i32([0, new, 2 * new, 3 * new, tokens])
    q = c.queries(tokens).cuda()
    clean = q.clone()
    hit = torch.zeros((tokens, hq), dtype=torch.bool, device="cuda")
    hit[::2, ::2] = True
    hit[new - 1, hq - 1] = True
    q[..., 3] = torch.where(hit, torch.full_like(q[..., 3], -math.inf), q[..., 3])
    args = (cu, lens, table, kc, vc, c.kcb, c.vcb)
    out, lse = vq.vq_paged_attention(q, *args, max_new=new, window=window, return_lse=True)
    want, want_lse = vq.vq_paged_attention(clean, *args, max_new=new, window=window, return_lse=True)
    assert vq.vq_kernel_status() == 0
    row = torch.arange(tokens, device="cuda")
    pos = lens[row // new] - new + row % new
    sees = ((pos >= 0) & (row // new < 3))[:, None]
    nan = hit & sees
    assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()
    blind = ~sees.expand(-1, hq)
    assert (out[blind] == 0).all() and torch.isneginf(lse[blind]).all()
    rest = ~nan
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[6] != "f16"])
@pytest.mark.parametrize("new", [1, 60])
def test_scores_of_minus_infinity_weigh_nothing(vq, shape, new):
    """Keys whose product with the query leaves fp32's range downwards, for the first 300
    tokens and some later ones, beside keys of score 0: the mean of the others' values.

    n values of weight 1: their sum is off by n 2^-22 of the largest (any order, rounded
    or cut off), its quotient and the weights' 2^-21, and it is rounded once."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    held = 1100
    c = Cache(32, [held, 400], hq, hkv, dim, sub, n_c, page, dtype)
    c.kcb.zero_()
    c.kcb[:, 1, 0] = -2.0 ** 100
    c.kc[:] = 0
    far = np.zeros((2, held), bool)
    far[:, :300] = True
    far[:, 300::5] = True
    for r, length in enumerate(c.lens):
        for t in range(length):
            if far[r, t]:
                c.kc[c.table[r][t // page], :, t % page, 0] = 1
    lens, table, kc, vc = c.device()
    q = torch.ones((2 * new, hq, dim), dtype=DTYPES[dtype], device="cuda")
    q[..., 0] = 2.0 ** 100
    out, lse = vq.vq_paged_attention(q, i32([0, new, 2 * new]), lens, table, kc, vc, c.kcb, c.vcb, max_new=new, return_lse=True)
    assert vq.vq_kernel_status() == 0
    book = c.vcb_h.double().numpy()
    for r, length in enumerate(c.lens):
        where = np.arange(length)
        pages = np.array(c.table[r])[where // page]
        near = np.flatnonzero(~far[r, :length])
        for h in range(hkv):
            codes = c.vc[pages, h, where % page].astype(int)
            values = book[h][codes].reshape(length, dim)
            for i in {0, new - 1}:
                seen = near[near <= length - new + i]
                want = values[seen].mean(0)
                tol = np.abs(values).max() * (len(seen) * 2.0 ** -22 + 2.0 ** -20) + HALF_EPS[dtype] * (np.abs(want) + 0.01)
                for head in range(h * hq // hkv, (h + 1) * hq // hkv):
                    got = out[r * new + i, head].double().cpu().numpy()
                    assert (np.abs(got - want) <= tol).all()
                    assert abs(lse[r * new + i, head].item() - math.log(len(seen))) <= 2.0 ** -18
