"""A step in which requests are refused pages: what the append and the attention make of
their rows."""
import ctypes

import numpy as np
import pytest
import torch

import paged_reference as ref
from test_paged import HALF_EPS, HALF_STEP, SHAPES, Cache, i32
from test_paged_abi import ATTEND, INVALID, OK, P, call

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


@pytest.mark.parametrize("change, want", [
    (dict(slots=P + 4), INVALID), (dict(slots=P, tokens=0), OK), (dict(tokens=0), OK), (dict(), INVALID),
    (dict(slots=P, hq=5), INVALID)])
def test_refusals_of_the_arguments(vq, change, want):
    """(The call without a change has a workspace of no bytes.)"""
    names = list(ATTEND)
    names.insert(names.index("lens") + 1, "slots")
    base = {name: ATTEND.get(name, 0) for name in names}
    assert call(vq.load_library().vq_paged_attention_slots, base, **change) == want


def test_binding_refusals(vq):
    from test_streams import half, i32 as fake_i32, u8
    from test_streams import fake

    def attend(slots):
        vq.vq_paged_attention(half(4, 4, 64), fake_i32(3), fake_i32(2), fake_i32(2, 5), u8(9, 2, 16, 8), u8(9, 2, 16, 8),
                              half(2, 256, 8), half(2, 256, 8), slots=slots)

    for bad in (fake((3,), torch.int64), fake((4,), torch.int32), fake((4, 1), torch.int64), [0, 1, 2, 3]):
        with pytest.raises(ValueError, match="slots"):
            attend(bad)


def refused_step(vq, shape, news, window=0, seed=41):
    """Reserve for requests of various lengths from a pool that lacks pages for some of
    them, and attend; returns what the reference says beside what came."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    rng = np.random.default_rng(seed)
    held = [int(rng.integers(0, 400)) for _ in news]
    c = Cache(seed, [h + n for h, n in zip(held, news)], hq, hkv, dim, sub, n_c, page, dtype)
    table = [list(row) for row in c.table]
    free = []
    for r, (h, n) in enumerate(zip(held, news)):  # the new tokens' pages are not taken yet
        for b in range(ref.blocks_of(h, page), ref.blocks_of(h + n, page)):
            free.append(table[r][b])
            table[r][b] = -1
    free = free[:len(free) // 2]
    tokens = sum(news) + 2
    d_table = i32(table)
    lens, _, cu, slots = vq.vq_paged_reserve(i32(held), i32(list(news)), i32(free or [0]), i32([len(free)]), d_table, page,
                                             tokens)
    _, _, kc, vc = c.device()
    q = c.queries(tokens)
    args = (q.cuda(), cu, lens, d_table, kc, vc, c.kcb, c.vcb)
    out, lse = vq.vq_paged_attention(*args, max_new=max(news), window=window, return_lse=True, slots=slots)
    plain = vq.vq_paged_attention(*args, max_new=max(news), window=window, return_lse=True)
    assert vq.vq_kernel_status() == 0
    granted = [a > b for a, b in zip(lens.tolist(), held)]
    return c, q, cu.tolist(), lens.tolist(), d_table.tolist(), slots, granted, (out, lse), plain


@gpu
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2], SHAPES[5], SHAPES[7], SHAPES[9], SHAPES[11]])
@pytest.mark.parametrize("news", [[1] * 30, [70, 40, 3, 1, 90, 2, 1, 55], [3, 5, 2] * 4])
@pytest.mark.parametrize("window", [0, 60])
def test_rows_of_refused_requests_are_zeros(vq, shape, news, window):
    c, q, cu, lens, table, slots, granted, (out, lse), plain = refused_step(vq, shape, news, window)
    if all(granted):
        pytest.skip("no page was wanting")
    assert any(granted)
    eps = HALF_EPS[c.dtype]
    # the definition with the refused requests empty
    want, want_lse, tol, tol_lse = ref.attention(
        q.double().numpy(), cu, [n if g else 0 for n, g in zip(lens, granted)], table, c.kc, c.vc,
        c.kcb_h.double().numpy(), c.vcb_h.double().numpy(), window, 0.0, 0.0 if c.dtype == "f32" else eps,
        HALF_STEP[c.dtype])
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(got - want) <= tol + eps * (np.abs(want) + tol) + HALF_STEP[c.dtype]).all()
    fine = np.isfinite(want_lse)
    assert np.array_equal(np.isneginf(got_lse), ~fine)
    assert (np.abs(got_lse[fine] - want_lse[fine]) <= tol_lse[fine]).all()
    hidden = torch.zeros(q.shape[0], dtype=torch.bool)
    for r, g in enumerate(granted):
        if not g:
            hidden[cu[r]:cu[r + 1]] = True
    assert (slots.cpu()[:cu[-1]] < 0).equal(hidden[:cu[-1]])
    assert (out[hidden.cuda()] == 0).all() and torch.isneginf(lse[hidden.cuda()]).all()


@gpu
@pytest.mark.parametrize("news", [[1] * 700, [9] * 650])
def test_more_requests_than_are_staged(vq, news):
    """Lengths read from memory instead of shared memory: refused rows are zeros, and the
    others are those of a call that does not know of refusals, but for the work split."""
    c, q, cu, lens, table, slots, granted, (out, lse), (plain, plain_lse) = refused_step(vq, (4, 2, 64, 8, 256, 16, "f16"), news)
    assert any(granted) and not all(granted)
    rows = torch.tensor(granted + [False]).repeat_interleave(torch.tensor(list(news) + [2])).cuda()
    assert (out[~rows] == 0).all() and torch.isneginf(lse[~rows]).all()
    assert (out[rows] - plain[rows]).abs().max() < 2e-3 and (lse[rows] - plain_lse[rows]).abs().max() < 1e-5


@gpu
def test_refused_rows_through_the_checked_build():
    from test_checked_build import libs, using  # noqa: F401

    from product_vq_kv_gb300 import build as b
    import product_vq_kv_gb300 as vq
    import product_vq_kv_gb300._binding as bind

    b.build(checked=True)
    with using(bind, bind._configure(ctypes.CDLL(b.CHECKED_LIB_PATH))):
        for shape in (SHAPES[0], SHAPES[2], SHAPES[9]):
            refused_step(vq, shape, [70, 40, 3, 1, 90, 2, 1, 55])
            assert bind.vq_kernel_status() == 0
