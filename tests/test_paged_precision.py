"""What the 16-bit weights of the paged attention keep, on the GPU: masses made of many
small weights, and rows that one token decides."""
import math

import numpy as np
import pytest
import torch

import paged_reference as ref
from test_paged import HALF_EPS, HALF_STEP, SHAPES, Cache

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim, sub", [(64, 8), (128, 8), (256, 4)])
@pytest.mark.parametrize("new", [1, 100])
def test_many_small_weights_beside_large_ones(vq, dtype, dim, sub, new):
    """Every 64th run of 128 tokens has 8 tokens, 16 apart, of score 26 (in powers of
    two) and value 0; the n other tokens have score 0 and value 256.  With the large ones
    in reach of every part of the work, out = 256 n 2^-26 / (large + n 2^-26).

    The numerator is a sum of equal positive terms: off by a relative n 2^-22 at most
    in any order, rounded or cut off.  In the sum of weights the small ones stand beside
    the large ones, and what is lost of them there is at most all, n 2^-26.  The exponent
    26 is a sum of dim exact products, times a rounded factor: off by 28 x 2^-23, and the
    weights by that times ln 2 and the exponential's 2^-21.  The output is rounded once."""
    held, page, requests, hkv = 65536, 256, 8, 8
    pages = held // page
    kcb = torch.zeros((hkv, 2, sub), dtype=DTYPES[dtype], device="cuda")
    vcb = kcb.clone()
    kcb[:, 1] = 1.0
    vcb[:, 0] = 256.0
    t = torch.arange(held, device="cuda")
    large = (t // 128 % 64 == 0) & (t % 16 == 5)
    order = torch.randperm(pages, device="cuda")
    codes = large.to(torch.uint8).reshape(pages, 1, page, 1).expand(pages, hkv, page, dim // sub)
    kc = torch.empty((pages, hkv, page, dim // sub), dtype=torch.uint8, device="cuda")
    kc[order] = codes
    table = order.int()[None].repeat(requests, 1)
    q = torch.ones((requests * new, 2 * hkv, dim), dtype=DTYPES[dtype], device="cuda")
    cu = i32([new * r for r in range(requests + 1)])
    out, lse = vq.vq_paged_attention(q, cu, i32([held] * requests), table, kc, kc, kcb, vcb, max_new=new,
                                     scale=26 * math.log(2) / dim, return_lse=True)
    assert vq.vq_kernel_status() == 0
    many = large.sum().item()
    n = torch.arange(held - new, held, dtype=torch.float64, device="cuda").add(1 - many).repeat(requests)[:, None, None]
    want = 256 * n * 2.0 ** -26 / (many + n * 2.0 ** -26)
    rel = held * 2.0 ** -22 + held * 2.0 ** -26 / many + 28 * 2.0 ** -23 + 2.0 ** -21 + torch.finfo(DTYPES[dtype]).eps / 2
    assert ((out.double() - want).abs() <= rel * want).all()
    want_lse = (26 * math.log(2) + torch.log(many + n * 2.0 ** -26))[:, :, 0]
    assert ((lse.double() - want_lse).abs() <= held * 2.0 ** -26 / many + 34 * 2.0 ** -23 + 2.0 ** -21).all()


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2] in (64, 128, 256) and s[3] in (4, 8) and s[5] >= 16
                                   and s[6] != "f32"])
@pytest.mark.parametrize("gain", [1.0, 4.0, 30.0])
@pytest.mark.parametrize("new", [1, 3])
def test_a_few_rows_keep_their_weights_in_two_pieces(vq, shape, gain, new):
    """A weight is off by half a step of the type twice over (what the first piece
    leaves is exact in fp32 and rounded again), and in fp16 by half its least step, 2^-25,
    where the maximum's weight is 2^7 or more."""
    hq, hkv, dim, sub, n_c, page, dtype = shape
    if new * hq // hkv > 24:
        pytest.skip("a chunk")
    lens = [new, 17, 130, 300, 900]
    c = Cache(21, lens, hq, hkv, dim, sub, n_c, page, dtype, gain=gain)
    cu = [new * r for r in range(len(lens) + 1)]
    q = c.queries(cu[-1])
    d_lens, table, kc, vc = c.device()
    out, lse = vq.vq_paged_attention(q.cuda(), i32(cu), d_lens, table, kc, vc, c.kcb, c.vcb, max_new=new, return_lse=True)
    eps = HALF_EPS[dtype]
    want, want_lse, tol, tol_lse = ref.attention(
        q.double().numpy(), cu, c.lens, c.table, c.kc, c.vc, c.kcb_h.double().numpy(), c.vcb_h.double().numpy(),
        weight_eps=eps * eps, weight_abs=2.0 ** -32 if dtype == "f16" else HALF_STEP[dtype])
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol + eps * (np.abs(want) + tol) + HALF_STEP[dtype]).all()
    assert (np.abs(lse.double().cpu().numpy() - want_lse) <= tol_lse).all()
