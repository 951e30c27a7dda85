"""Refusals of the paged calls, on the host: nothing here launches."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # an address that is never used


@pytest.fixture(scope="module")
def lib():
    from product_vq_kv_gb300.build import build
    import product_vq_kv_gb300._binding as bind

    return bind._configure(ctypes.CDLL(build()))


RESERVE = dict(lens=P, new=P, requests=4, free=P, count=P, pages=10, table=P, blocks=8, page=16, total=5,
               lens_out=P, count_out=P, cu=P, slots=P)
TRIM = dict(lens=P, keep=P, requests=4, table=P, blocks=8, page=16, free=P, count=P, pages=10, lens_out=P,
            count_out=P)
APPEND = dict(k=P, v=P, k_stride=256, v_stride=256, slots=P, tokens=4, heads=2, dim=128, sub=8, n_c=256, kcb=P,
              vcb=P, smooth=0, kc=P, vc=P, pages=4, page=16, stride=512, dtype=0)
ATTEND = dict(q=P, q_stride=512, cu=P, lens=P, requests=2, tokens=3, max_new=2, table=P, blocks=8, kc=P, vc=P,
              pages=4, page=16, stride=512, kcb=P, vcb=P, hq=4, hkv=2, dim=128, sub=8, n_c=256, window=0, scale=0.0,
              dtype=0, out=P, lse=P, ws=P, ws_bytes=0)


def call(fn, base, **change):
    args = {**base, **change}
    assert set(args) == set(base)
    return fn(*[None if isinstance(v, int) and v == 0 and isinstance(base[k], int) and base[k] == P else v
                for k, v in args.items()], None)


@pytest.mark.parametrize("change, want", [
    (dict(page=0), INVALID), (dict(page=24), INVALID), (dict(page=2048), UNSUPPORTED), (dict(requests=-1), INVALID),
    (dict(requests=8193), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(blocks=-1), INVALID), (dict(blocks=1 << 27), UNSUPPORTED), (dict(total=-1), INVALID),
    (dict(total=(1 << 30) + 1), UNSUPPORTED), (dict(lens=0), INVALID), (dict(new=0), INVALID),
    (dict(free=0), INVALID), (dict(count=0), INVALID), (dict(table=0), INVALID), (dict(lens_out=0), INVALID),
    (dict(count_out=0), INVALID), (dict(cu=0), INVALID), (dict(slots=0), INVALID), (dict(lens=P + 2), INVALID),
    (dict(slots=P + 4), INVALID), (dict(table=P + 1), INVALID)])
def test_reserve_refusals(lib, change, want):
    assert call(lib.vq_paged_reserve, RESERVE, **change) == want


@pytest.mark.parametrize("change, want", [
    (dict(page=3), INVALID), (dict(page=4096), UNSUPPORTED), (dict(requests=-1), INVALID),
    (dict(requests=8193), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(blocks=-2), INVALID), (dict(lens=0), INVALID),
    (dict(keep=0), INVALID), (dict(table=0), INVALID), (dict(free=0), INVALID), (dict(count=0), INVALID),
    (dict(lens_out=0), INVALID), (dict(count_out=0), INVALID), (dict(keep=P + 3), INVALID)])
def test_trim_refusals(lib, change, want):
    assert call(lib.vq_paged_trim, TRIM, **change) == want


@pytest.mark.parametrize("change, want", [
    (dict(dtype=7), INVALID), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(sub=0), INVALID),
    (dict(sub=7), INVALID), (dict(dim=0), INVALID), (dict(sub=64), UNSUPPORTED), (dict(dim=520), UNSUPPORTED),
    (dict(heads=1025), UNSUPPORTED), (dict(n_c=0), UNSUPPORTED), (dict(n_c=257), UNSUPPORTED), (dict(page=12), INVALID),
    (dict(page=0), INVALID), (dict(page=2048), UNSUPPORTED), (dict(stride=511), INVALID), (dict(k_stride=255), INVALID),
    (dict(v_stride=255), INVALID), (dict(pages=-1), INVALID), (dict(tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(k_stride=1 << 40), UNSUPPORTED), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID),
    (dict(kcb=0), INVALID), (dict(vcb=0), INVALID), (dict(kc=0), INVALID), (dict(vc=0), INVALID),
    (dict(k=P + 1), INVALID), (dict(slots=P + 4), INVALID), (dict(smooth=P + 2), INVALID), (dict(vcb=P + 1), INVALID),
    (dict(pages=1 << 40, stride=1 << 40), INVALID), (dict(tokens=0), OK), (dict(pages=0, kc=0, vc=0), OK)])
def test_append_refusals(lib, change, want):
    assert call(lib.vq_paged_append, APPEND, **change) == want


@pytest.mark.parametrize("change, want", [
    (dict(dtype=-1), INVALID), (dict(requests=-1), INVALID), (dict(tokens=-1), INVALID), (dict(max_new=-1), INVALID),
    (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=5), INVALID), (dict(hq=2048), UNSUPPORTED),
    (dict(sub=5), INVALID), (dict(dim=0), INVALID), (dict(dim=1024), UNSUPPORTED), (dict(n_c=0), UNSUPPORTED),
    (dict(n_c=300), UNSUPPORTED), (dict(page=48), INVALID), (dict(page=2048), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(stride=100), INVALID), (dict(q_stride=511), INVALID),
    (dict(q_stride=1 << 40), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(blocks=-1), INVALID), (dict(blocks=1 << 27), UNSUPPORTED), (dict(requests=1 << 25), UNSUPPORTED),
    (dict(tokens=(1 << 30) + 1), UNSUPPORTED), (dict(q=0), INVALID), (dict(cu=0), INVALID), (dict(lens=0), INVALID),
    (dict(table=0), INVALID), (dict(kc=0), INVALID), (dict(vc=0), INVALID), (dict(kcb=0), INVALID),
    (dict(vcb=0), INVALID), (dict(out=0), INVALID), (dict(ws=0), INVALID), (dict(q=P + 1), INVALID),
    (dict(lse=P + 2), INVALID), (dict(cu=P + 2), INVALID), (dict(ws=P + 8), INVALID), (dict(), INVALID),
    (dict(tokens=0), OK)])
def test_attention_refusals(lib, change, want):
    """(The call without a change has a workspace of no bytes.)"""
    assert call(lib.vq_paged_attention, ATTEND, **change) == want


def test_workspace_bytes(lib):
    fn = lib.vq_paged_attention_workspace_bytes
    assert fn(2, 3, 1, 4, 2, 128, 8, 256, 16) > 0
    assert fn(2, 1000000, 0, 4, 2, 128, 8, 256, 16) < 1 << 30
    for bad in ((-1, 3, 1, 4, 2, 128, 8, 256, 16), (2, 3, 1, 5, 2, 128, 8, 256, 16), (2, 3, 1, 4, 2, 128, 7, 256, 16),
                (2, 3, 1, 4, 2, 128, 8, 257, 16), (2, 3, 1, 4, 2, 128, 8, 256, 17)):
        assert fn(*bad) == 0


def test_binding_refusals():
    """The wrappers check types and shapes before any pointer is taken."""
    import product_vq_kv_gb300 as vq

    i = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros((4, 8), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        vq.vq_paged_reserve(i.long(), i, i, one, table, 16, 3)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_reserve(i, i, i, one, table, 16, 3)
    with pytest.raises(ValueError, match="shape"):
        vq.vq_paged_trim(table, i, table, 16, i, one)
    x = torch.zeros((4, 2, 128), dtype=torch.float16)
    codes = torch.zeros((3, 2, 16, 16), dtype=torch.uint8)
    books = torch.zeros((2, 256, 8), dtype=torch.float16)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="dtype"):
        vq.vq_paged_append(x.double(), x.double(), slots, books, books, codes, codes)
    with pytest.raises(ValueError, match="contiguous within a token"):
        vq.vq_paged_append(x.transpose(1, 2), x, slots, books, books, codes, codes)
    with pytest.raises(ValueError, match="must not overlap"):
        vq.vq_paged_append(x[:1].expand(4, 2, 128), x, slots, books, books, codes, codes)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_attention(x, i[:2], i[:1], table[:1], codes, codes, books, books)
    with pytest.raises(TypeError, match="Tensor"):
        vq.vq_paged_attention(None, i[:2], i[:1], table[:1], codes, codes, books, books)
