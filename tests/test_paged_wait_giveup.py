"""The give-up path of the paged chunk attention's bounded waits, on the GPU.

Should a wait give up, its block must not free its tensor memory while a product that
it issued may still write there; the rows that it has not written become NaN, also those
that other blocks hold parts of, and the device status word says so.  In the library the
limit has never been reached; ``tests/harness/paged_polls.cu`` builds the same kernel with
0 or 1 polls a wait.  No wait is left unbounded and no access differs from the library's:
the waits only run out early.
"""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


@pytest.fixture(scope="module")
def harness(vq):
    import product_vq_kv_gb300._binding as bind
    import tc_harness

    lib, like = tc_harness.load(), bind.load_library()
    lib.polls_paged_attention.restype = ctypes.c_int32
    lib.polls_paged_attention.argtypes = like.vq_paged_attention.argtypes
    return lib


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def status(lib, clear=True):
    bits = ctypes.c_uint32(0)
    assert lib.polls_paged_status(ctypes.byref(bits), 1 if clear else 0) == 0
    return bits.value


def case(dim, hq, hkv, new, held, window):
    """One request (its new tokens all go to the chunk kernel)."""
    gen = torch.Generator(device="cuda").manual_seed(dim + new)
    page = 16
    pages = -(-held // page)
    q = torch.randn((new, hq, dim), generator=gen, device="cuda").half()
    kc, vc = (torch.randint(0, 256, (pages, hkv, page, dim // 8), generator=gen, device="cuda", dtype=torch.uint8)
              for _ in range(2))
    kcb, vcb = (torch.randn((hkv, 256, 8), generator=gen, device="cuda").half() for _ in range(2))
    return dict(q=q, cu=i32([0, new]), lens=i32([held]), table=torch.randperm(pages, generator=gen, device="cuda").int()[None],
                kc=kc, vc=vc, kcb=kcb, vcb=vcb, window=window)


def run(vq, lib, polls, c):
    new, hq, dim = c["q"].shape
    pages, hkv, page, ns = c["kc"].shape
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full((new, hq), 7.0, device="cuda")
    ws = torch.zeros(vq.vq_paged_attention_workspace_bytes(1, new, new, hq, hkv, dim, 8, 256, page), dtype=torch.uint8,
                     device="cuda")
    lib.polls_paged_set(polls)
    p = torch.Tensor.data_ptr
    assert lib.polls_paged_attention(
        p(c["q"]), hq * dim, p(c["cu"]), p(c["lens"]), 1, new, new, p(c["table"]), pages, p(c["kc"]), p(c["vc"]), pages,
        page, hkv * page * ns, p(c["kcb"]), p(c["vcb"]), hq, hkv, dim, 8, 256, c["window"], 0.0, 0, p(out), p(lse), p(ws),
        ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return out, lse


def library(vq, c):
    return vq.vq_paged_attention(c["q"], c["cu"], c["lens"], c["table"], c["kc"], c["vc"], c["kcb"], c["vcb"],
                                 max_new=c["q"].shape[0], window=c["window"], return_lse=True)


CASES = [(128, 8, 2, 100, 700, 0), (128, 32, 8, 900, 2000, 0), (128, 12, 4, 300, 1500, 500)]


@pytest.mark.parametrize("args", CASES)
def test_no_polls_mark_every_row(vq, harness, args):
    c = case(*args)
    status(harness)
    out, lse = run(vq, harness, 0, c)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    assert status(harness) & vq.VQ_KSTATUS_WAIT_GAVE_UP
    assert status(harness) == 0
    out, lse = library(vq, c)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and vq.vq_kernel_status() == 0


@pytest.mark.parametrize("args", CASES + [(256, 6, 2, 300, 900, 0), (256, 12, 4, 700, 1500, 400)])
def test_one_poll_leaves_rows_right_or_marked(vq, harness, args):
    c = case(*args)
    want, want_lse = library(vq, c)
    some = 0
    for _ in range(4):
        status(harness)
        out, lse = run(vq, harness, 1, c)
        marked = torch.isnan(out).any(-1)
        assert torch.equal(marked, torch.isnan(out).all(-1)) and torch.equal(marked, torch.isnan(lse))
        assert torch.equal(out[~marked], want[~marked]) and torch.equal(lse[~marked], want_lse[~marked])
        gave_up = bool(status(harness) & vq.VQ_KSTATUS_WAIT_GAVE_UP)
        assert gave_up or not marked.any()
        some += int(marked.sum())
    print(f"[one poll] {args}: {some} rows marked")
    again, _ = library(vq, c)
    assert torch.equal(again, want) and vq.vq_kernel_status() == 0
