"""Memory that a call takes for work on another stream than the current one: on which
stream it is allocated (on the host, with fakes), and what the results are."""
import contextlib

import pytest
import torch

import product_vq_kv_gb300 as vq
import product_vq_kv_gb300._binding as bind


class FakeCuda(torch.Tensor):
    """A host tensor that says it is on the GPU; nothing is launched on it."""

    @property
    def is_cuda(self):
        return True


class FakeStream:
    cuda_stream = 77


def fake(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(FakeCuda)


@pytest.fixture
def allocations(monkeypatch):
    """The stream (None: the current one) of every torch.empty of a call."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(shape, dtype=None, device=None):
        seen.append(current[-1])
        return fake(shape, dtype)

    def empty_like(t):
        return empty(t.shape, t.dtype)

    class Library:
        def __getattr__(self, name):
            return lambda *args: 64 if name.endswith("workspace_bytes") else 0

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", empty_like)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(bind, "load_library", Library)
    monkeypatch.setattr(bind, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(bind, "_paged_workspace", lambda *sizes: 64)
    return seen


def i32(*shape):
    return fake(shape, torch.int32)


def half(*shape):
    return fake(shape, torch.float16)


def u8(*shape):
    return fake(shape, torch.uint8)


PAGED = {
    "reserve": (4, lambda kw: vq.vq_paged_reserve(i32(3), i32(3), i32(9), i32(1), i32(3, 5), 16, 7, **kw)),
    "trim": (2, lambda kw: vq.vq_paged_trim(i32(3), i32(3), i32(3, 5), 16, i32(9), i32(1), **kw)),
    "attention": (3, lambda kw: vq.vq_paged_attention(half(4, 4, 64), i32(3), i32(2), i32(2, 5), u8(9, 2, 16, 8),
                                                      u8(9, 2, 16, 8), half(2, 256, 8), half(2, 256, 8),
                                                      return_lse=True, **kw)),
}

DENSE = {
    "encode": (1, lambda kw: vq.vq_encode(half(9, 8), half(16, 8), **kw)),
    "grouped": (1, lambda kw: vq.vq_encode_grouped(half(2, 9, 8), half(2, 16, 8), **kw)),
    "u8": (1, lambda kw: vq.vq_encode_grouped_u8(half(2, 9, 8), half(2, 16, 8), **kw)),
    "smooth": (1, lambda kw: vq.vq_encode_grouped_smooth(half(2, 9, 8), fake((2, 64), torch.float32), half(2, 16, 8), 64,
                                                         **kw)),
    "scalar": (2, lambda kw: vq.vq_scalar_quantize(half(9, 8), fake((16,), torch.float32), **kw)),
    "scalar back": (1, lambda kw: vq.vq_scalar_dequantize(u8(9, 8), fake((16,), torch.float32), **kw)),
    "rotate": (1, lambda kw: vq.vq_hadamard_rotate(half(9, 8), fake((8,), torch.float32), **kw)),
    "hadamard": (1, lambda kw: vq.vq_hadamard_quantize(half(9, 8), fake((8,), torch.float32),
                                                       fake((4,), torch.float32), **kw)),
    "decode": (1, lambda kw: vq.vq_dequantize_grouped(u8(2, 9), half(2, 16, 8), **kw)),
    "attention": (2, lambda kw: vq.vq_attention_decode(half(1, 4, 64), u8(1, 2, 5, 8), half(2, 256, 8), u8(1, 2, 5, 8),
                                                       half(2, 256, 8), **kw)),
    "static attention": (1, lambda kw: vq.vq_attention_decode_static(half(1, 4, 64), u8(1, 2, 5, 8), half(2, 256, 8),
                                                                     u8(1, 2, 5, 8), half(2, 256, 8), **kw)),
}


@pytest.mark.parametrize("name", DENSE)
def test_dense_allocations_are_made_on_the_streams_of_their_work(allocations, monkeypatch, name):
    monkeypatch.setattr(bind, "_stream_handle", lambda stream, device: 0)
    count, call = DENSE[name]
    call({})
    assert allocations == [None] * count
    allocations.clear()
    side = FakeStream()
    call({"stream": side})
    assert allocations == [side] * count


@pytest.mark.parametrize("name", PAGED)
def test_paged_allocations_are_made_on_the_streams_of_their_work(allocations, name):
    count, call = PAGED[name]
    call({})
    assert allocations == [None] * count
    allocations.clear()
    side = FakeStream()
    call({"stream": side})
    assert allocations == [side] * count


# ------------------------------------------------------------------ results


def paged_case(seed, new):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    requests, hq, hkv, dim, page, blocks = 6, 8, 2, 128, 16, 200
    tokens, pages = requests * new, requests * blocks
    q = torch.randn((tokens, hq, dim), generator=gen, device="cuda").half()
    cu = torch.arange(0, tokens + 1, new, dtype=torch.int32, device="cuda")
    lens = torch.randint(1000, page * blocks, (requests,), generator=gen, device="cuda").int()
    table = torch.randperm(pages, generator=gen, device="cuda").int().reshape(requests, blocks)
    kc, vc = (torch.randint(0, 256, (pages, hkv, page, dim // 8), generator=gen, device="cuda", dtype=torch.uint8)
              for _ in range(2))
    kcb, vcb = (torch.randn((hkv, 256, 8), generator=gen, device="cuda").half() for _ in range(2))
    return q, cu, lens, table, kc, vc, kcb, vcb


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 40])
def test_paged_attention_on_side_streams_without_workspaces(new):
    """Calls that overlap on two side streams, and work of the current stream on memory
    that it takes right behind them: what the same calls give one after the other."""
    cases = [paged_case(s, new) for s in range(2)]
    want = [vq.vq_paged_attention(*c, max_new=new, return_lse=True) for c in cases]
    sides = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for side, case in zip(sides, cases):
            got.append(vq.vq_paged_attention(*case, max_new=new, return_lse=True, stream=side))
        scratch = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (1 << 12, 1 << 18, 1 << 22)]
        del scratch
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


@pytest.mark.gpu
def test_attention_decode_on_side_streams_without_workspaces():
    gen = torch.Generator(device="cuda").manual_seed(3)
    cases = []
    for _ in range(2):
        q = torch.randn((4, 8, 128), generator=gen, device="cuda").half()
        kc, vc = (torch.randint(0, 256, (4, 2, 3000, 16), generator=gen, device="cuda", dtype=torch.uint8)
                  for _ in range(2))
        kcb, vcb = (torch.randn((2, 256, 8), generator=gen, device="cuda").half() for _ in range(2))
        cases.append((q, kc, kcb, vc, vcb))
    want = [vq.vq_attention_decode(*c) for c in cases]
    sides = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got += [vq.vq_attention_decode(*case, stream=side) for side, case in zip(sides, cases)]
        scratch = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (1 << 12, 1 << 18, 1 << 22)]
        del scratch
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 2])
