"""The calls on the cache in 4 bits and on shared pages through the bounds-checked build:
every kernel index checked before its access, the outputs the library build's bit for bit,
and the status word clear."""
import pytest
import torch

from test_checked_build import both, libs  # noqa: F401  (a fixture)
from test_paged_checked import equal, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, dim, n_c, tokens, rotate", [
    (torch.float16, 128, 16, 77, True), (torch.bfloat16, 256, 16, 300, False), (torch.float32, 64, 16, 19, True),
    (torch.float16, 96, 9, 33, False), (torch.bfloat16, 8, 16, 40, True), (torch.float32, 512, 3, 21, True)])
def test_append(libs, dtype, dim, n_c, tokens, rotate):  # noqa: F811
    import product_vq_kv_gb300 as vq

    gen = torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randn((tokens, 6, dim), generator=gen, device="cuda").to(dtype)
    cents = torch.randn(n_c, generator=gen, device="cuda")
    signs = torch.randint(0, 2, (dim,), generator=gen, device="cuda").float() * 2 - 1 if rotate else None
    slots = torch.randperm(16 * 32, generator=gen, device="cuda")[:tokens].clone()
    slots[::5] = -1

    def run():
        kc = torch.zeros((32, 2, 16, dim // 2), dtype=torch.uint8, device="cuda")
        ks = torch.zeros((32, 2, 16), dtype=dtype, device="cuda")
        vc, vs = torch.zeros_like(kc), torch.zeros_like(ks)
        vq.vq_paged_scalar_append(packed[:, 2:4], packed[:, 4:], slots, cents, cents, kc, vc, ks, vs, k_signs=signs)
        return kc, vc, ks, vs

    assert equal(*both(libs, run))


@pytest.mark.parametrize("dtype, dim, page", [
    (torch.float16, 128, 16), (torch.bfloat16, 256, 32), (torch.float16, 64, 64), (torch.bfloat16, 64, 16),
    (torch.float16, 256, 16), (torch.bfloat16, 128, 16), (torch.float32, 128, 16), (torch.float16, 96, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_attention(libs, dtype, dim, page, window):  # noqa: F811
    import product_vq_kv_gb300 as vq

    gen = torch.Generator(device="cuda").manual_seed(2)
    lens, new = [1, 400, 129, 260, 64, 0], [1, 3, 129, 150, 1, 2]
    blocks = 400 // page + 1
    pages = 6 * blocks
    table = torch.randperm(pages, generator=gen, device="cuda").int().reshape(6, blocks)
    table[3, 1] = -1
    table[1, 0] = pages + 7
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1] + 2, 6, dim), generator=gen, device="cuda").to(dtype)
    kc, vc = (torch.randint(0, 256, (pages, 2, page, dim // 2), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.rand((pages, 2, page), generator=gen, device="cuda").to(dtype) for _ in range(2))
    cents = torch.randn(13, generator=gen, device="cuda")

    def run():
        return vq.vq_paged_scalar_attention(q, i32(cu), i32(lens), table, kc, vc, ks, vs, cents, cents, max_new=150,
                                            window=window, return_lse=True)

    assert equal(*both(libs, run))


@pytest.mark.parametrize("seats, width, page", [(5, 3, 4), (300, 140, 16), (2000, 3, 1)])
def test_fork_compact_and_copy(libs, seats, width, page):  # noqa: F811
    import product_vq_kv_gb300 as vq

    gen = torch.Generator(device="cuda").manual_seed(3)
    lens = torch.randint(0, width * page + 1, (seats,), generator=gen, device="cuda").int()
    pages = seats * width + 37
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = order[:seats * width].reshape(seats, width).contiguous()
    parents = torch.randint(-1, seats, (seats,), generator=gen, device="cuda").int()
    data = torch.randint(0, 256, (2, pages, 50), generator=gen, device="cuda", dtype=torch.uint8)

    def run():
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        free[:37] = order[seats * width:]
        pool = data.clone()
        kept, forked, count, copies = vq.vq_paged_fork(lens, parents, table, page, free, i32([37]))
        vq.vq_paged_copy(copies, [pool, pool[:, :, :16].contiguous()], layered=True)
        out = vq.vq_paged_compact(kept, forked, page, free, count)
        vq.vq_paged_copy(out[3], [pool], layered=True)
        return (kept, forked, count, copies, free, pool, *out)

    assert equal(*both(libs, run))
