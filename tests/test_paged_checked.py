"""The paged calls through the bounds-checked build (``libvqenc_checked.so``):
every kernel index checked before its access, the outputs the library build's
bit for bit, and the status word clear."""
import pytest
import torch

from test_checked_build import both, libs  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("new, page, pages", [([1, 0, 40], 16, 9), ([17] * 70, 4, 200), ([3] * 1500, 8, 2000)])
def test_reserve_and_trim(libs, new, page, pages):  # noqa: F811
    import product_vq_kv_gb300 as vq

    n = len(new)

    def run():
        table = torch.full((n, 10), -1, dtype=torch.int32, device="cuda")
        free, lens = torch.arange(pages, dtype=torch.int32, device="cuda"), i32([5 if i % 3 else 0 for i in range(n)])
        lens, count, cu, slots = vq.vq_paged_reserve(lens, i32(new), free, i32([pages]), table, page, sum(new) + 3)
        kept, left = vq.vq_paged_trim(lens, lens // 2, table, page, free, count)
        return lens, count, cu, slots, table, kept, left, free

    assert equal(*both(libs, run))


@pytest.mark.parametrize("dtype, dim, sub, n_c, tokens, smooth", [
    (torch.float16, 128, 8, 256, 77, True), (torch.bfloat16, 256, 4, 100, 300, False), (torch.float32, 64, 8, 64, 19, True),
    (torch.float16, 96, 3, 50, 33, False)])
def test_append(libs, dtype, dim, sub, n_c, tokens, smooth):  # noqa: F811
    import product_vq_kv_gb300 as vq

    gen = torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randn((tokens, 6, dim), generator=gen, device="cuda").to(dtype)
    kcb, vcb = (torch.randn((2, n_c, sub), generator=gen, device="cuda").to(dtype) for _ in range(2))
    slots = torch.randperm(16 * 32, generator=gen, device="cuda")[:tokens].clone()
    slots[::5] = -1
    f = torch.rand((2, dim), generator=gen, device="cuda") + 0.5 if smooth else None

    def run():
        kc = torch.zeros((32, 2, 16, dim // sub), dtype=torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        vq.vq_paged_append(packed[:, 2:4], packed[:, 4:], slots, kcb, vcb, kc, vc, k_smooth=f)
        return kc, vc

    assert equal(*both(libs, run))


@pytest.mark.parametrize("dtype, dim, sub, page", [
    (torch.float16, 128, 8, 16), (torch.bfloat16, 256, 4, 32), (torch.float16, 64, 4, 64), (torch.bfloat16, 64, 8, 16),
    (torch.float16, 256, 8, 16), (torch.bfloat16, 128, 4, 16), (torch.float32, 128, 8, 16), (torch.float16, 96, 8, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_attention(libs, dtype, dim, sub, page, window):  # noqa: F811
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
    kc, vc = (torch.randint(0, 256, (pages, 2, page, dim // sub), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2))
    kcb, vcb = (torch.randn((2, 200, sub), generator=gen, device="cuda").to(dtype) for _ in range(2))

    def run():
        return vq.vq_paged_attention(q, i32(cu), i32(lens), table, kc, vc, kcb, vcb, max_new=150, window=window,
                                     return_lse=True)

    assert equal(*both(libs, run))
