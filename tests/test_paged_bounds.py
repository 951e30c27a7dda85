"""Calls at the edge of the paged cache's contract through the bounds-checked build: no
access leaves its buffer, and the next call is right."""
import numpy as np
import pytest
import torch

from test_checked_build import libs, using  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype, hq, dim, sub", [
    (torch.float16, 8, 128, 8), (torch.bfloat16, 2, 256, 4), (torch.float16, 4, 64, 8), (torch.float32, 8, 128, 8)])
def test_attention_descending_offsets_stay_inside(libs, dtype, hq, dim, sub):  # noqa: F811
    """Offsets that descend: the walk over the items finds others than the plan did, and
    the parts that its notes name are inside the workspace all the same."""
    import product_vq_kv_gb300 as vq

    bind, _, checked = libs
    rng = np.random.default_rng(3)
    page, hkv = 16, 2
    pages = 320
    kc, vc = (torch.randint(0, 256, (pages, hkv, page, dim // sub), device="cuda", dtype=torch.uint8) for _ in range(2))
    kcb, vcb = (torch.randn((hkv, 256, sub), device="cuda").to(dtype) for _ in range(2))
    batches = [([69, 88, 54, 9, 118, 81, 113], [5000, 5000, 5, 5000, 100, 100], 95)]
    for _ in range(12):
        requests, tokens = int(rng.integers(2, 9)), int(rng.integers(20, 200))
        batches.append((rng.integers(0, tokens + 30, requests + 1).tolist(),
                        rng.choice([5, 100, 5000], requests).tolist(), tokens))
    for cu, lens, tokens in batches:
        table = torch.randint(0, pages, (len(lens), 313), device="cuda", dtype=torch.int32)
        q = torch.randn((tokens, hq, dim), device="cuda").to(dtype)
        args = (q, i32(cu), i32(lens), table, kc, vc, kcb, vcb)
        with using(bind, checked):
            bind.vq_kernel_status(clear=True)
            for max_new in (0, 1, 200):
                out, lse = vq.vq_paged_attention(*args, max_new=max_new, return_lse=True)
                assert out.shape == q.shape and lse.shape == (tokens, hq)
            assert bind.vq_kernel_status() == 0
