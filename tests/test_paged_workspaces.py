"""Workspaces of exactly the bytes that are asked for, and of one byte less, over a CUDA
runtime without a device."""
import pytest

from test_host_calls import OK, P, lib  # noqa: F401  (a fixture)

INVALID = 1


def fork(lib, pages, ws):  # noqa: F811
    return lib.vq_paged_fork(P, P, None, 4, P, 8, 16, P, P, pages, P, P + (1 << 30), P, P, P, ws, None)


def compact(lib, pages, ws):  # noqa: F811
    return lib.vq_paged_compact(P, 4, P, 8, 16, P, P, pages, P, P, P, P, P, P, ws, None)


@pytest.mark.parametrize("pages", [1, 31, 33, 256, 257, 100000])
@pytest.mark.parametrize("name", ["fork", "compact"])
def test_workspaces_of_shared_pages(lib, name, pages):  # noqa: F811
    call = {"fork": fork, "compact": compact}[name]
    need = getattr(lib, f"vq_paged_{name}_workspace_bytes")(pages)
    # flags of one byte twice and a word a page; a bit a page
    assert need >= (6 * pages if name == "fork" else (pages + 31) // 32 * 4)
    assert call(lib, pages, need) == OK
    assert call(lib, pages, need - 1) == INVALID


# requests, tokens, max_new, query heads, KV heads, head size, page, dtype: what the few-row
# kernel takes, the chunk kernel, both, and the general kernel
ATTENTION = {
    "few rows": (32, 32, 1, 8, 2, 128, 16, 0), "items of 4 rows": (5, 5, 1, 2, 2, 64, 32, 1), "drafts": (8, 40, 5, 12, 4, 256, 64, 1),
    "chunk": (1, 700, 700, 8, 2, 128, 16, 0), "both": (16, 2063, 2048, 32, 8, 128, 16, 1), "both, unknown": (3, 900, 0, 4, 1, 256, 16, 0),
    "fp32": (3, 900, 0, 4, 1, 128, 16, 2), "head size 96": (3, 30, 10, 4, 2, 96, 16, 0), "small pages": (3, 30, 10, 4, 2, 128, 8, 1),
}


@pytest.mark.parametrize("name", ATTENTION)
def test_workspaces_of_attention(lib, name):  # noqa: F811
    requests, tokens, most, hq, hkv, dim, page, dtype = ATTENTION[name]
    need = lib.vq_paged_scalar_attention_workspace_bytes(requests, tokens, most, hq, hkv, dim, page)

    def call(ws):
        return lib.vq_paged_scalar_attention(P, hq * dim, P, P, None, requests, tokens, most, P, 80, P, P, P, P, 4, page,
                                             hkv * page * dim // 2, hkv * page, P, P, hq, hkv, dim, 16, 0, 0.0, dtype, P, P, P,
                                             ws, None)

    assert need > 0 and call(need) == OK
    assert call(need - 1) == INVALID
