"""The calls on shared pages and on the cache in 4 bits over a CUDA runtime without a
device: what a failed launch leaves behind, and the limits of shared memory."""
import ctypes

import pytest

from test_host_calls import CUDA, OK, P, lib  # noqa: F401  (a fixture)


def fork(lib, seats=4, pages=10):  # noqa: F811
    return lib.vq_paged_fork(P, P, None, seats, P, 8, 16, P, P, pages, P, P + (1 << 30), P, P, P, 1 << 30, None)


def compact(lib, requests=4, pages=10):  # noqa: F811
    return lib.vq_paged_compact(P, requests, P, 8, 16, P, P, pages, P, P, P, P, P, P, 1 << 30, None)


def copy(lib, n=3):  # noqa: F811
    from product_vq_kv_gb300._binding import VqPagePool

    array = (VqPagePool * 2)(VqPagePool(P, 64, 64, 0, 1), VqPagePool(P, 77, 70, 7700, 3))
    return lib.vq_paged_copy(P, n, ctypes.addressof(array), 2, 10, None)


def append(lib, dim=128, n_c=16, dtype=0, signs=P):  # noqa: F811
    return lib.vq_paged_scalar_append(P, P, 2 * dim, 2 * dim, P, 4, 2, dim, n_c, P, P, signs, P, P, P, P, 4, 16, 16 * dim, 32,
                                      dtype, None)


def attend(lib, requests=2, tokens=300, max_new=200, dtype=0, dim=128, page=16):  # noqa: F811
    ws = lib.vq_paged_scalar_attention_workspace_bytes(requests, tokens, max_new, 4, 2, dim, page)
    return lib.vq_paged_scalar_attention(P, 4 * dim, P, P, None, requests, tokens, max_new, P, 80, P, P, P, P, 4, page,
                                         page * dim, 2 * page, P, P, 4, 2, dim, 16, 0, 0.0, dtype, P, P, P, ws, None)


CALLS = {
    "fork": fork, "fork of many": lambda lib: fork(lib, 8192, 1 << 20), "compact": compact,
    "compact, many pages": lambda lib: compact(lib, 8192, 1 << 20), "compact without a table": lambda lib: compact(lib, 0),
    "copy": copy, "append": append, "append, wide": lambda lib: append(lib, 512, dtype=2),
    "append, few centroids": lambda lib: append(lib, 64, 5, 1, None), "attention of chunks": attend,
    "attention of few rows": lambda lib: attend(lib, 2, 2, 1), "attention, dim 256": lambda lib: attend(lib, dim=256),
    "attention, dim 64": lambda lib: attend(lib, dim=64, dtype=1), "attention, general": lambda lib: attend(lib, dtype=2),
    "attention, small pages": lambda lib: attend(lib, page=8),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_reported_once(lib, name):  # noqa: F811
    """The launch that fails is that call's error and no later one's."""
    call = CALLS[name]
    before = lib.fake_launches()
    assert call(lib) == OK and lib.fake_launches() > before
    for n in range(1, lib.fake_launches() - before + 1):
        lib.fake_fail_in(n)
        assert call(lib) == CUDA
        assert lib.fake_last_error() == 0
    assert call(lib) == OK


def test_a_kernel_has_one_limit_of_shared_memory(lib):  # noqa: F811
    for seats in (1, 5000, 8192):
        assert fork(lib, seats) == compact(lib, seats) == OK
    for dim in (64, 128, 256):
        for dtype in (0, 1, 2):
            for n in (1, 200):
                assert attend(lib, 2, 2 * n, n, dtype, dim) == append(lib, dim, 16, dtype) == OK
    assert lib.fake_most_limits() <= 1
