"""Refusals of the calls on shared pages, on the host: nothing here launches."""
import ctypes

import pytest
import torch

from test_paged_abi import P, call, lib  # noqa: F401  (a fixture)

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAR = P + (1 << 30)

FORK = dict(lens=P, parents=P, keep=P, seats=4, table=P, blocks=8, page=16, free=P, count=P, pages=10, lens_out=P,
            table_out=FAR, count_out=P, copies=P, ws=P, ws_bytes=1 << 20)
COMPACT = dict(lens=P, requests=4, table=P, blocks=8, page=16, free=P, count=P, pages=10, table_out=P, free_out=P,
               count_out=P, moves=P, map=P, ws=P, ws_bytes=1 << 20)


@pytest.mark.parametrize("change, want", [
    (dict(page=0), INVALID), (dict(page=24), INVALID), (dict(page=2048), UNSUPPORTED), (dict(seats=-1), INVALID),
    (dict(seats=8193), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(blocks=-1), INVALID), (dict(blocks=1 << 27), UNSUPPORTED), (dict(lens=0), INVALID), (dict(parents=0), INVALID),
    (dict(table=0), INVALID), (dict(table_out=0), INVALID), (dict(free=0), INVALID), (dict(count=0), INVALID),
    (dict(lens_out=0), INVALID), (dict(count_out=0), INVALID), (dict(copies=0), INVALID), (dict(ws=0), INVALID),
    (dict(ws=P + 8), INVALID), (dict(ws_bytes=100), INVALID), (dict(lens=P + 2), INVALID), (dict(keep=P + 1), INVALID),
    (dict(copies=P + 2), INVALID), (dict(table_out=P), INVALID), (dict(table_out=P + 4 * 31), INVALID),
    (dict(table=FAR + 4 * 31), INVALID)])
def test_fork_refusals(lib, change, want):  # noqa: F811
    args = {**FORK, **change}
    assert lib.vq_paged_fork(*[v or None if k in ("lens", "parents", "table", "table_out", "free", "count", "lens_out",
                                                  "count_out", "copies", "ws") else v for k, v in args.items()], None) == want


@pytest.mark.parametrize("change, want", [
    (dict(page=3), INVALID), (dict(page=4096), UNSUPPORTED), (dict(requests=-1), INVALID),
    (dict(requests=8193), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(blocks=-2), INVALID), (dict(lens=0), INVALID),
    (dict(table=0), INVALID), (dict(table_out=0), INVALID), (dict(free=0), INVALID), (dict(free_out=0), INVALID),
    (dict(count=0), INVALID), (dict(count_out=0), INVALID), (dict(moves=0), INVALID), (dict(map=0), INVALID),
    (dict(map=P + 3), INVALID), (dict(moves=P + 1), INVALID), (dict(ws=0), INVALID), (dict(ws=P + 8), INVALID),
    (dict(pages=1 << 30), INVALID)])
def test_compact_refusals(lib, change, want):  # noqa: F811
    assert call(lib.vq_paged_compact, COMPACT, **change) == want


POOL = dict(base=P, page_stride=64, page_bytes=64, layer_stride=0, layers=1)


@pytest.mark.parametrize("change, pool, want", [
    (dict(n=-1), {}, INVALID), (dict(count=-1), {}, INVALID), (dict(count=9), {}, UNSUPPORTED), (dict(pages=-1), {}, INVALID),
    (dict(pages=1 << 31), {}, UNSUPPORTED), (dict(n=(1 << 30) + 1), {}, UNSUPPORTED), (dict(pairs=None), {}, INVALID),
    (dict(pairs=P + 2), {}, INVALID), ({}, dict(base=None), INVALID), ({}, dict(page_stride=63), INVALID),
    ({}, dict(layers=-1), INVALID), ({}, dict(page_bytes=-1), INVALID), ({}, dict(page_stride=1 << 62), INVALID),
    ({}, dict(layers=2, layer_stride=100), INVALID), ({}, dict(layers=2, layer_stride=-640), INVALID),
    ({}, dict(layers=3, layer_stride=64, page_stride=190), INVALID), ({}, dict(layers=2, layer_stride=1 << 62), INVALID),
    ({}, dict(page_bytes=1 << 50, page_stride=1 << 50), UNSUPPORTED),
    (dict(n=0), {}, OK), (dict(pages=0), {}, OK), (dict(count=0), {}, OK), ({}, dict(layers=0), OK), ({}, dict(page_bytes=0), OK)])
def test_copy_refusals(lib, change, pool, want):  # noqa: F811
    from product_vq_kv_gb300._binding import VqPagePool

    args = {**dict(pairs=P, n=3, count=1, pages=10), **change}
    array = (VqPagePool * 1)(VqPagePool(**{**POOL, **pool}))
    assert lib.vq_paged_copy(args["pairs"], args["n"], ctypes.addressof(array), args["count"], args["pages"], None) == want


def test_workspace_bytes(lib):  # noqa: F811
    assert lib.vq_paged_fork_workspace_bytes(0) == 0
    assert lib.vq_paged_fork_workspace_bytes(1000) >= 6000
    assert lib.vq_paged_compact_workspace_bytes(0) == lib.vq_paged_compact_workspace_bytes(-1) == 0
    assert lib.vq_paged_compact_workspace_bytes(33) >= 8
    assert lib.vq_paged_fork_workspace_bytes(-1) == lib.vq_paged_fork_workspace_bytes(1 << 31) == 0


def test_binding_refusals():
    import product_vq_kv_gb300 as vq

    i, one = torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros((4, 8), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_fork(i, i, table, 16, i, one)
    with pytest.raises(TypeError):
        vq.vq_paged_fork(i.long(), i, table, 16, i, one)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_compact(i, table, 16, i, one)
    with pytest.raises(TypeError, match="Tensor"):
        vq.vq_paged_compact(None, table, 16, i, one)
    with pytest.raises(ValueError, match="shape"):
        vq.vq_paged_copy(i, [table])
