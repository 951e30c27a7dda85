"""The paged attention's work split, on the host: the code that its kernels walk their
work with (``tests/harness/host/paged_walk.cu``), against what every block may do."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from product_vq_kv_gb300 import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "harness", "host", "paged_walk.cu")
LIB = os.path.join(HERE, "harness", "_build", "libpaged_walk.so")


@pytest.fixture(scope="module")
def walk():
    if not os.path.exists(LIB) or any(os.path.getmtime(p) > os.path.getmtime(LIB) for p in [SRC] + lib_build.DEPENDS):
        os.makedirs(os.path.dirname(LIB), exist_ok=True)
        tmp = f"{LIB}.{os.getpid()}"
        subprocess.run([lib_build.nvcc(), *lib_build.ARCH, "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I",
                        lib_build.CSRC, "-I", os.path.join(lib_build.ROOT, "include"), "-o", tmp, SRC], check=True)
        os.replace(tmp, LIB)
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    fn = ctypes.CDLL(LIB).paged_walk
    fn.restype = i64
    ptr = np.ctypeslib.ndpointer(np.int32, flags="C")
    out = np.ctypeslib.ndpointer(np.int64, flags="C")
    fn.argtypes = [ptr, ptr, i64, i64, i64, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, i64, i64, out, out,
                   ctypes.POINTER(i64)]

    def run(cu, lens, tokens, max_blocks=1000, page_shift=4, window=0, hkv=2, group=4, gc=4, tile=2, item_cost=4,
            no_split=0, cls=0, cls_tokens=6, threads=256, grid=304):
        room = 200000
        segments, notes = np.zeros((room, 10), np.int64), np.zeros((grid, 7), np.int64)
        n = i64()
        count = fn(np.array(cu, np.int32), np.array(lens + [0], np.int32), len(lens), tokens, max_blocks, page_shift,
                   window, hkv, group, gc, tile, item_cost, no_split, cls, cls_tokens, threads, grid, room, segments,
                   notes, ctypes.byref(n))
        assert count >= 0
        return segments[:count], notes[:n.value]

    return run


def random_batch(rng):
    requests = int(rng.integers(0, 12))
    new = rng.integers(0, 60, requests) * (rng.random(requests) < 0.8)
    held = np.exp(rng.uniform(0, 9, requests)).astype(int)
    lens = [int(n + h) if rng.random() < 0.9 else int(rng.integers(-3, 9)) for n, h in zip(new, held)]
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    return cu, lens, cu[-1] + int(rng.integers(0, 9))


SHAPES = [  # threads, grid, item cost, tile
    dict(threads=256, grid=304, item_cost=4, tile=2), dict(threads=512, grid=152, item_cost=0, tile=64),
    dict(threads=128, grid=608, item_cost=0, tile=1), dict(threads=256, grid=152, item_cost=4, tile=8, group=1, gc=1)]


@pytest.mark.parametrize("shape", SHAPES)
def test_every_unit_of_every_row_is_done_once(walk, shape):
    rng = np.random.default_rng(1)
    for _ in range(60):
        cu, lens, tokens = random_batch(rng)
        window = int(rng.choice([0, 0, 300]))
        kw = {**dict(hkv=2, group=4, gc=4), **shape}
        segments, notes = walk(cu, lens, tokens, window=window, **kw)
        done = {}
        for b, hx, tok0, ntok, pos0, k0, units, whole, slot, r in segments.tolist():
            for t in range(tok0, tok0 + ntok):
                at = done.setdefault((hx, t), {"request": r, "units": []})
                assert at["request"] == r
                at["units"] += range(k0, k0 + 128 * units, 128)
        heads = kw["hkv"] * -(-kw["group"] // kw["gc"])
        assert set(done) == {(hx, t) for hx in range(heads) for t in range(tokens)}
        for (hx, t), at in done.items():
            r = at["request"]
            assert (r == len(lens)) == (t >= cu[-1]) and (r == len(lens) or cu[r] <= t < cu[r + 1])
            units = sorted(at["units"])
            assert units == list(range(units[0], units[-1] + 1, 128))  # each once, without a gap
            if r < len(lens) and lens[r] > 0:
                p = lens[r] - (cu[r + 1] - t)
                low = max(0, p - window + 1) if window else 0
                assert p < low or (units[0] <= low and units[-1] + 128 > p)
        # the parts of a split item: the slots its note names, and no other
        slots = {}
        for b, hx, tok0, ntok, pos0, k0, units, whole, slot, r in segments.tolist():
            if not whole:
                slots.setdefault((tok0, hx), []).append(slot)
        named = {}
        for b, tok0, head0, gc, rows, first, last in notes.tolist():
            assert b == first and 0 <= first < last < shape["grid"]
            hx = head0 // kw["group"] * -(-kw["group"] // kw["gc"]) + head0 % kw["group"] // kw["gc"]
            named[(tok0, hx)] = [2 * first + 1] + [2 * c for c in range(first + 1, last + 1)]
        assert named == slots


@pytest.mark.parametrize("shape", SHAPES)
def test_descending_offsets_name_no_slot_past_the_workspace(walk, shape):
    """Offsets that descend lay the items out differently for the walk and the plan: the
    walk ends, its tokens and the slots of its notes stay inside the buffers."""
    rng = np.random.default_rng(2)
    batches = [([69, 88, 54, 9, 118, 81, 113], [5000, 5000, 5, 5000, 100, 100], 95)]
    for _ in range(150):
        requests = int(rng.integers(2, 9))
        tokens = int(rng.integers(20, 200))
        batches.append((rng.integers(0, tokens + 30, requests + 1).tolist(),
                        rng.choice([5, 100, 5000], requests).tolist(), tokens))
    for cu, lens, tokens in batches:
        for tile in (shape["tile"], 4):
            segments, notes = walk(cu, lens, tokens, **{**dict(hkv=2, group=4, gc=4), **shape, "tile": tile})
            if len(segments):
                assert (segments[:, 2] >= 0).all() and (segments[:, 2] + segments[:, 3] <= tokens).all()
                assert (segments[:, 8] < 2 * shape["grid"]).all()
            for b, tok0, head0, gc, rows, first, last in notes.tolist():
                assert 0 <= first < shape["grid"] and last < shape["grid"]
                assert 0 < rows <= tile * gc and tok0 + -(-rows // gc) <= tokens
