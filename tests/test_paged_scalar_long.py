"""The paged cache in 4 bits at length and at its edges: caches of thousands of tokens against
the definition in 64 bits on the device, pools past 2^32 bytes, waits that give up, calls
side by side, captured calls."""
import ctypes
import math

import pytest
import torch

import scalar_reference as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
CENTS = [-2.73, -2.07, -1.62, -1.26, -0.94, -0.66, -0.39, -0.13, 0.13, 0.39, 0.66, 0.94, 1.26, 1.62, 2.07, 2.73]


@pytest.fixture(scope="module")
def vq():
    from product_vq_kv_gb300.build import build

    build()
    import product_vq_kv_gb300 as m

    m.load_library()
    return m


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def make(seed, dim, dtype, hq, hkv, page, lens, news, spread=0.5, late=False, holes=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-max(lens) // page) + 1
    pages = sum(-(-n // page) for n in lens) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.randint(0, 256, (pages, hkv, page, dim // 2), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.exp(spread * torch.randn((pages, hkv, page), generator=gen, device="cuda")) for _ in range(2))
    at = 0
    for r, n in enumerate(lens):
        held = -(-n // page)
        table[r, :held] = order[at:at + held]
        at += held
        if late:  # keys grow along the sequence: the maxima come late, step by step; values shrink
            grow = torch.linspace(-4, 2, held * page, device="cuda").reshape(held, 1, page)
            ks[table[r, :held].long()] *= torch.exp(grow)
            vs[table[r, :held].long()] *= torch.exp(-grow)
        if holes:
            table[r, held // 3] = -1
            table[r, held // 2:held // 2 + 5] = pages + 9
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], hq, dim), generator=gen, device="cuda").to(dtype)
    cents = torch.tensor(CENTS, device="cuda")
    return dict(q=q, cu=cu, lens=lens, table=table, kc=kc, vc=vc, ks=ks.to(dtype), vs=vs.to(dtype), cents=cents, dtype=dtype)


def run(vq, c, window=0, known=True, **kw):
    most = max(b - a for a, b in zip(c["cu"], c["cu"][1:]))
    return vq.vq_paged_scalar_attention(c["q"], i32(c["cu"]), i32(c["lens"]), c["table"], c["kc"], c["vc"], c["ks"], c["vs"],
                                        c["cents"], c["cents"], max_new=most if known else 0, window=window, return_lse=True, **kw)


def check(c, out, lse, window=0, chunk=False):
    """Against the definition in 64 bits, with the bounds of scalar_reference.attention; the
    few-row kernel (not `chunk`) rounds its weights to two pieces."""
    u = 2.0 ** -24
    dtype = c["dtype"]
    eps, tiny = ref.HALF_EPS[dtype], ref.HALF_STEP[dtype]
    h, step = (eps, tiny) if chunk else (eps ** 2, 2.0 ** -31 if dtype is F16 else tiny)
    tokens, hq, dim = c["q"].shape
    pages, hkv, page, _ = c["kc"].shape
    scale, cents = 1 / math.sqrt(dim), c["cents"].to(dtype).double()
    kappa = scale / math.log(2)
    for r, length in enumerate(c["lens"]):
        a, b = c["cu"][r], c["cu"][r + 1]
        t = torch.arange(length, device="cuda")
        entry = c["table"][r].long()[t // page]
        ok = (entry >= 0) & (entry < pages)
        entry = entry.clamp(0, pages - 1)
        pos = length - (b - a) + torch.arange(b - a, device="cuda")
        seen = ok[None, :] & (t[None, :] <= pos[:, None])
        if window:
            seen &= t[None, :] > pos[:, None] - window
        some = seen.any(1)
        assert (out[a:b][~some] == 0).all() and torch.isneginf(lse[a:b][~some]).all()
        if not some.any():
            continue
        n = seen.sum(1, keepdim=True).double()
        for hd in range(hkv):
            rows = []
            for codes, scales in ((c["kc"], c["ks"]), (c["vc"], c["vs"])):
                byte = codes[entry, hd, t % page].long()
                x = torch.stack([cents[byte & 15], cents[byte >> 4]], -1).reshape(length, dim)
                rows.append(x * scales[entry, hd, t % page].double()[:, None])
            keys, values = rows
            for g in range(hq // hkv):
                head = hd * (hq // hkv) + g
                q = c["q"][a:b, head].double()
                s = (scale * (q @ keys.t())).masked_fill(~seen, -math.inf)
                top = s.amax(1, keepdim=True)
                w = torch.exp(s - top)
                total = w.sum(1, keepdim=True)
                want = w @ values / total
                want_lse = (top + torch.log(total))[:, 0]
                d = (dim + 6) * u * kappa * (q.abs() @ keys.abs().t())
                e = math.log(2) * (d + 2 * u * ((top - s) / math.log(2) + 40)) + 2.0 ** -21 + h
                e = e.masked_fill(~seen, 0)
                big = values[seen.any(0)].abs().max()
                tol = 1.1 * (big * (2 * (w * e).sum(1, keepdim=True) / total + 2 * n * step + 4 * (n + 200) * u) + tiny)
                tol_lse = 1.1 * (e.amax(1) + n[:, 0] * step + (n[:, 0] + 200) * u) + 4 * u * want_lse.abs()
                off = (out[a:b, head].double() - want).abs() - (tol + eps * (want.abs() + tol) + tiny)
                assert (off[some] <= 0).all(), f"request {r} head {head}: beyond the bound by {off[some].max():.3g}"
                assert ((lse[a:b, head].double() - want_lse).abs() <= tol_lse)[some].all()


SHAPES = [(128, BF16, 32, 8, 16), (128, F16, 16, 4, 64), (64, F16, 32, 8, 16), (64, BF16, 24, 8, 128), (256, F16, 12, 4, 16),
          (256, BF16, 16, 4, 32)]


@pytest.mark.parametrize("dim, dtype, hq, hkv, page", SHAPES)
@pytest.mark.parametrize("kind", ["plain", "window", "late", "holes"])
def test_long_chunks(vq, dim, dtype, hq, hkv, page, kind):
    window = 2600 if kind == "window" else 0
    c = make(dim, dim, dtype, hq, hkv, page, [5000, 3333], [771, 300], late=kind == "late", holes=kind == "holes")
    out, lse = run(vq, c, window, known=kind != "holes")
    assert vq.vq_kernel_status() == 0
    check(c, out, lse, window, chunk=True)


@pytest.mark.parametrize("dim, dtype, hq, hkv, page", SHAPES)
@pytest.mark.parametrize("kind", ["plain", "window", "late", "holes"])
@pytest.mark.parametrize("news", [[1, 1, 1], [2, 1, 3]])
def test_long_decodes(vq, dim, dtype, hq, hkv, page, kind, news):
    window = 7777 if kind == "window" else 0
    c = make(dim + 1, dim, dtype, hq, hkv, page, [20000, 3001, 9999], news, late=kind == "late", holes=kind == "holes")
    out, lse = run(vq, c, window)
    check(c, out, lse, window)


def test_values_of_every_size(vq):
    """Values whose scales span fp16's range: the weights' factor follows them, and a token of
    large values and no weight takes nothing from the others."""
    c = make(5, 128, F16, 8, 2, 16, [3000], [1])
    gen = torch.Generator(device="cuda").manual_seed(6)
    c["vs"] = torch.exp2(torch.randint(-20, 13, c["vs"].shape, generator=gen, device="cuda").float()).half()
    check(c, *run(vq, c))
    c["vs"] = torch.full_like(c["vs"], 2.0 ** -14)
    page, at = c["table"][0, 10].item(), 3  # one token: keys of no size beside the others', values of the largest
    c["ks"].fill_(4.0)
    c["ks"][page, :, at] = 0.0
    c["vs"][page, :, at] = 8192.0
    check(c, *run(vq, c))
    c["vs"].zero_()  # no value at all
    out, lse = run(vq, c)
    assert not out.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dim, dtype, low, high", [(64, F16, -20, 13), (128, F16, -20, 13), (128, BF16, -90, 90), (256, F16, -20, 13),
                                                   (256, BF16, -90, 90)])
def test_values_of_every_size_in_chunks(vq, dim, dtype, low, high):
    """The same for a chunk, whose rows' references follow the scales block by block."""
    c = make(dim + 7, dim, dtype, 8, 2, 16, [3000], [700])
    gen = torch.Generator(device="cuda").manual_seed(6)
    c["vs"] = torch.exp2(torch.randint(low, high, c["vs"].shape, generator=gen, device="cuda").float()).to(dtype)
    check(c, *run(vq, c), chunk=True)
    pages = c["table"][0, :188].long()
    c["vs"][pages] = torch.exp2(torch.linspace(low, high - 1, 188, device="cuda")).to(dtype)[:, None, None]  # growing
    check(c, *run(vq, c), chunk=True)
    c["vs"][pages] = torch.exp2(torch.linspace(high - 1, low, 188, device="cuda")).to(dtype)[:, None, None]
    check(c, *run(vq, c), chunk=True)
    # tokens that the first rows do not see, far larger: their results stay those without them
    c["vs"].fill_(2.0 ** -14)
    want, want_lse = run(vq, c)
    c["vs"][c["table"][0, 186].long()] = 8192.0
    out, lse = run(vq, c)
    assert torch.equal(out[:600], want[:600]) and torch.equal(lse[:600], want_lse[:600])
    c["vs"].zero_()
    out, lse = run(vq, c)
    assert not out.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("new", [1, 90])
def test_past_32_bits(vq, new):
    """Pages past 2^32 bytes of codes: the bits of the same cache in a small pool."""
    hkv, page, dim = 8, 16, 128
    c = make(7, dim, F16, 16, hkv, page, [700], [new])
    want = run(vq, c)
    held, pages = -(-700 // page), 560000
    kc, vc = (torch.empty((pages, hkv, page, dim // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, hkv, page), dtype=F16, device="cuda") for _ in range(2))
    here = c["table"][0, :held].long()
    there = torch.arange(pages - held, pages, device="cuda").flip(0)
    for big, small in ((kc, "kc"), (vc, "vc"), (ks, "ks"), (vs, "vs")):
        big[there] = c[small][here]
    table = c["table"].clone()
    table[0, :held] = there.int()
    got = run(vq, {**c, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and the append
    x = torch.randn((9, hkv, dim), device="cuda").half()
    slots = (pages - 1) * page + torch.arange(9, device="cuda")
    vq.vq_paged_scalar_append(x, x, slots, c["cents"], c["cents"], kc, vc, ks, vs)
    code, scale = ref.encode_rows(x.cpu(), CENTS)
    assert torch.equal(kc[-1, :, :9].transpose(0, 1).cpu(), torch.from_numpy(ref.pack(code)))
    assert torch.equal(vs[-1, :, :9].t().cpu(), scale)


# ------------------------------------------------------------------ side by side


def test_streams_and_graphs(vq):
    """Calls on two streams at once, and two captured graphs replayed in turn and at once:
    each its own workspace, each the bits of a call alone."""
    cases = [make(20, 128, F16, 16, 4, 16, [4000, 300], [1, 1]), make(21, 128, BF16, 16, 4, 16, [2500], [400])]
    alone = [run(vq, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(vq, c, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, a in zip(got, alone):
            assert torch.equal(g[0], a[0]) and torch.equal(g[1], a[1])
    graphs, outs = [], []
    for c, s in zip(cases, streams):
        fixed = (i32(c["cu"]), i32(c["lens"]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(vq.vq_paged_scalar_attention(c["q"], *fixed, c["table"], c["kc"], c["vc"], c["ks"], c["vs"], c["cents"],
                                                     c["cents"], max_new=400, return_lse=True))
        graphs.append((graph, fixed))
    want = [vq.vq_paged_scalar_attention(c["q"], *f, c["table"], c["kc"], c["vc"], c["ks"], c["vs"], c["cents"], c["cents"],
                                         max_new=400, return_lse=True) for c, (_, f) in zip(cases, graphs)]
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_workspace_is_checked(vq):
    c = make(22, 128, F16, 8, 2, 16, [100], [1])
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(vq.VQError):
        run(vq, c, workspace=small)
    need = vq.vq_paged_scalar_attention_workspace_bytes(1, 1, 1, 8, 2, 128, 16)
    out = run(vq, c, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out[0], run(vq, c)[0])


# ------------------------------------------------------------------ waits that give up


@pytest.fixture(scope="module")
def harness(vq):
    import product_vq_kv_gb300._binding as bind
    import tc_harness

    lib, like = tc_harness.load(), bind.load_library()
    lib.polls_scalar_attention.restype = ctypes.c_int32
    lib.polls_scalar_attention.argtypes = like.vq_paged_scalar_attention.argtypes
    return lib


def status(lib):
    bits = ctypes.c_uint32(0)
    assert lib.polls_scalar_status(ctypes.byref(bits), 1) == 0
    return bits.value


@pytest.mark.parametrize("polls, dim, hq, hkv, new, held", [(0, 128, 8, 2, 100, 700), (0, 128, 32, 8, 900, 2000), (1, 128, 12, 4, 300, 1500),
                                                           (1, 128, 32, 8, 900, 2000), (1, 256, 12, 4, 700, 1500)])
def test_waits_that_give_up(vq, harness, polls, dim, hq, hkv, new, held):
    """No row is wrong: each is right or NaN, and the status word tells; the GPU goes on."""
    c = make(30, dim, F16, hq, hkv, 16, [held], [new])
    want, want_lse = run(vq, c)
    out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
    ws = torch.zeros(vq.vq_paged_scalar_attention_workspace_bytes(1, new, new, hq, hkv, dim, 16), dtype=torch.uint8, device="cuda")
    harness.polls_scalar_set(polls)
    status(harness)
    p, pages = torch.Tensor.data_ptr, c["kc"].shape[0]
    cu, lens = i32(c["cu"]), i32(c["lens"])
    assert harness.polls_scalar_attention(
        p(c["q"]), hq * dim, p(cu), p(lens), None, 1, new, new, p(c["table"]), c["table"].shape[1], p(c["kc"]), p(c["vc"]),
        p(c["ks"]), p(c["vs"]), pages, 16, hkv * 8 * dim, hkv * 16, p(c["cents"]), p(c["cents"]), hq, hkv, dim, 16, 0, 0.0, 0,
        p(out), p(lse), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    marked = torch.isnan(out).any(-1)
    assert torch.equal(marked, torch.isnan(out).all(-1)) and torch.equal(marked, torch.isnan(lse))
    assert torch.equal(out[~marked], want[~marked]) and torch.equal(lse[~marked], want_lse[~marked])
    gave_up = bool(status(harness) & vq.VQ_KSTATUS_WAIT_GAVE_UP)
    assert gave_up or not marked.any()
    if polls == 0:
        assert marked.all() and gave_up
    again, _ = run(vq, c)
    assert torch.equal(again, want) and vq.vq_kernel_status() == 0


@pytest.mark.parametrize("dim, dtype, hq, hkv, page", SHAPES)
def test_many_requests(vq, dim, dtype, hq, hkv, page):
    """More requests than a block keeps the lengths of, of one token, of none and of chunks."""
    gen = torch.Generator().manual_seed(dim)
    lens = torch.randint(1, 900, (61,), generator=gen).tolist()
    news = [min(n, (0, 1, 3, 40, 150)[i % 5]) for i, n in enumerate(lens)]
    c = make(dim + 9, dim, dtype, hq, hkv, page, lens, news, holes=True)
    for known in (True, False):
        check(c, *run(vq, c, known=known), chunk=True)
