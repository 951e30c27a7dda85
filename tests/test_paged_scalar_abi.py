"""Refusals of the calls on the paged cache in 4 bits, on the host: nothing here launches."""
import pytest
import torch

from test_paged_abi import P, call, lib  # noqa: F401  (a fixture)

OK, INVALID, UNSUPPORTED = 0, 1, 2

APPEND = dict(k=P, v=P, k_stride=256, v_stride=256, slots=P, tokens=4, heads=2, dim=128, n_c=16, kcent=P, vcent=P,
              signs=P, kc=P, vc=P, ks=P, vs=P, pages=4, page=16, stride=2048, sstride=32, dtype=0)
ATTEND = dict(q=P, q_stride=512, cu=P, lens=P, slots=P, requests=2, tokens=3, max_new=2, table=P, blocks=8, kc=P, vc=P, ks=P,
              vs=P, pages=4, page=16, stride=2048, sstride=32, kcent=P, vcent=P, hq=4, hkv=2, dim=128, n_c=16, window=0,
              scale=0.0, dtype=0, out=P, lse=P, ws=P, ws_bytes=0)


@pytest.mark.parametrize("change, want", [
    (dict(dtype=7), INVALID), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID),
    (dict(dim=127), INVALID), (dict(dim=514), UNSUPPORTED), (dict(dim=96), UNSUPPORTED), (dict(heads=1025), UNSUPPORTED),
    (dict(n_c=0), UNSUPPORTED), (dict(n_c=17), UNSUPPORTED), (dict(page=12), INVALID), (dict(page=0), INVALID),
    (dict(page=2048), UNSUPPORTED), (dict(stride=2047), INVALID), (dict(sstride=31), INVALID), (dict(k_stride=255), INVALID),
    (dict(v_stride=255), INVALID), (dict(pages=-1), INVALID), (dict(tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(k_stride=1 << 40), UNSUPPORTED), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID),
    (dict(kcent=0), INVALID), (dict(vcent=0), INVALID), (dict(kc=0), INVALID), (dict(vc=0), INVALID), (dict(ks=0), INVALID),
    (dict(vs=0), INVALID), (dict(k=P + 1), INVALID), (dict(slots=P + 4), INVALID), (dict(signs=P + 2), INVALID),
    (dict(vs=P + 1), INVALID), (dict(kcent=P + 2), INVALID), (dict(pages=1 << 40, stride=1 << 40), INVALID),
    (dict(pages=1 << 30, sstride=1 << 40), INVALID), (dict(tokens=0), OK), (dict(pages=0, kc=0, vc=0, ks=0, vs=0), OK)])
def test_append_refusals(lib, change, want):  # noqa: F811
    assert call(lib.vq_paged_scalar_append, APPEND, **change) == want


@pytest.mark.parametrize("change, want", [
    (dict(dtype=-1), INVALID), (dict(requests=-1), INVALID), (dict(tokens=-1), INVALID), (dict(max_new=-1), INVALID),
    (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=5), INVALID), (dict(hq=2048), UNSUPPORTED),
    (dict(dim=0), INVALID), (dict(dim=3), INVALID), (dict(dim=1024), UNSUPPORTED), (dict(n_c=0), UNSUPPORTED),
    (dict(n_c=17), UNSUPPORTED), (dict(page=48), INVALID), (dict(page=2048), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(stride=100), INVALID), (dict(sstride=31), INVALID), (dict(q_stride=511), INVALID),
    (dict(q_stride=1 << 40), UNSUPPORTED), (dict(pages=-1), INVALID), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(blocks=-1), INVALID), (dict(blocks=1 << 27), UNSUPPORTED), (dict(requests=1 << 25), UNSUPPORTED),
    (dict(tokens=(1 << 30) + 1), UNSUPPORTED), (dict(q=0), INVALID), (dict(cu=0), INVALID), (dict(lens=0), INVALID),
    (dict(table=0), INVALID), (dict(kc=0), INVALID), (dict(vc=0), INVALID), (dict(ks=0), INVALID), (dict(vs=0), INVALID),
    (dict(kcent=0), INVALID), (dict(vcent=0), INVALID), (dict(out=0), INVALID), (dict(ws=0), INVALID), (dict(q=P + 1), INVALID),
    (dict(lse=P + 2), INVALID), (dict(cu=P + 2), INVALID), (dict(ws=P + 8), INVALID), (dict(slots=P + 4), INVALID),
    (dict(vcent=P + 1), INVALID), (dict(ks=P + 1), INVALID), (dict(), INVALID), (dict(tokens=0), OK)])
def test_attention_refusals(lib, change, want):  # noqa: F811
    """(The call without a change has a workspace of no bytes.)"""
    assert call(lib.vq_paged_scalar_attention, ATTEND, **change) == want


def test_workspace_bytes(lib):  # noqa: F811
    fn = lib.vq_paged_scalar_attention_workspace_bytes
    assert fn(2, 3, 1, 4, 2, 128, 16) > 0
    assert fn(2, 1000000, 0, 4, 2, 128, 16) < 1 << 30
    for bad in ((-1, 3, 1, 4, 2, 128, 16), (2, 3, 1, 5, 2, 128, 16), (2, 3, 1, 4, 2, 127, 16), (2, 3, -1, 4, 2, 128, 16),
                (2, 3, 1, 4, 2, 128, 17)):
        assert fn(*bad) == 0


def test_binding_refusals():
    """The wrappers check types and shapes before any pointer is taken."""
    import product_vq_kv_gb300 as vq

    x = torch.zeros((4, 2, 128), dtype=torch.float16)
    codes, scales = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2, 16), dtype=torch.float16)
    cents, slots = torch.zeros(16), torch.zeros(4, dtype=torch.int64)
    i = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros((4, 8), dtype=torch.int32)
    with pytest.raises(TypeError, match="dtype"):
        vq.vq_paged_scalar_append(x.double(), x.double(), slots, cents, cents, codes, codes, scales, scales)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_scalar_append(x, x, slots, cents, cents, codes, codes, scales, scales)
    with pytest.raises(TypeError, match="Tensor"):
        vq.vq_paged_scalar_attention(None, i[:2], i[:1], table[:1], codes, codes, scales, scales, cents, cents)
    with pytest.raises(ValueError, match="CUDA"):
        vq.vq_paged_scalar_attention(x, i[:2], i[:1], table[:1], codes, codes, scales, scales, cents, cents)


@pytest.mark.parametrize("name, change", [
    ("codes must be uint8", dict(kc=lambda t: t.int())), ("scales must be", dict(vs=lambda t: t.float())),
    ("centroids must be float32", dict(kcent=lambda t: t.half())), ("one shape", dict(vc=lambda t: t[:2])),
    ("shape of the codes", dict(ks=lambda t: t[..., :8], vs=lambda t: t[..., :8])), ("one shape", dict(vcent=lambda t: t[:8])),
    ("expected codes", dict(kc=lambda t: t[0])), ("must be a torch.Tensor", dict(vs=lambda t: 3))])
def test_page_tensors(name, change):
    """The checks of pages and centroids, one at a time (a stand-in for the device)."""
    import product_vq_kv_gb300._binding as bind

    args = dict(kc=torch.zeros((3, 2, 16, 64), dtype=torch.uint8), vc=torch.zeros((3, 2, 16, 64), dtype=torch.uint8),
                ks=torch.zeros((3, 2, 16), dtype=torch.float16), vs=torch.zeros((3, 2, 16), dtype=torch.float16),
                kcent=torch.zeros(16), vcent=torch.zeros(16))
    for k, f in change.items():
        args[k] = f(args[k])
    with pytest.raises((TypeError, ValueError), match=name):
        bind._scalar_page_tensors(*args.values(), torch.float16, torch.device("cpu"))
