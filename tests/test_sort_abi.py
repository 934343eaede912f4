"""CPU checks of the entry points of the moves between token and expert order: what they
refuse, before any launch."""

import pytest

FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks first
FAR = 1 << 34   # arrays that do not overlap those at FAKE


@pytest.fixture(scope="module")
def L():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    pkg._lib.load()
    return pkg._lib


def test_sort_refusals(L):
    def f(x=FAKE, sc=None, idx=2 * FAKE, T=4, k=2, E=8, rb=64, sb=0, off=FAR, perm=FAR + FAKE, inv=FAR + 2 * FAKE,
          rows=FAR + 3 * FAKE, rsc=None):
        return L.moe_sort_tokens(x, sc, idx, T, k, E, rb, sb, off, perm, inv, rows, rsc, None)
    for kw in (dict(T=0), dict(k=0), dict(k=9), dict(E=0), dict(E=257), dict(k=33, E=256), dict(T=1 << 23, k=4), dict(rb=0),
               dict(rb=24), dict(rb=65552), dict(sb=-1), dict(sb=4097)):
        assert f(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=None), dict(idx=None), dict(off=None), dict(perm=None), dict(inv=None), dict(rows=None), dict(x=FAKE + 8),
               dict(idx=2 * FAKE + 2), dict(rows=FAR + 8), dict(inv=FAR + 2 * FAKE + 2), dict(sc=3 * FAKE), dict(sb=4), dict(sb=4, sc=3 * FAKE),
               dict(sb=4, rsc=FAR + 4 * FAKE), dict(rsc=FAR + 4 * FAKE), dict(rows=FAKE), dict(rows=FAKE + 240), dict(perm=FAKE),
               dict(inv=2 * FAKE), dict(rows=FAKE - 496), dict(sb=4, sc=3 * FAKE, rsc=3 * FAKE)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_unsort_refusals(L):
    def f(y=FAKE, inv=2 * FAKE, w=3 * FAKE, T=4, k=2, H=64, dt=0, out=FAR):
        return L.moe_unsort_tokens(y, inv, w, T, k, H, dt, out, None)

    def b(d=FAKE, y=2 * FAKE, inv=3 * FAKE, w=4 * FAKE, T=4, k=2, H=64, dt=0, dy=FAR, dw=FAR + FAKE):
        return L.moe_unsort_tokens_backward(d, y, inv, w, T, k, H, dt, dy, dw, None)
    for call in (f, b):
        for kw in (dict(T=0), dict(k=0), dict(k=33), dict(T=1 << 22, k=5), dict(H=0), dict(H=12), dict(H=32776),
                   dict(H=16392, dt=2)):
            assert call(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
        for kw in (dict(inv=None), dict(y=FAKE + 8), dict(inv=3 * FAKE + 2), dict(w=4 * FAKE + 1), dict(dt=3), dict(dt=-1)):
            assert call(**kw) == L.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(y=None), dict(out=None), dict(out=FAR + 8), dict(out=FAKE), dict(out=FAKE + 1008), dict(out=2 * FAKE),
               dict(out=3 * FAKE)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(d=None), dict(y=None), dict(dy=None, dw=None), dict(dy=FAR + 8), dict(dw=FAR + 2), dict(dy=FAKE),
               dict(dy=2 * FAKE), dict(dw=4 * FAKE), dict(dw=3 * FAKE)):
        assert b(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_route_backward_refusals(L):
    def f(dw=FAKE, l=2 * FAKE, idx=3 * FAKE, w=4 * FAKE, T=4, k=2, E=8, gating=0, out=FAR):
        return L.moe_route_backward(dw, l, idx, w, T, k, E, gating, out, None)
    for kw in (dict(T=0), dict(k=0), dict(k=9), dict(E=257), dict(k=33, E=256), dict(T=1 << 24, k=2)):
        assert f(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(dw=None), dict(l=None), dict(idx=None), dict(w=None), dict(out=None), dict(out=FAR + 2), dict(w=4 * FAKE + 1),
               dict(gating=1), dict(gating=6), dict(gating=8), dict(out=2 * FAKE), dict(out=FAKE), dict(out=4 * FAKE)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_no_gradient_is_cut_in_silence(L):
    """Tensors that require grad are refused while autograd records, and outside of that are
    as any other (these, on the CPU, are refused for not being on a GPU)."""
    import torch
    import mxfp4_expert_layer_gb300 as pkg
    idx = torch.zeros(4, 2, dtype=torch.int32)

    def t(*s, grad=False):
        return torch.zeros(*s, requires_grad=grad)
    calls = {
        "x": lambda g: pkg.sort_tokens(t(4, 64, grad=g), idx, 8),
        "scales": lambda g: pkg.sort_tokens(t(4, 64), idx, 8, scales=t(4, 2, grad=g)),
        "d_rows": lambda g: pkg.sort_tokens_backward(t(8, 64, grad=g), idx),
        "y": lambda g: pkg.unsort_tokens(t(8, 64, grad=g), idx, t(4, 2)),
        "topk_w": lambda g: pkg.unsort_tokens(t(8, 64), idx, t(4, 2, grad=g)),
        "d_out": lambda g: pkg.unsort_tokens_backward(t(4, 64, grad=g), t(8, 64), idx, t(4, 2)),
        "d_topk_w": lambda g: pkg.route_backward(t(4, 2, grad=g), t(4, 8), idx, t(4, 2)),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"{name} requires grad.*explicit calls"):
            call(True)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(True)
        with pytest.raises(ValueError, match="CUDA"):
            call(False)
    with pytest.raises(TypeError):
        pkg.sort_tokens(t(4, 64), 3, 8)
    with pytest.raises(ValueError, match="bf16 or f16"):
        pkg.unsort_tokens(t(8, 64).double(), idx, t(4, 2))
