"""CPU checks of the projections' entry points: sizes, and what they refuse before any launch."""

import pytest

FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks first
FAR = 1 << 36   # arrays that do not overlap those at FAKE


@pytest.fixture(scope="module")
def L():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    pkg._lib.load()
    return pkg._lib


def test_sizes(L):
    for T in (1, 16, 64, 128):
        assert L.moe_linear_workspace_bytes(T, 4096, 2880, 0) == 0  # few tokens and batches: one launch
    assert L.moe_linear_workspace_bytes(4096, 4096, 4096, 1) >= 4096 * 4096 * 2
    for T, K, N in ((0, 64, 64), ((1 << 24) + 1, 64, 64), (4, 60, 64), (4, 64, 60), (4, 0, 64), (4, 64, 0),
                    (4, (1 << 17) + 8, 64), (4, 64, (1 << 20) + 8)):
        assert L.moe_linear_workspace_bytes(T, K, N, 1) == 0


def test_forward_refusals(L):
    def f(x=FAKE, w=2 * FAKE, b=3 * FAKE, r=None, T=4, K=64, N=32, act=2, dt=0, odt=0, pre=None, out=FAR, ws=None, n=0):
        return L.moe_linear_forward(x, w, b, r, T, K, N, act, dt, odt, pre, out, ws, n, None)
    for kw in (dict(T=0), dict(K=60), dict(N=12), dict(K=(1 << 17) + 8), dict(N=(1 << 20) + 8), dict(T=(1 << 24) + 1)):
        assert f(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(b=FAKE + 4), dict(r=FAKE + 8),
               dict(out=FAR + 8), dict(act=3), dict(act=-1), dict(dt=2), dict(odt=1), dict(odt=3), dict(pre=FAR + FAKE),
               dict(act=0, pre=FAR + FAKE + 4), dict(out=FAKE), dict(out=FAKE + 496), dict(out=2 * FAKE), dict(out=3 * FAKE),
               dict(r=FAR + 16), dict(act=0, pre=FAR), dict(act=0, pre=FAKE), dict(act=0, pre=4 * FAKE, r=4 * FAKE)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw
    need = L.moe_linear_workspace_bytes(160, 16384, 1024, 0)
    assert need > 0
    big = dict(T=160, K=16384, N=1024, w=64 * FAKE)
    assert f(**big, ws=FAR + 64 * FAKE, n=need - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    assert f(**big, ws=None, n=need) == L.MOE_ERR_INVALID_ARG
    assert f(**big, ws=FAR + 16, n=need) == L.MOE_ERR_INVALID_ARG


def test_backward_refusals(L):
    ws = L.moe_linear_workspace_bytes(4, 64, 32, 1)

    def f(d=FAKE, x=2 * FAKE, w=3 * FAKE, pre=None, T=4, K=64, N=32, act=2, dt=0, odt=0, dx=FAR, dw=FAR + FAKE, db=FAR + 2 * FAKE,
          wp=FAR + 3 * FAKE, n=ws):
        return L.moe_linear_backward(d, x, w, pre, T, K, N, act, dt, odt, dx, dw, db, wp, n, None)
    for kw in (dict(T=0), dict(K=60), dict(N=12)):
        assert f(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(d=None), dict(x=None), dict(w=None), dict(dx=None, dw=None, db=None), dict(act=0), dict(pre=4 * FAKE),
               dict(d=FAKE + 8), dict(dx=FAR + 8), dict(dw=FAR + 8), dict(db=FAR + 4), dict(wp=None), dict(wp=FAR + 16), dict(dt=2),
               dict(odt=1), dict(act=3), dict(dx=FAKE), dict(dw=2 * FAKE), dict(db=3 * FAKE), dict(act=0, pre=FAR)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw
    assert f(n=ws - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL


def test_no_gradient_is_cut_in_silence(L):
    import torch
    import mxfp4_expert_layer_gb300 as pkg

    def t(*s, grad=False, dt=torch.bfloat16):
        return torch.zeros(*s, dtype=dt, requires_grad=grad)
    given = dict(x=t(4, 64), weight=t(32, 64), bias=t(32, dt=torch.float32), residual=t(4, 32))
    for name, v in given.items():
        def call(grad):
            return pkg.linear_forward(**dict(given, **{name: t(*v.shape, grad=grad, dt=v.dtype)}))
        with pytest.raises(ValueError, match=f"{name} requires grad.*explicit calls"):
            call(True)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(True)
        with pytest.raises(ValueError, match="CUDA"):
            call(False)
    with pytest.raises(ValueError, match="d_out requires grad"):
        pkg.linear_backward(t(4, 32, grad=True), given["x"], given["weight"])
    with pytest.raises(ValueError, match="out_dtype"):
        pkg.linear_forward(given["x"], given["weight"], out_dtype=torch.float16)
