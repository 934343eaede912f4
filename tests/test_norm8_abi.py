"""CPU checks of the 8-bit norm's entry point: what it refuses, before any launch."""

import pytest

FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks first
FAR = 1 << 34


@pytest.fixture(scope="module")
def L():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    pkg._lib.load()
    return pkg._lib


def test_refusals(L):
    def f(block=FAKE, nw=2 * FAKE, gate=None, kind=0, res=3 * FAKE, a=1.0, nxt=4 * FAKE, eps=1e-5, T=4, H=64, dt=0, sdt=0,
          scale=0, ro=FAR, codes=FAR + FAKE, sc=FAR + 2 * FAKE, out=None):
        return L.moe_block_norm_8bit(block, nw, gate, kind, res, a, nxt, eps, T, H, dt, sdt, scale, ro, codes, sc, out, None)
    for kw in (dict(T=0), dict(H=0), dict(H=12), dict(H=8200), dict(H=40), dict(T=(1 << 24) + 1)):
        assert f(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
    assert f(H=40, scale=1, codes=None) == L.MOE_ERR_INVALID_ARG  # (a row scale takes any width)
    for kw in (dict(block=None), dict(nxt=None), dict(codes=None), dict(sc=None), dict(codes=FAR + FAKE + 8), dict(sc=FAR + 4),
               dict(ro=FAR + 8), dict(out=FAR + 3 * FAKE + 8), dict(scale=2), dict(scale=-1), dict(eps=-1.0), dict(a=float("inf")),
               dict(dt=2), dict(sdt=1), dict(kind=1), dict(gate=FAKE),
               dict(codes=FAKE), dict(codes=3 * FAKE), dict(codes=FAR), dict(sc=FAR), dict(sc=4 * FAKE), dict(sc=FAR + FAKE + 240),
               dict(ro=FAKE), dict(ro=3 * FAKE + 16), dict(out=3 * FAKE), dict(out=FAKE + 16), dict(out=FAR), dict(out=FAR + FAKE),
               dict(out=2 * FAKE)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_no_gradient_is_cut_in_silence(L):
    import torch
    import mxfp4_expert_layer_gb300 as pkg

    def t(*s, grad=False):
        return torch.zeros(*s, dtype=torch.bfloat16, requires_grad=grad)
    given = dict(block=t(4, 64), residual=t(4, 64), norm_weight=t(64), gate=t(64), next_weight=t(64))
    for name, v in given.items():
        with pytest.raises(ValueError, match=f"{name} requires grad.*explicit calls"):
            pkg.block_norm_8bit(**dict(given, **{name: t(*v.shape, grad=True)}))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.block_norm_8bit(**given)
    with pytest.raises(ValueError, match="row"):
        pkg.block_norm_8bit(**given, scales="tensor")
