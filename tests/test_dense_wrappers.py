"""CPU checks of the dense operators' Python entry points: what they refuse before any
tensor has to be on a GPU."""

import pytest


@pytest.fixture(scope="module")
def pkg():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    return pkg


def bf16(*shape, grad=False):
    import torch
    return torch.zeros(*shape, dtype=torch.bfloat16, requires_grad=grad)


def calls(pkg):
    """(name of the argument that requires grad, call with it)."""
    z, w = bf16(4, 64), bf16(64)
    norm = dict(block=z, residual=z, norm_weight=w, gate=w, next_weight=w)
    for name in norm:
        yield name, lambda t, n=name: pkg.block_norm(**dict(norm, **{n: t(*norm[n].shape)}))
    ffn = dict(x=z, w_gateup=bf16(32, 64), w_down=bf16(64, 16))
    for name in ffn:
        yield name, lambda t, n=name: pkg.ffn_forward(**dict(ffn, **{n: t(*ffn[n].shape)}))
    back = dict(d_out=z, x=z, gateup=bf16(4, 32).float(), w_gateup=bf16(32, 64), w_down=bf16(64, 16))
    yield "d_out", lambda t: pkg.ffn_backward(**dict(back, d_out=t(4, 64)))
    for name in ("d_residual_out", "d_out"):
        given = dict(d_residual_out=z, d_out=z, block=z, residual_out=z, next_weight=w)
        yield name, lambda t, n=name, g=given: pkg.block_norm_backward(**dict(g, **{n: t(4, 64)}))


def test_no_gradient_is_cut_in_silence(pkg):
    """Results carry no history, so a tensor that requires grad is refused while autograd
    records; outside of that (where these CPU tensors are refused for not being on a GPU)
    it is as any other."""
    import torch
    seen = 0
    for name, call in calls(pkg):
        with pytest.raises(ValueError, match=f"{name}.*explicit calls"):
            call(lambda *s: bf16(*s, grad=True))
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(lambda *s: bf16(*s, grad=True))
        with pytest.raises(ValueError, match="CUDA"):
            call(bf16)
        seen += 1
    assert seen == 11


@pytest.mark.gpu
def test_with_parameters_under_no_grad(pkg):
    import torch
    from tests import test_gpu_ffn as ffn
    from tests import test_gpu_matvec as matvec
    m = ffn.make(20, 64, 72, torch.bfloat16)
    want = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    p = {k: torch.nn.Parameter(v) for k, v in m.items()}
    with pytest.raises(ValueError, match="explicit calls"):
        pkg.ffn_forward(p["x"], p["wgu"], p["wd"])
    with torch.no_grad():
        out, gu = pkg.ffn_forward(p["x"], p["wgu"], p["wd"], save=True)
    assert torch.equal(out, want)
    grads = pkg.ffn_backward(m["dy"], p["x"], gu, p["wgu"], p["wd"])  # (explicit already)
    for a, b in zip(grads, pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"])):
        assert torch.equal(a, b)
    v = matvec.make(3, 64, 128, torch.bfloat16)
    w = pkg.MatvecMXFP4(v["codes"], v["scales"], bias=v["bias"])
    x = v["x"].clone().requires_grad_()
    with pytest.raises(ValueError, match="x requires grad.*explicit calls"):
        w(x)
    with torch.no_grad():
        assert torch.equal(w(x), w(v["x"]))


def test_flags_without_a_truth_value(pkg):
    """A flag whose truth value raises passes that error on (these calls would else go on
    to refuse their CPU tensors, or on a GPU to return with an error set)."""
    class Flag:
        def __bool__(self):
            raise KeyError("no truth value")
    z, w = bf16(4, 64), bf16(64)
    wgu, wd, gu = bf16(32, 64), bf16(64, 16), bf16(4, 32).float()
    for call in (lambda: pkg.ffn_forward(z, wgu, wd, save=Flag()),
                 lambda: pkg.ffn_backward(z, z, gu, wgu, wd, need_x=Flag()),
                 lambda: pkg.ffn_backward(z, z, gu, wgu, wd, need_weights=Flag()),
                 lambda: pkg.block_norm_backward(z, z, z, z, next_weight=w, has_residual=Flag())):
        with pytest.raises(KeyError, match="no truth value"):
            call()


def test_a_products_output_over_its_input(pkg):
    """Blocks of the MXFP4 product write their outputs while others still read x: outputs
    over any part of x are refused, outputs beside it are not."""
    from mxfp4_expert_layer_gb300 import _lib as L
    base = 1 << 20  # never dereferenced: what passes the checks finds no GPU, or is not run

    def call(x, out, T=2, rows=64, K=96, kind=L.MOE_WEIGHTS_DOWN):
        return L.moe_matvec_mxfp4(x, base << 4, None, T, rows, K, kind, 0, 0, out, None, 0, None)
    n_x, n_out = 2 * 96 * 2, 2 * 64 * 2
    for out in (base, base + 16, base + n_x - 16, base - n_out + 16):
        assert call(base, out) == L.MOE_ERR_INVALID_ARG
    assert call(base, base - n_out // 2, kind=L.MOE_WEIGHTS_GATEUP, rows=128) == L.MOE_ERR_INVALID_ARG
    import torch
    if not torch.cuda.is_available():
        for out in (base + n_x, base - n_out):
            assert call(base, out) == L.MOE_ERR_CUDA
