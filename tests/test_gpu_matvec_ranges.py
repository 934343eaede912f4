"""MXFP4 products (moe_matvec_mxfp4) of bf16 values at the ends of their range, with row
scales that bring the result back to the middle.  Bound: as in test_gpu_matvec.py, whose
terms are all relative to the values; powers of two are taken out and put back exactly as
long as the value itself is inside f32's range."""

import pytest
import torch

from tests import test_gpu_matvec as matvec

pytestmark = pytest.mark.gpu

# (tokens, K): x resident, packed by one, two and four column groups
FORMS = [(3, 256), (3, 4096), (13, 256), (40, 256)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,K", FORMS)
def test_tokens_of_subnormals(T, K, gated):
    """Tokens whose values are all below 2^-126, the smallest normal value, and one of zeros."""
    import mxfp4_expert_layer_gb300 as pkg
    m = matvec.make(T, 96, K, torch.bfloat16, seed=T + K, lo=250, hi=255, bias=False)
    g = torch.Generator(device="cuda").manual_seed(1)
    tiny = torch.randint(-63, 64, (T, K), generator=g, device="cuda").double() * 2.0 ** -133  # a bf16's smallest step
    m["x"] = tiny.to(torch.bfloat16)
    assert torch.equal(m["x"].double(), tiny)
    m["x"][1] = 0
    _, y = matvec.check(m, gated)
    assert y[0].any() and not y[1].any()
    assert pkg.dense_status() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,K", FORMS)
def test_large_values_against_small_scales(T, K, gated):
    """Values around 2^120 against row scales of 2^-127 to 2^-123: the sums with the tokens'
    scales alone are past f32's largest value, the results are ordinary."""
    m = matvec.make(T, 96, K, torch.bfloat16, seed=T + K, lo=0, hi=5)
    m["x"] *= 2.0 ** 120
    assert torch.isfinite(m["x"]).all()
    m["x"][-1] *= 2.0 ** -120  # beside them, an ordinary token: its products vanish beside the bias
    _, y = matvec.check(m, gated)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("T,K", FORMS)
def test_small_values_against_a_large_scale_of_zero_codes(T, K):
    """Values around 2^-120 in rows whose largest scale, 2^127, has only zero codes, and whose
    other scales are around 2^35: the sums with the tokens' scales alone are below f32's
    smallest value, the results around 2^-80."""
    m = matvec.make(T, 96, K, torch.bfloat16, seed=T + K, lo=160, hi=165, bias=False)
    m["x"] *= 2.0 ** -120
    m["codes"][:, 16:32] = 0
    m["scales"][:, 1] = 254
    _, y = matvec.check(m, False)
    assert y.float().abs().max() > 2.0 ** -85


@pytest.mark.parametrize("T", [1, 9, 30])
def test_clusters_along_k_repeat(T):
    """Few rows and a long K: the blocks of a cluster take a share of K each and meet at its
    barrier straight after their last stages, many times over."""
    import mxfp4_expert_layer_gb300 as pkg
    m = matvec.make(T, 260, 16384, torch.bfloat16, seed=T)
    w, want = matvec.check(m, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(200):
            got = w(m["x"])
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert pkg.dense_status() == 0
