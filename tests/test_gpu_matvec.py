"""GPU parity of the few-token products with MXFP4 weights (moe_matvec_mxfp4) against the
64-bit product with the dequantised weights.

Bound.  The weights are exact (group scales down to 2^-126 of their row's largest); f16 x
is exact, bf16 x is exact down to 2^-28 of its token's largest value and off by at most
2^-39 of that below.  The sums are f32: tensor core steps of 16 products (counted as
2^-22 of the terms' magnitude each: products of different sizes are aligned before they
are added), a group's scaling, a warp's chain of groups and the warps' sums: a step and
K / 32 + 8 roundings of 2^-24, less than 8 + K / 128 of 2^-22.  One rounding at the end."""

import pytest
import torch

from tests import dense_ref as ref
from tests.dense_ref import U32, floor_of, half_step, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def make(T, rows, K, dtype, seed=0, lo=120, hi=125, bias=True, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    return dict(x=torch.randn(T, K, generator=g, device=dev).to(dtype),
                codes=torch.randint(0, 256, (rows, K // 2), generator=g, device=dev, dtype=torch.uint8),
                scales=torch.randint(lo, hi, (rows, K // 32), generator=g, device=dev, dtype=torch.uint8),
                bias=torch.randn(rows, generator=g, device=dev) if bias else None)


def expect(m, gated, act="silu"):
    """(value, tolerance) of the call."""
    x, w = m["x"].double(), ref.dequantise(m["codes"], m["scales"])
    K, dt = x.shape[1], m["x"].dtype
    y, mag = x @ w.t(), x.abs() @ w.t().abs()
    err = 4 * U32 * (8 + K / 128) * mag
    if dt == torch.bfloat16:
        err = err + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * w.abs().sum(1)
    if m["bias"] is not None:
        y = y + m["bias"].double()
        err = err + U32 * (mag + m["bias"].double().abs())
    if gated:
        n = y.shape[1] // 2
        g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
        a = ref.act(g, act)
        # both activations have slopes within 1.2; exp and division in f32 add 16 roundings
        err = (1.2 * eg + 16 * U32 * a.abs()) * (u.abs() + eu) + a.abs() * eu
        y = a * u
    return y, half_step(dt) * y.abs() + err * (1 + half_step(dt)) + floor_of(dt)


def check(m, gated, act="silu"):
    import mxfp4_expert_layer_gb300 as pkg
    w = pkg.MatvecMXFP4(m["codes"], m["scales"], kind=pkg.MOE_WEIGHTS_GATEUP if gated else pkg.MOE_WEIGHTS_DOWN,
                        bias=m["bias"], act=pkg.MOE_ACT_SILU if act == "silu" else pkg.MOE_ACT_GELU)
    y = w(m["x"])
    want, tol = expect(m, gated, act)
    within(y, want, tol)
    return w, y


@pytest.mark.parametrize("gated,act", [(False, "silu"), (True, "silu"), (True, "gelu")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64])
def test_token_counts(T, dtype, gated, act):
    check(make(T, 2 * 200, 416, dtype, seed=T), gated, act)


@pytest.mark.parametrize("rows,K", [(1, 32), (2, 64), (17, 96), (33, 128), (50257, 160), (2880, 2880), (96, 16384),
                                    (5120, 512), (10000, 288), (20000, 256), (40000, 224), (64, 65536)])
@pytest.mark.parametrize("T", [1, 11])
def test_plain_shapes(rows, K, T):
    """Odd row counts, K of one group, K tails inside a unit, one to four tiles a block."""
    check(make(T, rows, K, torch.bfloat16, seed=rows + K), False)


@pytest.mark.parametrize("half,K", [(1, 32), (7, 64), (9, 2880), (2881, 96), (14336, 512), (6000, 256)])
@pytest.mark.parametrize("T", [1, 13])
def test_gated_shapes(half, K, T):
    check(make(T, 2 * half, K, torch.float16, seed=half + K), True)


def test_every_code_and_the_ends_of_the_scale():
    """Each code against each low nibble and every scale byte from 0 (2^-127) to 2^96."""
    K = 32
    scales = torch.arange(0, 224, device="cuda", dtype=torch.uint8).view(-1, 1)
    rows = scales.numel()
    codes = torch.arange(16, device="cuda", dtype=torch.uint8).repeat(rows, 1)
    codes = codes | (codes << 4)
    for dtype, std in ((torch.bfloat16, 1.0), (torch.bfloat16, 2.0 ** 20)):
        x = (torch.randn(3, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * std).to(dtype)
        check(dict(x=x, codes=codes.contiguous(), scales=scales.contiguous(), bias=None), False)


def test_group_scales_far_below_their_row():
    """Scales from 2^-127 to 2^30 in one row: groups below 2^-126 of the largest drop out."""
    m = make(3, 48, 1024, torch.bfloat16, seed=2, lo=0, hi=158, bias=False)
    check(m, False)
    m = make(20, 48, 2048, torch.float16, seed=2, lo=1, hi=140, bias=False)
    check(m, True)


def test_wide_ranges_of_x():
    """Values from 2^-100 to 2^100 of the others in one row, zero rows, rows of subnormals."""
    m = make(6, 64, 1024, torch.bfloat16, seed=3)
    m["x"][0] *= 2.0 ** 100
    m["x"][1] *= 2.0 ** -100
    m["x"][2, ::3] *= 2.0 ** 30
    m["x"][3] = 0
    m["x"][4] *= 2.0 ** -126
    _, y = check(m, False)
    assert torch.equal(y[3], m["bias"].to(y.dtype))


def test_infinities_and_nans_stay_with_their_token():
    m = make(5, 96, 512, torch.bfloat16, seed=4)
    _, clean = check(m, False)
    m["x"][1, 7] = float("inf")
    m["x"][3, 300] = float("nan")
    import mxfp4_expert_layer_gb300 as pkg
    y = pkg.MatvecMXFP4(m["codes"], m["scales"], bias=m["bias"])(m["x"])
    w7 = ref.dequantise(m["codes"], m["scales"])[:, 7]
    for t in (0, 2, 4):
        assert torch.equal(y[t], clean[t])
    assert torch.isnan(y[3]).all()
    assert torch.equal(y[1] == float("inf"), w7 > 0) and torch.equal(torch.isnan(y[1]), w7 == 0)


def test_rows_behind_the_last_are_left_and_calls_repeat():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(9, 4000, 2880, torch.bfloat16, seed=5)
    w = pkg.MatvecMXFP4(m["codes"], m["scales"], bias=m["bias"])
    out = torch.full((11, 4000), 3.0, dtype=torch.bfloat16, device="cuda")
    w(m["x"], out=out[:9])
    assert (out[9:] == 3).all()
    assert torch.equal(out[:9], w(m["x"]))


def test_nan_scales_are_refused():
    import mxfp4_expert_layer_gb300 as pkg
    from mxfp4_expert_layer_gb300 import _lib as L
    m = make(1, 32, 64, torch.bfloat16)
    m["scales"][30, 1] = 255
    with pytest.raises(L.MoEError) as e:
        pkg.MatvecMXFP4(m["codes"], m["scales"])
    assert e.value.status == L.MOE_ERR_NAN_SCALE


def test_captured_graph_follows_its_inputs():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(4, 512, 1024, torch.bfloat16, seed=6)
    w = pkg.MatvecMXFP4(m["codes"], m["scales"], bias=m["bias"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w(m["x"])
    for seed in (7, 8):
        m["x"].copy_(torch.randn(m["x"].shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        want, tol = expect(m, False)
        within(y, want, tol)
