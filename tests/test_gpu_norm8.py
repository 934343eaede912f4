"""GPU parity of the norm around a block with an 8-bit output (moe_block_norm_8bit) against
the 64-bit statement of y from the stored stream.

Bounds.  y is an f32 value off by at most 32 roundings of 2^-24 of itself (as block_norm's out
before its rounding); its scale by as much, two more in the row form (a product and a largest).
A code is one rounding of y / scale: half a step, 2^-4 of it, or 2^-10 among the subnormals
(steps of 2^-9); the quotient's own 3 roundings are counted with y's."""

import pytest
import torch

from tests import dense_ref as ref
from tests import test_gpu_block_norm as norm
from tests.dense_ref import U32

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3_HALF = 2.0 ** -4
FUZZ = 40 * U32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def call(m, a, scales, with_out=False):
    import mxfp4_expert_layer_gb300 as pkg
    return pkg.block_norm_8bit(m["z"], m["r"], norm_weight=m["w"], gate=m["g"], residual_scale=a, next_weight=m["v"],
                               eps=norm.EPS, scales=scales, with_out=with_out)


def values(codes, scales):
    """What the codes and scales stand for, and the scale of each value, in 64 bits."""
    T, H = codes.shape
    wide = scales.double().repeat_interleave(H // scales.shape[1], 1)
    return codes.double() * wide, wide


def check_codes(codes, scales, y):
    """codes and scales of the finite y (64 bits)."""
    T, H = y.shape
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == (T, H)
    top = y.abs().view(T, scales.shape[1], -1).amax(2)
    s = scales.double()
    if scales.dtype == F32:
        want = torch.clamp(top / 448, min=2.0 ** -126)
        assert scales.shape == (T, 1) and ((s - want).abs() <= FUZZ * want).all()
    else:
        assert scales.dtype == torch.float8_e8m0fnu and scales.shape == (T, H // 32)
        # the least power of two, 2^-126 at least, that holds the largest value
        assert (top * (1 - FUZZ) <= 448 * s).all()
        assert ((top * (1 + FUZZ) > 224 * s) | (s == 2.0 ** -126)).all()
    got, wide = values(codes, scales)
    tol = (E4M3_HALF + 2 * FUZZ) * y.abs() + 2.0 ** -10 * wide
    bad = (got - y).abs() > tol
    assert not bad.any(), (int(bad.sum()), got[bad][:3], y[bad][:3])


def check(m, a, scales):
    import mxfp4_expert_layer_gb300 as pkg
    n = call(m, a, scales)
    s, y = norm.forward(m, a)
    assert n.out is None and torch.equal(n.residual, s)  # the same stream as block_norm's, bit for bit
    kept = s.double()
    check_codes(n.codes, n.scales, kept / ref.rms(kept, norm.EPS) * m["v"].double())
    both = call(m, a, scales, with_out=True)
    assert torch.equal(both.out, y) and torch.equal(both.residual, s)
    assert torch.equal(both.codes.view(torch.uint8), n.codes.view(torch.uint8))
    assert torch.equal(both.scales.view(torch.uint8), n.scales.view(torch.uint8))
    assert pkg.dense_status() == 0
    return n


@pytest.mark.parametrize("scales", ["mx", "row"])
@pytest.mark.parametrize("gate", ["none", "feature", "token", "full"])
@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("T,H", [(1, 2880), (5, 32), (37, 288), (700, 96)])
def test_shapes_types_gates(T, H, dtype, stream, gate, scales):
    check(norm.make(T, H, dtype, stream, gate, seed=T + H), 0.7, scales)


@pytest.mark.parametrize("scales", ["mx", "row"])
@pytest.mark.parametrize("T,H", [(1, 8192), (3, 8192), (2, 4128), (1000, 2880), (641, 4096), (2001, 2880), (1300, 4096),
                                 (10007, 288), (18301, 32), (9800, 512), (5000, 256)])
def test_widths_and_many_rows(T, H, scales):
    for gate in ("token", "feature", "full"):
        check(norm.make(T, H, BF16, F32 if H == 4096 else BF16, gate, seed=H), 1.0, scales)


@pytest.mark.parametrize("T,H", [(3, 8), (17, 2888), (9, 8184), (10007, 264)])
def test_rows_of_any_eight(T, H):
    check(norm.make(T, H, F16, F16, "token", seed=H), 0.5, "row")


@pytest.mark.parametrize("scales", ["mx", "row"])
@pytest.mark.parametrize("post,residual,gate", [(False, True, "none"), (True, False, "feature"), (False, False, "token"),
                                                (False, True, "full")])
def test_absent_arguments(post, residual, gate, scales):
    check(norm.make(19, 320, BF16, BF16, gate, seed=3, post=post, residual=residual), 0.5, scales)


@pytest.mark.parametrize("scales", ["mx", "row"])
@pytest.mark.parametrize("T", [3, 20000])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e30, 3e35])
def test_sizes_at_both_ends(T, size, scales):
    """y near the ends of f32: scales of 2^-126 with codes among the subnormals, and large
    powers of two."""
    m = norm.make(T, 64, BF16, BF16, "none", seed=1)
    m["v"] = (m["v"].float() * size).to(BF16)
    check(m, 1.0, scales)


@pytest.mark.parametrize("T,H", [(2, 256), (2, 2880), (9800, 512)])
def test_zeros_and_what_is_not_finite(T, H):
    """A row of zeros has the least scale and zeros; an infinity or a NaN of y its group's, or
    its row's, NaN scale and NaN codes, and touches nothing else."""
    for scales in ("mx", "row"):
        m = norm.make(T, H, BF16, BF16, "none", seed=2)
        clean = call(m, 1.0, scales)
        m["z"][0], m["r"][0] = 0, 0
        n = call(m, 1.0, scales)
        assert not n.codes[0].double().any() and (n.scales[0].double() == 2.0 ** -126).all()
        assert torch.equal(n.codes[1:].view(torch.uint8), clean.codes[1:].view(torch.uint8))
        for bad in (float("nan"), float("inf")):
            m = norm.make(T, H, BF16, BF16, "none", seed=2)
            m["v"][45] = bad
            n = call(m, 1.0, scales)
            hit = torch.zeros(T, H, dtype=torch.bool, device="cuda")
            hit[:, 32:64] = True
            if scales == "row":
                hit[:] = True
            assert torch.equal(torch.isnan(n.codes.double()), hit)
            assert torch.equal(torch.isnan(n.scales.double()), hit.view(T, n.scales.shape[1], -1).any(2))
            assert torch.equal(n.codes.view(torch.uint8)[~hit], clean.codes.view(torch.uint8)[~hit])
            m = norm.make(T, H, BF16, BF16, "none", seed=2)
            m["z"][1, 7] = bad  # every y of the row is NaN: NaN / NaN, or (with an infinite rms) 0 and NaN
            n = call(m, 1.0, scales)
            assert torch.isnan(n.scales[1].double()).all() if bad != bad else torch.isnan(n.scales[1].double()).any()
            keep = torch.arange(T, device="cuda") != 1
            assert torch.equal(n.codes.view(torch.uint8)[keep], clean.codes.view(torch.uint8)[keep])


def test_captured_and_in_place_through_the_c_entry():
    import mxfp4_expert_layer_gb300 as pkg
    L = pkg._lib
    for T, H in ((7, 2880), (9800, 512)):
        for scales in ("mx", "row"):
            m = norm.make(T, H, BF16, BF16, "token", seed=T)
            want = call(m, 0.7, scales, with_out=True)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = call(m, 0.7, scales, with_out=True)
            graph.replay()
            for a, b in zip(got, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            codes, sc = torch.empty_like(want.codes), torch.empty_like(want.scales)
            z, r = m["z"].clone(), m["r"].clone()
            L.check("moe_block_norm_8bit", L.moe_block_norm_8bit(
                z.data_ptr(), m["w"].data_ptr(), m["g"].data_ptr(), L.MOE_GATE_TOKEN, r.data_ptr(), 0.7, m["v"].data_ptr(),
                norm.EPS, T, H, 0, 0, L.MOE_SCALE_MX if scales == "mx" else L.MOE_SCALE_ROW, r.data_ptr(), codes.data_ptr(),
                sc.data_ptr(), z.data_ptr(), torch.cuda.current_stream().cuda_stream))
            for a, b in ((r, want.residual), (z, want.out), (codes, want.codes), (sc, want.scales)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            # without the stream: the codes alone
            L.check("moe_block_norm_8bit", L.moe_block_norm_8bit(
                m["z"].data_ptr(), m["w"].data_ptr(), m["g"].data_ptr(), L.MOE_GATE_TOKEN, m["r"].data_ptr(), 0.7,
                m["v"].data_ptr(), norm.EPS, T, H, 0, 0, L.MOE_SCALE_MX if scales == "mx" else L.MOE_SCALE_ROW, None,
                codes.view(torch.uint8).zero_().data_ptr(), sc.data_ptr(), None, torch.cuda.current_stream().cuda_stream))
            assert torch.equal(codes.view(torch.uint8), want.codes.view(torch.uint8))


def test_refusals():
    import mxfp4_expert_layer_gb300 as pkg
    m = norm.make(4, 40, BF16, BF16, "none", seed=1)
    z, r, v = m["z"], m["r"], m["v"]
    for kw in (dict(block=z.float()), dict(residual=r.half()), dict(next_weight=v.half()), dict(next_weight=v[:8]),
               dict(next_weight=None), dict(scales="block"), dict(block=z[0]), dict(residual=r[:2])):
        with pytest.raises(ValueError):
            pkg.block_norm_8bit(**dict(dict(block=z, residual=r, next_weight=v, scales="row"), **kw))
    for kw in (dict(scales="mx"), dict(eps=-1.0), dict(residual_scale=float("nan")), dict(block=z[:0], residual=r[:0])):
        with pytest.raises(pkg._lib.MoEError):
            pkg.block_norm_8bit(**dict(dict(block=z, residual=r, next_weight=v, scales="row"), **kw))
    check(m, 1.0, "row")


def test_more_than_2_31_elements():
    T, H = 270000, 8192
    m = norm.make(T, H, BF16, BF16, "none", seed=1)
    for scales in ("mx", "row"):
        n = call(m, 1.0, scales)
        for part in (slice(0, 50), slice(T // 2, T // 2 + 50), slice(T - 50, T)):
            kept = n.residual[part].double()
            check_codes(n.codes[part], n.scales[part], kept / ref.rms(kept, norm.EPS) * m["v"].double())
