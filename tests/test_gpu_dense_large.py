"""The dense operators on arrays of more than 2^31 elements or bytes: every offset of a row,
a column of the saved products or a weight passes 32 bits.  The last rows are checked; the
gradients that sum over tokens get their terms from these rows alone (the others' incoming
gradients are zero, which adds exact zeros)."""

import pytest
import torch

from tests import test_gpu_block_norm as norm
from tests import test_gpu_ffn as ffn
from tests import test_gpu_matvec as matvec
from tests.dense_ref import half_step, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    yield
    torch.cuda.empty_cache()


def test_norms():
    import mxfp4_expert_layer_gb300 as pkg
    T, H, last = (1 << 18) + 5, 8192, 5
    assert T * H > 1 << 31
    m = norm.make(last, H, BF16, BF16, "feature", seed=1)

    def whole(t):
        big = torch.zeros(T, H, dtype=t.dtype, device="cuda")
        big[-last:] = t
        return big

    big = dict(m, z=whole(m["z"]).fill_(0.5), r=whole(m["r"]).fill_(-0.25), ds=whole(m["ds"]), dy=whole(m["dy"]))
    big["z"][-last:], big["r"][-last:] = m["z"], m["r"]
    s, y = norm.forward(big, 0.7)
    norm.check_forward(m, 0.7, s[-last:], y[-last:])
    assert torch.equal(s[0], s[T // 2]) and torch.equal(y[0], y[T // 2])
    g = pkg.block_norm_backward(big["ds"], big["dy"], big["z"], s, norm_weight=m["w"], gate=m["g"], residual_scale=0.7,
                                next_weight=m["v"], eps=norm.EPS)
    norm.check_backward(m, 0.7, s[-last:], g._replace(block=g.block[-last:], residual=g.residual[-last:]))
    assert not g.block[0].any() and not g.residual[T // 2].any()


def test_feed_forward():
    import mxfp4_expert_layer_gb300 as pkg
    T, H, I, last = 70001, 64, 16384, 40
    assert T * 2 * I > 1 << 31
    m = ffn.make(T, H, I, BF16, seed=2)
    m["dy"][:-last] = 0
    out, gu = pkg.ffn_forward(m["x"], m["wgu"], m["wd"], save=True)
    grads = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"])
    small = dict(m, x=m["x"][-last:].contiguous(), dy=m["dy"][-last:].contiguous())
    want, want_gu = ffn.check(small)  # (against the 64-bit statement)
    few = pkg.ffn_backward(small["dy"], small["x"], want_gu, m["wgu"], m["wd"])
    # the same sums in another order: a rounding of each 16-bit result and operand on both sides
    for a, b in ((out[-last:], want), (grads.x[-last:], few.x), (grads.w_gateup, few.w_gateup), (grads.w_down, few.w_down)):
        a, b = a.double(), b.double()
        assert (a - b).norm() <= 4 * half_step(BF16) * b.norm()
    assert (gu[-last:].double() - want_gu.double()).norm() <= 1e-5 * want_gu.double().norm()
    assert not grads.x[0].any()
    assert pkg.dense_status() == 0


@pytest.mark.parametrize("T", [1, 12])
def test_mxfp4_weights(T):
    import mxfp4_expert_layer_gb300 as pkg
    rows, K, last = 140001, 65536, 33
    assert rows * K // 2 > 1 << 32
    m = matvec.make(T, rows, K, BF16, seed=3)
    y = pkg.MatvecMXFP4(m["codes"], m["scales"], bias=m["bias"])(m["x"])
    end = dict(m, codes=m["codes"][-last:], scales=m["scales"][-last:], bias=m["bias"][-last:])
    within(y[:, -last:], *matvec.expect(end, False))
    assert pkg.dense_status() == 0
