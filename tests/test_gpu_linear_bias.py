"""The bias gradient of a projection, at the bound that its sums have: T rows go to at most 64 blocks
(16 rows each at least, four blocks to an SM over all columns), in a block to eight warps in turn, whose
sums are added in order, then eight threads add the blocks' in turn and in order.  With r rows a block:
r / 8 + 1 additions of a warp, 7 of the warps, 8 of a thread's blocks and 7 of the threads."""

import pytest
import torch

from tests import test_gpu_linear as linear
from tests.dense_ref import U32, floor_of, within

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def additions(T, N):
    columns = -(-N // 256)
    blocks = min(-(-4 * 160 // columns), -(-T // 16), 64)
    return -(-T // blocks) / 8 + 1 + 7 + 8 + 7


@pytest.mark.parametrize("T,N", [(1, 8), (17, 8), (100, 2880), (1001, 2880), (8192, 128), (8192, 8), (4096, 40000), (20000, 264)])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32)])
def test_sums(T, N, act, dtype, out):
    import mxfp4_expert_layer_gb300 as pkg
    m = linear.make(T, 8, N, dtype, out, residual=False, seed=T + N)
    m["d"] = (m["d"].float() + 0.5).to(m["d"].dtype)  # (sums that grow, as gradients of one sign do)
    pre = None if act == "none" else 3 * linear.make(T, 8, N, dtype, F32, seed=1)["d"]
    got = pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=linear.ACTS[act], need_x=False, need_weight=False).bias
    d = m["d"].double()
    if act == "none":
        dp, e = d, torch.zeros_like(d)
    else:
        p = pre.double().requires_grad_()
        (slope,) = torch.autograd.grad(linear.act64(p, act).sum(), p)
        dp, e = d * slope, d.abs() * 20 * U32 * (1 + p.detach().abs())
    within(got, dp.sum(0), (e + additions(T, N) * U32 * dp.abs()).sum(0) + floor_of(F32))
