"""Bounded waits of the projections' kernels: a wait that gives up is reported, the kernel (and
its cluster) drains and leaves, and what follows is as if it had not been."""

import pytest
import torch

from tests import test_gpu_linear as linear
from tests.test_gpu_dense_waits import limit  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def step(m, backward):
    import mxfp4_expert_layer_gb300 as pkg
    out, pre = linear.forward(m, "gelu", save=True)
    return (out, pre) + (tuple(pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=1)) if backward else ())


@pytest.mark.parametrize("T,K,N,out,backward", [
    (24, 64, 128, BF16, False), (64, 4096, 2880, BF16, False), (48, 1088, 20000, F32, False),  # batches: K whole, cut, many blocks
    (100, 4096, 520, F32, False), (128, 16384, 4096, BF16, False),                             # and of 128 tokens
    (90, 520, 1032, BF16, True), (160, 16384, 1024, F32, True),                                # one-SM tiles, K whole and cut
    (600, 512, 1024, BF16, True), (1001, 2880, 2880, F32, True)])                              # pair tiles
def test_no_time_out_goes_unreported(T, K, N, out, backward, limit):  # noqa: F811
    """Limits around the pipeline's own waits, so that some give up and some do not: the
    status word is clear only where every result is right, and the next call is right."""
    import mxfp4_expert_layer_gb300 as pkg
    m = linear.make(T, K, N, BF16, out, seed=T)
    want = step(m, backward)
    assert pkg.dense_status() == 0
    for ns in (1, 300, 1000, 1999, 2500, 5000, 10000, 60000):
        limit(ns)
        got = step(m, backward)
        torch.cuda.synchronize()
        limit(0)
        st = pkg.dense_status()
        assert st & ~0b111 == 0
        if st == 0:
            for a, b in zip(got, want):
                assert torch.equal(a, b), ns
        for a, b in zip(step(m, backward), want):
            assert torch.equal(a, b), ns
        assert pkg.dense_status() == 0


@pytest.mark.parametrize("T,K,N", [(17, 8, 8), (33, 1032, 264), (128, 1048, 136)])
def test_clusters_that_end_at_once(T, K, N):
    """Clusters of few K groups, many launches close behind one another: a block leaves when
    nothing is left to arrive in its shared memory."""
    import mxfp4_expert_layer_gb300 as pkg
    m = linear.make(T, K, N, torch.float16, seed=T)
    want, _ = linear.check(m, backward=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(100):
            got = linear.forward(m)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and pkg.dense_status() == 0
