"""Bounded waits of the dense GEMMs: a wait that gives up is reported whichever thread it
is, the kernel drains and leaves, and what follows is as if it had not been."""

import pytest
import torch

from tests import test_gpu_ffn as ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.fixture
def limit():
    """Sets the waits' limit (ns); the default and a clear status word afterwards."""
    import mxfp4_expert_layer_gb300 as pkg
    from mxfp4_expert_layer_gb300 import _lib as L

    def set_(ns):
        assert L.moe_set_wait_limit_ns(ns) == L.MOE_OK
    yield set_
    set_(0)
    torch.cuda.synchronize()
    pkg.dense_status()


def training_step(m):
    import mxfp4_expert_layer_gb300 as pkg
    out, gu = pkg.ffn_forward(m["x"], m["wgu"], m["wd"], save=True)
    return (out, gu) + tuple(pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"]))


@pytest.mark.parametrize("T,H,I", [(64, 1024, 512),      # one-SM tiles, K split
                                   (600, 512, 1024), (1001, 2880, 2880)])  # pair tiles, one and more rounds
def test_no_time_out_goes_unreported(T, H, I, limit):
    """Limits around the pipeline's own waits, so that some give up and some do not: the
    status word is clear only where every result is right, and the next call is right."""
    import mxfp4_expert_layer_gb300 as pkg
    m = ffn.make(T, H, I, torch.bfloat16, seed=T)
    want = training_step(m)
    assert pkg.dense_status() == 0
    for ns in (1, 300, 1000, 1999, 2500, 5000, 10000, 20000, 60000):
        limit(ns)
        got = training_step(m)
        torch.cuda.synchronize()
        limit(0)
        st = pkg.dense_status()
        assert st & ~0b111 == 0
        if st == 0:
            for a, b in zip(got, want):
                assert torch.equal(a, b), ns
        for a, b in zip(training_step(m), want):
            assert torch.equal(a, b), ns
        assert pkg.dense_status() == 0


@pytest.mark.parametrize("T,H,I", [(129, 8, 8), (300, 8, 264), (513, 264, 8)])
def test_pairs_that_end_at_once(T, H, I):
    """Pair tiles of one to five K groups, many launches close behind one another: a pair's
    blocks leave as soon as their barriers have had every arrival."""
    import mxfp4_expert_layer_gb300 as pkg
    m = ffn.make(T, H, I, torch.float16, seed=T)
    want = training_step(m)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(50):
            got = training_step(m)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert pkg.dense_status() == 0


@pytest.mark.parametrize("T", [100, 600])  # one-SM and pair tiles
def test_a_time_out_holds_up_its_own_launch_only(T, limit):
    """A launch whose wait gave up stays 20 ms for its copies to land.  Later launches do
    not, also while nobody has read the status word: ten of them take less than those 20 ms
    (each a few microseconds of work), and are right."""
    import mxfp4_expert_layer_gb300 as pkg
    m = ffn.make(T, 512, 1024, torch.bfloat16, seed=T)
    want = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    limit(1)
    pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    torch.cuda.synchronize()
    limit(0)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(5):
        got = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    end.record()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert start.elapsed_time(end) < 20
    assert pkg.dense_status() != 0
