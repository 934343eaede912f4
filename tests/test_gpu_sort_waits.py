"""Bounded waits of the moves between token and expert order: a wait for a row that gives up is
reported, no row is asked for into a place that still waits for its last one, the kernel leaves,
and what follows is as if it had not been."""

import pytest
import torch

from tests import test_gpu_sort as sort
from tests.test_gpu_dense_waits import limit  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


# each takes the kernels with rings of row copies: more than 2048 assignments, and tokens for several
# rounds of every resident block; one group of rows and two, one chunk of columns and several
@pytest.mark.parametrize("T,k,E,H,dtype", [(3000, 4, 32, 2880, BF16), (2500, 9, 32, 2888, F32), (2000, 2, 8, 16384, BF16),
                                           (16000, 2, 8, 64, BF16)])
def test_no_time_out_goes_unreported(T, k, E, H, dtype, limit):  # noqa: F811
    """Limits around a copy's own time, so that some waits give up and some do not: the status
    word is clear only where every result is right, and the next calls are right."""
    import mxfp4_expert_layer_gb300 as pkg
    x, y, d = sort.rows_of(T, H, dtype, 1), sort.rows_of(T * k, H, dtype, 2), sort.rows_of(T, H, dtype, 3)
    idx, w = sort.routing(T, k, E, 0.1, seed=T), torch.rand(T, k, device="cuda")
    inv = sort.order(idx, E)[2]
    calls = {"sort": lambda: [t for t in pkg.sort_tokens(x, idx, E) if t is not None],
             "unsort": lambda: [pkg.unsort_tokens(y, inv, w)],
             "unsort backward": lambda: list(pkg.unsort_tokens_backward(d, y, inv, w)),
             "d_y alone": lambda: [pkg.unsort_tokens_backward(d, None, inv, w, need_w=False).y]}
    want = {name: call() for name, call in calls.items()}
    assert pkg.dense_status() == 0
    gave_up = set()
    for name, call in calls.items():
        for ns in (1, 300, 1000, 1999, 2500, 5000, 10000, 60000):
            limit(ns)
            got = call()
            torch.cuda.synchronize()
            limit(0)
            st = pkg.dense_status()
            assert st & ~0b111 == 0
            if st:
                gave_up.add(name)
            else:
                for a, b in zip(got, want[name]):
                    assert torch.equal(a, b), (name, ns)
            for a, b in zip(call(), want[name]):
                assert torch.equal(a, b), (name, ns)
            assert pkg.dense_status() == 0
    # a copy from HBM takes hundreds of ns: the first waits of a launch cannot all be met in 1 ns
    assert gave_up >= {"unsort", "unsort backward", "d_y alone"}


def test_time_outs_between_calls_that_have_none(limit):  # noqa: F811
    """Launches that give up in the middle of a stream, and in a captured graph, leave the others alone."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 4000, 4, 16, 2880
    x, y, w = sort.rows_of(T, H, BF16, 1), sort.rows_of(T * k, H, BF16, 2), torch.rand(T, k, device="cuda")
    idx = sort.routing(T, k, E, seed=T)
    s = pkg.sort_tokens(x, idx, E)
    want = (s.rows, pkg.unsort_tokens(y, s.inv_perm, w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        limit(1)
        pkg.unsort_tokens(y, s.inv_perm, w)
        limit(0)
        got = (pkg.sort_tokens(x, idx, E).rows, pkg.unsort_tokens(y, s.inv_perm, w))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert pkg.dense_status() != 0 and pkg.dense_status() == 0
