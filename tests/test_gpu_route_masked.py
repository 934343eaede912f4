"""The logits' gradient of tokens whose weights are not finite, or whose gradient is zero: a token
that a mask leaves no expert, a padding token whose logits nobody reads, a dropped assignment."""

import pytest
import torch

from tests import test_gpu_sort as sort
from tests.dense_ref import U32, floor_of, within

pytestmark = pytest.mark.gpu
F32 = torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.mark.parametrize("gating", list(sort.GATINGS))
@pytest.mark.parametrize("E", [8, 48, 256])
def test_a_mask_that_leaves_nothing(E, gating):
    """Logits of -inf alone, or NaN: route's weights are then NaN; the token's assignments are dropped,
    so that its weights' gradient is zero, and so is its logits'."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k = 40, 4
    logits = sort.rows_of(T, E, F32, 1)
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    gone[::3] = True
    logits[::6], logits[3::6] = -INF, NAN
    logits, idx, w = pkg.route(None, None, k, logits=logits, from_logits=True, gating=sort.GATINGS[gating])
    w[3::6] = NAN
    d_w = sort.rows_of(T, k, F32, 2)
    d_w[gone] = 0
    got = pkg.route_backward(d_w, logits, idx, w, gating=sort.GATINGS[gating])
    assert (got[gone] == 0).all()
    want, mag = sort.logits_grad(d_w[~gone], logits[~gone], idx[~gone], w[~gone], gating)
    within(got[~gone], want, 128 * U32 * mag + floor_of(F32))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("gating", ["topk", "sigmoid"])
def test_weights_of_dropped_assignments(gating, bad):
    """Weights that are not finite where the gradient is zero leave the token's other experts
    what they are without them."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E = 20, 4, 32
    logits = sort.rows_of(T, E, F32, 1)
    logits, idx, w = pkg.route(None, None, k, logits=logits, from_logits=True, gating=sort.GATINGS[gating])
    d_w = sort.rows_of(T, k, F32, 2)
    d_w[:, 1] = 0
    zeroed, w = w.clone(), w.clone()
    zeroed[:, 1], w[:, 1] = 0, bad
    got = pkg.route_backward(d_w, logits, idx, w, gating=sort.GATINGS[gating])
    want = pkg.route_backward(d_w, logits, idx, zeroed, gating=sort.GATINGS[gating])
    others = torch.ones(T, E, dtype=torch.bool, device="cuda").scatter_(1, idx[:, 1:2].long(), False)
    assert torch.equal(got[others], want[others]) and torch.isfinite(got[others]).all()


def test_a_step_with_a_masked_token():
    """From logits to their gradient through the moves, one token masked whole: the router's
    weight gradient stays finite."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 30, 2, 16, 64
    x, d_out = sort.rows_of(T, H, torch.bfloat16, 1), sort.rows_of(T, H, torch.bfloat16, 2)
    logits = sort.rows_of(T, E, F32, 3)
    logits[7] = -INF
    logits, idx, w = pkg.route(None, None, k, logits=logits, from_logits=True)
    kept = idx.clone()
    kept[7] = -1
    s = pkg.sort_tokens(x, kept, E)
    out = pkg.unsort_tokens(s.rows, s.inv_perm, w)
    g = pkg.unsort_tokens_backward(d_out, s.rows, s.inv_perm, w)
    d_logits = pkg.route_backward(g.topk_w, logits, idx, w)
    for t in (out, g.y, g.topk_w, d_logits):
        assert torch.isfinite(t.float()).all()
    assert not d_logits[7].any()
