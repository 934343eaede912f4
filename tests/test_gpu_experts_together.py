"""The operators around experts of one's own as a program uses them, each stage held to its own
bound on what the stage before gave it: a training step (router projection, routing, tokens
sorted, experts, tokens back, and every gradient back to the input), and a serving step with
8-bit rows (projection onto the stream, norm with codes, routing, codes and scales sorted,
experts, tokens back), eager, captured and from several threads."""

import threading

import pytest
import torch

from tests import test_gpu_block_norm as norm
from tests import test_gpu_linear as linear
from tests import test_gpu_norm8 as norm8
from tests import test_gpu_sort as sort
from tests.dense_ref import U32, floor_of, half_step, within

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def experts(E, H, I, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
    return dict(up=r(E, I, H, std=H ** -0.5), up_b=torch.randn(E, I, generator=g, device="cuda"),
                down=r(E, H, I, std=I ** -0.5))


@pytest.mark.parametrize("gating", ["topk", "all", "sigmoid"])
@pytest.mark.parametrize("T,k,E,dtype", [(13, 2, 8, F16), (333, 4, 16, BF16), (1500, 2, 8, BF16)])
def test_training_step(T, k, E, dtype, gating):
    """Experts whose feed-forward is two projections, on a batch whose last tokens are padding;
    some experts may get no token."""
    import mxfp4_expert_layer_gb300 as pkg
    H, I, code = 136, 200, sort.GATINGS[gating]
    m = linear.make(T, H, E, dtype, F32, residual=False, seed=T)          # the router
    w, d_out = experts(E, H, I, dtype, T + 1), sort.rows_of(T, H, dtype, T + 2)
    x = m["x"]
    logits, _ = linear.check(m, backward=False)
    logits, idx, topk_w = pkg.route(None, None, k, logits=logits, from_logits=True, gating=code)
    kept = idx.clone()
    kept[T - T // 8:] = -1
    kept[0, 0] = E  # one assignment over its expert's capacity
    s = pkg.sort_tokens(x, kept, E)
    sort.check_sort(s, x, kept, E)
    at = s.offsets.tolist()
    # each expert on its rows; what lies behind the last is left as it is
    y = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    saved = {}
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        up = dict(x=s.rows[rows], w=w["up"][e], b=w["up_b"][e], r=None, d=torch.empty(at[e + 1] - at[e], I, dtype=dtype, device="cuda"))
        h, pre = linear.forward(up, "gelu", save=True)
        linear.check_forward(up, "gelu", h, pre)
        saved[e] = up, h, pre
        pkg.linear_forward(h, w["down"][e], out=y[rows])
    out = pkg.unsort_tokens(y, s.inv_perm, topk_w)
    sort.check_unsort(out, y, s.inv_perm, topk_w)
    # and back
    g = pkg.unsort_tokens_backward(d_out, y, s.inv_perm, topk_w)
    sort.check_unsort_grads(g, d_out, y, s.inv_perm, topk_w)
    d_rows = torch.zeros_like(s.rows)
    for e, (up, h, pre) in saved.items():
        rows = slice(at[e], at[e + 1])
        down = dict(x=h, w=w["down"][e], b=None, r=None, d=g.y[rows])
        gd = pkg.linear_backward(g.y[rows], h, w["down"][e], need_bias=False)
        linear.check_backward(down, "none", None, gd)
        up = dict(up, d=gd.x)
        gu = pkg.linear_backward(gd.x, up["x"], up["w"], pre, act=pkg.MOE_ACT_GELU)
        linear.check_backward(up, "gelu", pre, gu)
        d_rows[rows] = gu.x
    d_x = pkg.sort_tokens_backward(d_rows, s.inv_perm)
    sort.check_unsort(d_x, d_rows, s.inv_perm, None)
    d_logits = pkg.route_backward(g.topk_w, logits, idx, topk_w, gating=code)
    want, mag = sort.logits_grad(g.topk_w, logits, idx, topk_w, gating)
    within(d_logits, want, 128 * U32 * mag + floor_of(F32))
    router = dict(m, d=d_logits)
    gr = pkg.linear_backward(d_logits, x, m["w"])
    linear.check_backward(router, "none", None, gr)
    # padding tokens take no part
    assert not d_logits[T - T // 8:].any() and not d_x[T - T // 8:].any() and not out[T - T // 8:].any()
    assert pkg.dense_status() == 0


def serving_state(T, H, E, seed):
    o = linear.make(T, 264, H, BF16, BF16, seed=seed)                      # attention's output projection, onto the stream
    n = norm.make(T, H, BF16, BF16, "none", seed=seed + 1, post=False)
    router = linear.make(T, H, E, BF16, F32, residual=False, seed=seed + 2)
    up = linear.make(4 * T, H, 96, BF16, BF16, residual=False, seed=seed + 3)
    down = linear.make(4 * T, 96, H, BF16, BF16, bias=False, residual=False, seed=seed + 4)
    return dict(o=o, n=n, router=router, up=up, down=down)


def serving_step(st, E, scales):
    """One expert for all rows, so that the step has one shape and can be captured."""
    import mxfp4_expert_layer_gb300 as pkg
    stream = pkg.linear_forward(st["o"]["x"], st["o"]["w"], st["o"]["b"], st["o"]["r"])
    zero = torch.zeros_like(stream)
    n = pkg.block_norm_8bit(zero, stream, next_weight=st["n"]["v"], eps=norm.EPS, scales=scales, with_out=True)
    logits = pkg.linear_forward(n.out, st["router"]["w"], st["router"]["b"], out_dtype=F32)
    logits, idx, w = pkg.route(None, None, 4, logits=logits, from_logits=True)
    s = pkg.sort_tokens(n.codes, idx, E, scales=n.scales)
    T4, H = s.rows.shape
    rows = (s.rows.float().view(T4, s.scales.shape[1], -1) * s.scales.float()[:, :, None]).view(T4, H).to(BF16)
    h = pkg.linear_forward(rows, st["up"]["w"], st["up"]["b"], act=pkg.MOE_ACT_SILU)
    y = pkg.linear_forward(h, st["down"]["w"])
    out = pkg.unsort_tokens(y, s.inv_perm, w)
    return stream, n, logits, idx, w, s, rows, h, y, out


def flat(r):
    return [t for v in r for t in (v if isinstance(v, tuple) else (v,)) if t is not None]


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(flat(a), flat(b)))


@pytest.mark.parametrize("scales", ["mx", "row"])
@pytest.mark.parametrize("T", [1, 5, 64, 700])
def test_serving_step(T, scales):
    import mxfp4_expert_layer_gb300 as pkg
    H, E = 288, 32
    st = serving_state(T, H, E, T)
    got = serving_step(st, E, scales)
    stream, n, logits, idx, w, s, rows, h, y, out = got
    linear.check_forward(st["o"], "none", stream, None)
    kept = n.residual.double()
    norm8.check_codes(n.codes, n.scales, kept / norm.ref.rms(kept, norm.EPS) * st["n"]["v"].double())
    linear.check_forward(dict(st["router"], x=n.out), "none", logits, None)
    sort.check_sort(s, n.codes, idx, E, n.scales)
    # the sorted codes stand for what the token's codes stood for, which is y to half a step of 8 bits
    token = (s.perm // 4).long()
    value, wide = norm8.values(n.codes, n.scales)
    assert torch.equal(rows, value[token].to(BF16))
    yv = (kept / norm.ref.rms(kept, norm.EPS) * st["n"]["v"].double())[token]
    assert ((rows.double() - yv).abs() <= (2.0 ** -4 + half_step(BF16) + 80 * U32) * 1.1 * yv.abs() + 2.0 ** -10 * wide[token]).all()
    linear.check_forward(dict(st["up"], x=rows), "silu", h, linear.forward(dict(st["up"], x=rows), "silu", save=True)[1])
    linear.check_forward(dict(st["down"], x=h), "none", y, None)
    sort.check_unsort(out, y, s.inv_perm, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = serving_step(st, E, scales)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(got, again)
    assert pkg.dense_status() == 0


def test_two_graphs_and_eager_calls_at_once():
    """Two captured steps replayed on two streams at one time, and eager calls beside them: no
    workspace is shared."""
    H, E = 288, 32
    states = [serving_state(T, H, E, seed) for T, seed in ((64, 1), (700, 2))]
    want = [serving_step(st, E, "mx") for st in states]
    graphs, got = [], []
    for st in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(serving_step(st, E, "mx"))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = serving_step(states[0], E, "mx")
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1]) and same(eager, want[0])


def test_from_several_threads():
    H, E = 288, 32
    states = [serving_state(T, H, E, seed) for T, seed in ((1, 1), (64, 2), (700, 3), (300, 4))]
    want = [serving_step(st, E, "row") for st in states]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                if not same(serving_step(states[i], E, "row"), want[i]):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(states))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
