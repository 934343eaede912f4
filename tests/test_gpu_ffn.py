"""GPU parity of the dense gated feed-forward block (moe_ffn_forward, moe_ffn_backward)
against the 64-bit statement.

Bounds.  A product of K terms on the tensor cores is off by at most (K / 16 + 8) steps of
2^-22 of its terms' magnitude (each step adds 16 aligned products; splitting K or the
order changes nothing in that count).  h, dg and du are rounded to the 16-bit type (half a
step each) before the next product, and the result once more.  act has a slope within
1.2 and its f32 evaluation 16 roundings; act' changes by at most 1.2 per unit of g
(0.5 for SiLU, 0.8 + for GELU), g itself being off by its product's bound."""

import pytest
import torch

from tests import dense_ref as ref
from tests.dense_ref import U32, floor_of, half_step, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def make(T, H, I, dtype, seed=0, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(dtype)  # noqa: E731
    return dict(x=r(T, H), wgu=r(2 * I, H, std=H ** -0.5), wd=r(H, I, std=I ** -0.5), dy=r(T, H))


def step(K):
    return 4 * U32 * (K / 16 + 8)


def check(m, act="silu", backward=True):
    import mxfp4_expert_layer_gb300 as pkg
    code = pkg.MOE_ACT_SILU if act == "silu" else pkg.MOE_ACT_GELU
    dt = m["x"].dtype
    hs, fl = half_step(dt), floor_of(dt)
    x, wgu, wd, dy = (m[k].double() for k in ("x", "wgu", "wd", "dy"))
    (T, H), I = x.shape, wd.shape[1]
    out, gu = pkg.ffn_forward(m["x"], m["wgu"], m["wd"], act=code, save=True)
    want_gu, e_gu = x @ wgu.t(), step(H) * (x.abs() @ wgu.t().abs())
    within(gu, want_gu, e_gu + U32 * want_gu.abs())
    g, u, eg, eu = want_gu[:, :I], want_gu[:, I:], e_gu[:, :I], e_gu[:, I:]
    g = g.clone().requires_grad_()
    a = ref.act(g, act)
    slope = torch.autograd.grad(a.sum(), g)[0]
    a, g = a.detach(), g.detach()
    ea = 1.2 * eg + 16 * U32 * (a.abs() + g.abs())
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu
    eh = eh + hs * (h.abs() + eh) + fl
    want = h @ wd.t()
    tol = eh @ wd.t().abs() + step(I) * (h.abs() @ wd.t().abs())
    within(out, want, tol + hs * (want.abs() + tol) + fl)
    assert torch.equal(pkg.ffn_forward(m["x"], m["wgu"], m["wd"], act=code), out)
    if backward:
        grads = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"], act=code)
        dh, edh = dy @ wd, step(H) * (dy.abs() @ wd.abs())
        es = 1.2 * eg + 16 * U32 * (1 + g.abs())
        dg, du = dh * u * slope, dh * a
        edg = edh * (u * slope).abs() + dh.abs() * (eu * slope.abs() + u.abs() * es) + 4 * U32 * dg.abs()
        edu = edh * a.abs() + dh.abs() * ea + 4 * U32 * du.abs()
        dgu = torch.cat((dg, du), 1)
        edgu = torch.cat((edg, edu), 1)
        edgu = edgu * (1 + hs) + hs * dgu.abs() + fl
        for got, A, B, eA, eB, K in ((grads.x, dgu, wgu, edgu, None, 2 * I), (grads.w_gateup, dgu.t(), x, edgu.t(), None, T),
                                     (grads.w_down, dy.t(), h, None, eh, T)):
            want = A @ B
            tol = step(K) * (A.abs() @ B.abs())
            tol = tol + (eA @ B.abs() if eA is not None else A.abs() @ eB)
            within(got, want, tol + hs * (want.abs() + tol) + fl)
    assert pkg.dense_status() == 0
    return out, gu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16])
def test_few_tokens(T, dtype, act):
    check(make(T, 200, 328, dtype, seed=T), act, backward=T in (1, 9))


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (2, 2880, 2880), (16, 64, 10000), (5, 4104, 72), (1, 8, 20000), (7, 24, 16)])
def test_few_token_shapes(T, H, I):
    check(make(T, H, I, torch.bfloat16, seed=H + I), backward=T == 7)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,I", [(17, 64, 64), (64, 8, 8), (100, 200, 328), (129, 136, 72), (300, 1000, 520)])
def test_small_tiles(T, H, I, dtype, act):
    """One-SM tiles, odd edges in every direction, K tails, split K."""
    check(make(T, H, I, dtype, seed=T + H), act)


@pytest.mark.parametrize("T,H,I,act", [(1001, 2880, 2880, "gelu"), (2048, 1024, 1032, "silu"), (257, 4104, 4096, "silu"),
                                       (4096, 264, 3000, "silu"), (1500, 2880, 1448, "silu")])
def test_pair_tiles(T, H, I, act):
    """Tiles on pairs of SMs, several rounds of the persistent schedule, odd edges."""
    check(make(T, H, I, torch.bfloat16, seed=T), act)


def test_split_k_and_many_tokens_of_a_thin_block():
    check(make(64, 4096, 1024, torch.float16, seed=1))
    check(make(40, 256, 16384, torch.bfloat16, seed=2), backward=False)
    check(make(3000, 72, 40, torch.bfloat16, seed=3))


def test_values_far_from_zero():
    """Saturated gates both ways: act(g) = g or (nearly) 0, no overflow in e^-g."""
    m = make(130, 128, 136, torch.bfloat16, seed=4)
    m["wgu"] *= 60
    check(m, "silu")
    check(m, "gelu")


def test_an_infinity_stays_in_its_token():
    import mxfp4_expert_layer_gb300 as pkg
    for T in (5, 140):
        m = make(T, 128, 136, torch.bfloat16, seed=5)
        clean = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
        m["x"][3, 7] = float("nan")
        y = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
        keep = [i for i in range(T) if i != 3]
        assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[3]).all()


def test_rows_behind_the_last_and_gradients_asked_for():
    import mxfp4_expert_layer_gb300 as pkg
    for T in (7, 150):
        m = make(T, 136, 264, torch.bfloat16, seed=6)
        out = torch.full((T + 3, 136), 5.0, dtype=torch.bfloat16, device="cuda")
        _, gu = pkg.ffn_forward(m["x"], m["wgu"], m["wd"], out=out[:T], save=True)
        assert (out[T:] == 5).all()
        both = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"])
        only_x = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"], need_weights=False)
        only_w = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"], need_x=False)
        assert torch.equal(only_x.x, both.x) and only_x.w_gateup is None and only_x.w_down is None
        assert only_w.x is None and torch.equal(only_w.w_gateup, both.w_gateup) and torch.equal(only_w.w_down, both.w_down)


def test_gradients_against_differences():
    """Projections of the kernel's gradients against central differences of the 64-bit
    forward: dg, du and h are rounded once and the gradient once, half a step each."""
    import mxfp4_expert_layer_gb300 as pkg
    m = make(24, 64, 72, torch.float16, seed=7)
    _, gu = pkg.ffn_forward(m["x"], m["wgu"], m["wd"], save=True)
    grads = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"])
    args = [m[k].double() for k in ("x", "wgu", "wd")]
    dy = m["dy"].double()

    def loss(x, wgu, wd):
        g, u = (x @ wgu.t()).split(72, 1)
        return (dy * ((ref.act(g, "silu") * u) @ wd.t())).sum().item()

    for i, grad in enumerate(grads):
        d = torch.randn(args[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                        dtype=torch.float64)
        h = 1e-4
        up, down = (loss(*[t + s * h * d if j == i else t for j, t in enumerate(args)]) for s in (1, -1))
        # magnitude of the terms that were rounded: the product with absolute operands
        (x, wgu, wd), gu64 = args, args[0] @ args[1].t()
        g, u = gu64[:, :72].requires_grad_(), gu64[:, 72:].requires_grad_()
        hh = ref.act(g, "silu") * u
        dg, du = torch.autograd.grad(hh, (g, u), dy @ wd)
        dgu, hh = torch.cat((dg, du), 1).abs(), hh.detach().abs()
        mag = (dgu @ wgu.abs(), dgu.t() @ x.abs(), dy.t().abs() @ hh)[i]
        tol = (2.5 * half_step(torch.float16) * mag * d.abs()).sum().item() + 1e-5
        assert abs((grad.double() * d).sum().item() - (up - down) / (2 * h)) <= tol, i


def test_captured_twice_and_on_side_streams():
    import mxfp4_expert_layer_gb300 as pkg
    for T in (4, 70, 600):
        m = make(T, 512, 1024, torch.bfloat16, seed=8)

        def step_():
            out, gu = pkg.ffn_forward(m["x"], m["wgu"], m["wd"], save=True)
            return (out,) + tuple(pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"]))

        want = step_()
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step_()
            graphs.append((graph, got))
        streams = [torch.cuda.Stream() for _ in graphs]
        for (graph, _), s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    assert pkg.dense_status() == 0


def test_waits_that_give_up_are_reported():
    """With a 1 ns limit the pipeline's waits give up on an ordinary call: the status word
    says so, the blocks drain and leave, and the next call is right."""
    import mxfp4_expert_layer_gb300 as pkg
    from mxfp4_expert_layer_gb300 import _lib as L
    m = make(600, 512, 1024, torch.bfloat16, seed=9)
    want = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    assert pkg.dense_status() == 0
    assert L.moe_set_wait_limit_ns(1) == L.MOE_OK
    try:
        pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
        torch.cuda.synchronize()
    finally:
        assert L.moe_set_wait_limit_ns(0) == L.MOE_OK
    st = pkg.dense_status()
    assert st != 0 and st & ~0b111 == 0
    assert pkg.dense_status() == 0
    assert torch.equal(pkg.ffn_forward(m["x"], m["wgu"], m["wd"]), want)
