"""GPU parity of projections (moe_linear_forward, moe_linear_backward) against the 64-bit
statement.

Bounds.  A product of K terms on the tensor cores is off by at most (K / 16 + 8) steps of 2^-22
of its terms' magnitude (each step adds 16 aligned products, cut below the largest; splitting K
or the order changes nothing in that count); bias, activation and residual add 20 roundings of
2^-24 of what they are formed from, the result is rounded once.  act has a slope within 1.2, its
derivative one within 1.2.  dp is rounded to the 16-bit type before the products, and summed over
t unrounded: a chain of T / 8 terms for each of 8 warps and at most 256 partial sums."""

import pytest
import torch

from tests import dense_ref as ref
from tests.dense_ref import U32, floor_of, half_step, within

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = {"none": 2, "silu": 0, "gelu": 1}


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def make(T, K, N, dtype, out=None, bias=True, residual=True, seed=0, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s, std=1.0, dt=dtype: (torch.randn(*s, generator=g, device=dev) * std).to(dt)  # noqa: E731
    out = out or dtype
    return dict(x=r(T, K), w=r(N, K, std=K ** -0.5), b=r(N, std=0.5, dt=F32) if bias else None,
                r=r(T, N, std=2.0, dt=out) if residual else None, d=r(T, N, dt=out))


def step(K):
    return 4 * U32 * (K / 16 + 8)


def act64(v, act):
    return v if act == "none" else ref.act(v, act)


def forward(m, act="none", **kw):
    import mxfp4_expert_layer_gb300 as pkg
    return pkg.linear_forward(m["x"], m["w"], m["b"], m["r"], act=ACTS[act], out_dtype=m["d"].dtype, **kw)


def check_forward(m, act, out, pre):
    x, w = m["x"].double(), m["w"].double()
    want, e = x @ w.t(), step(x.shape[1]) * (x.abs() @ w.t().abs())
    if m["b"] is not None:
        want, e = want + m["b"].double(), e + U32 * (want.abs() + m["b"].double().abs())
    if act == "none":
        assert pre is None
    else:
        within(pre, want, e + U32 * want.abs())
    v = act64(want, act)
    ev = e if act == "none" else 1.2 * e + 16 * U32 * (v.abs() + want.abs())
    if m["r"] is not None:
        v = v + m["r"].double()
        ev = ev + 2 * U32 * (v.abs() + m["r"].double().abs())
    assert out.dtype == m["d"].dtype
    within(out, v, ev + half_step(out.dtype) * (v.abs() + ev) + floor_of(out.dtype))


def check_backward(m, act, pre, grads):
    x, w, d = (m[k].double() for k in "xwd")
    (T, K), N, dt = x.shape, w.shape[0], m["x"].dtype
    hs, fl = half_step(dt), floor_of(dt)
    if act == "none":
        dp, e = d, torch.zeros_like(d)
    else:
        p = pre.double().requires_grad_()
        (slope,) = torch.autograd.grad(act64(p, act).sum(), p)
        dp, e = d * slope, d.abs() * 20 * U32 * (1 + p.detach().abs())
    if grads.bias is not None:
        chain = T / 8 + 8 + 256
        within(grads.bias, dp.sum(0), (e + chain * U32 * dp.abs()).sum(0) + floor_of(F32))
    if not (act == "none" and m["d"].dtype == dt):
        e = e * (1 + hs) + hs * dp.abs() + fl
    for got, A, eA, B, n in ((grads.x, dp, e, w, N), (grads.weight, dp.t(), e.t(), x, T)):
        if got is None:
            continue
        want = A @ B
        tol = step(n) * (A.abs() @ B.abs()) + eA @ B.abs()
        within(got, want, tol + hs * (want.abs() + tol) + fl)


def check(m, act="none", backward=True):
    import mxfp4_expert_layer_gb300 as pkg
    out, pre = forward(m, act, save=True)
    check_forward(m, act, out, pre)
    assert torch.equal(forward(m, act), out)
    if backward:
        grads = pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=ACTS[act])
        check_backward(m, act, pre, grads)
    assert pkg.dense_status() == 0
    return out, pre


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16])
def test_few_tokens(T, dtype, out, act):
    check(make(T, 200, 328, dtype, out, seed=T), act, backward=T in (1, 9))


@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (2, 2880, 2880), (16, 64, 10000), (5, 4104, 72), (1, 20000, 8), (7, 24, 16),
                                   (1, 131072, 24), (16, 8, 1048576)])
def test_few_token_shapes(T, K, N):
    check(make(T, K, N, BF16, seed=K + N), backward=T == 7)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("T,K,N", [(17, 64, 64), (64, 8, 8), (100, 200, 328), (129, 136, 72), (300, 1000, 520)])
def test_small_tiles(T, K, N, dtype, out, act):
    """One-SM tiles, odd edges in every direction, K tails, split K."""
    check(make(T, K, N, dtype, out, seed=T + K), act)


@pytest.mark.parametrize("act,residual", [("none", True), ("gelu", False), ("silu", True)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("T,K,N", [(24, 64, 128), (32, 8, 8), (17, 520, 136), (33, 1096, 520), (61, 1160, 264), (64, 4096, 2880),
                                   (48, 1088, 20000), (100, 2880, 328), (128, 4104, 4096), (65, 16384, 136), (5, 72, 5000),
                                   (16, 14344, 512), (1, 72, 16400)])
def test_batches(T, K, N, dtype, out, act, residual):
    """Blocks of 128 weight rows: every width of the token side, K whole and cut in two to eight
    (by short K, by many rows), tokens that do not divide by the cut, partial blocks of rows."""
    check(make(T, K, N, dtype, out, residual=residual, seed=T + N), act, backward=False)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("T,K,N", [(24, 128, 64), (32, 8, 8), (1, 136, 520), (33, 520, 1096), (61, 264, 1160), (64, 2880, 4096),
                                   (48, 20000, 1088), (100, 328, 2880), (128, 4096, 4104), (65, 136, 16384), (5, 5000, 72)])
def test_gradients_of_batches(T, K, N, dtype, out, act):
    """The same sizes, with K and N changed, for the gradient into x."""
    check(make(T, K, N, dtype, out, seed=T + N), act)


@pytest.mark.parametrize("T,K,N,act,out", [(1001, 2880, 2880, "gelu", BF16), (2048, 1024, 1032, "silu", F32),
                                           (257, 4104, 4096, "none", F32), (4096, 264, 3000, "gelu", BF16),
                                           (1500, 2880, 1448, "none", BF16)])
def test_pair_tiles(T, K, N, act, out):
    """Tiles on pairs of SMs, several rounds of the persistent schedule, odd edges."""
    check(make(T, K, N, BF16, out, seed=T), act)


@pytest.mark.parametrize("out", [BF16, F32])
def test_split_k(out):
    check(make(64, 16384, 1024, BF16, out, seed=1), "silu")
    check(make(40, 30000, 264, BF16, out, seed=2), "none", backward=False)
    check(make(150, 16384, 1024, BF16, out, seed=4), "silu", backward=False)
    check(make(200, 8192, 136, BF16, out, seed=5), "gelu", backward=False)
    check(make(3000, 72, 40, BF16, out, seed=3), "gelu")


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("T,K,N", [(5, 136, 200), (70, 136, 200), (700, 520, 1032), (64, 16384, 1024)])
def test_absent_arguments(T, K, N, bias, residual):
    for act in ("none", "gelu"):
        check(make(T, K, N, F16, bias=bias, residual=residual, seed=N), act, backward=T == 70)


@pytest.mark.parametrize("T,K,N", [(1, 136, 200), (16, 520, 1000), (70, 136, 200), (700, 520, 1032), (64, 16384, 1024),
                                   (2048, 264, 4096), (40, 264, 1000), (100, 4096, 520), (80, 30000, 2000)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_onto_the_residual(T, K, N, out):
    """out may be the residual: the same bits as apart."""
    m = make(T, K, N, BF16, out, seed=T)
    want = forward(m, "silu")
    got = forward(m, "silu", out=m["r"])
    assert got.data_ptr() == m["r"].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("T,K,N", [(9, 64, 200), (200, 264, 136)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_any_gradient_alone(T, K, N, act):
    import mxfp4_expert_layer_gb300 as pkg
    for out in (BF16, F32):
        m = make(T, K, N, BF16, out, seed=4)
        _, pre = forward(m, act, save=True)
        every = pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=ACTS[act])
        for i in range(3):
            need = [j == i for j in range(3)]
            some = pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=ACTS[act], need_x=need[0], need_weight=need[1],
                                       need_bias=need[2])
            for j in range(3):
                assert (some[j] is not None) == need[j]
            check_backward(m, act, pre, some)
            if i == 2:
                assert torch.equal(some.bias, every.bias)


def test_gradient_against_differences():
    """f(x, w, b) = <d, act(x w^T + b)> in 64 bits at the 16-bit inputs."""
    import mxfp4_expert_layer_gb300 as pkg
    for act in ACTS:
        m = make(20, 16, 24, F16, F32, residual=False, seed=5)
        _, pre = forward(m, act, save=True)
        grads = pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=ACTS[act])
        x, w, b, d = (m[k].double() for k in "xwbd")
        h = 1e-4
        for t, g in ((x, grads.x), (w, grads.weight), (b, grads.bias)):
            mag = float(g.double().abs().max())
            for i in range(0, t.numel(), max(1, t.numel() // 20)):
                keep, f = t.view(-1)[i].item(), []
                for v in (keep + h, keep - h):
                    t.view(-1)[i] = v
                    f.append(float((d * act64(x @ w.t() + b, act)).sum()))
                t.view(-1)[i] = keep
                # h^2 / 6 of a third derivative below 100; dp and the result rounded to f16: their sum over 24 or 20
                # terms of at most 8 each, 2^-11 of it, and of the largest gradient
                assert abs((f[0] - f[1]) / (2 * h) - g.view(-1)[i].item()) < 1e-6 + 2 ** -11 * (24 * 8 + mag)


def test_not_finite_values_stay_in_their_rows_and_columns():
    import mxfp4_expert_layer_gb300 as pkg
    for T in (4, 70, 300):
        m = make(T, 72, 200, BF16, seed=6)
        m["x"][2, 5], m["b"][17], m["r"][3, 40] = float("nan"), float("inf"), float("-inf")
        out = forward(m, "none").float()
        bad = ~torch.isfinite(out)
        want = torch.zeros_like(bad)
        want[2], want[:, 17], want[3, 40] = True, True, True
        assert torch.equal(bad, want) and out[0, 17] == float("inf") and out[3, 40] == float("-inf")
        m = make(T, 72, 200, BF16, seed=7)
        m["d"][1, 9] = float("nan")
        g = pkg.linear_backward(m["d"], m["x"], m["w"])
        for t, row in ((g.x, 1), (g.weight, 9), (g.bias, 9)):
            bad = ~torch.isfinite(t.float())
            want = torch.zeros_like(bad)
            want[row] = True
            assert torch.equal(bad, want)


@pytest.mark.parametrize("T,K,N", [(4, 264, 520), (64, 4096, 1024), (300, 264, 1032)])
def test_captured_other_streams_and_repeats(T, K, N):
    import mxfp4_expert_layer_gb300 as pkg

    def step(m):
        out, pre = forward(m, "gelu", save=True)
        return (out, pre) + tuple(pkg.linear_backward(m["d"], m["x"], m["w"], pre, act=1))
    held = make(T, K, N, BF16, seed=1)
    step(held)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(held)
    side = torch.cuda.Stream()
    for seed in (2, 3):
        new = make(T, K, N, BF16, seed=seed)
        for k in held:
            held[k].copy_(new[k])
        graph.replay()
        eager = step(new)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step(new)
        torch.cuda.current_stream().wait_stream(side)
        for a, b, c in zip(captured, eager, other):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(20, 64, 32, BF16, seed=8)
    x, w, b, r, d = (m[k] for k in "xwbrd")
    pre = d.float()
    for call in (lambda: pkg.linear_forward(x, w.half()), lambda: pkg.linear_forward(x, w[:, :32]),
                 lambda: pkg.linear_forward(x, w, b.to(BF16)), lambda: pkg.linear_forward(x, w, b[:8]),
                 lambda: pkg.linear_forward(x, w, b, r.half()), lambda: pkg.linear_forward(x, w, b, r[:10]),
                 lambda: pkg.linear_forward(x, w, b, r.float(), out_dtype=BF16), lambda: pkg.linear_forward(x.float(), w),
                 lambda: pkg.linear_forward(x, w, out_dtype=F16), lambda: pkg.linear_forward(x, w, out=r.half()),
                 lambda: pkg.linear_forward(x.t(), w), lambda: pkg.linear_forward(x, w.t().contiguous().t()),
                 lambda: pkg.linear_backward(d.half(), x, w), lambda: pkg.linear_backward(d, x, w, pre.to(BF16), act=1),
                 lambda: pkg.linear_backward(d[:10], x, w)):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(20, 32, dtype=F32, device="cuda")
    for call in (lambda: pkg.linear_forward(x, w, act=3), lambda: pkg.linear_forward(x[:0], w),
                 lambda: pkg.linear_forward(make(20, 60, 32, BF16)["x"], make(20, 60, 32, BF16)["w"]),
                 lambda: pkg.linear_forward(x, w[:12]), lambda: pkg.linear_forward(x, w, out=x.view(-1)[:640].view(20, 32)),
                 lambda: pkg.linear_backward(d, x, w, pre), lambda: pkg.linear_backward(d, x, w, act=1),
                 lambda: pkg.linear_backward(d, x, w, wide, act=3),
                 lambda: pkg.linear_backward(d, x, w, need_x=False, need_weight=False, need_bias=False)):
        with pytest.raises(pkg._lib.MoEError):
            call()
    check(m)


def test_more_than_2_31_elements():
    """out beyond 2^31 elements, in f32 with pre: byte offsets beyond 2^33."""
    import mxfp4_expert_layer_gb300 as pkg
    T, K, N = 16500, 64, 131080
    m = make(T, K, N, BF16, F32, residual=False, seed=9)
    out, pre = forward(m, "silu", save=True)
    for part in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        check_forward(dict(m, x=m["x"][part], r=None), "silu", out[part], pre[part])
    d = m["d"]
    del out
    grads = pkg.linear_backward(d, m["x"], m["w"], pre, act=0)
    x, w, hs = m["x"].double(), m["w"].double(), half_step(BF16)
    cols = slice(N - 200, N)
    p = pre[:, cols].double().requires_grad_()
    (slope,) = torch.autograd.grad(act64(p, "silu").sum(), p)
    dp = d[:, cols].double() * slope
    e = d[:, cols].double().abs() * 20 * U32 * (1 + p.detach().abs())
    within(grads.bias[cols], dp.sum(0), (e + (T / 8 + 264) * U32 * dp.abs()).sum(0))
    e = e * (1 + hs) + hs * dp.abs()
    want = dp.t() @ x
    tol = step(T) * (dp.t().abs() @ x.abs()) + e.t() @ x.abs()
    within(grads.weight[cols], want, tol + hs * (want.abs() + tol))
