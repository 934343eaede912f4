"""GPU parity of the norms around a block (moe_block_norm and its backward) against the
64-bit statement, at the shapes, types, gates and absent arguments that they accept.

Bounds.  A result is one rounding to its type (half a step, relative) of an f32 value
whose own error is a small multiple of 2^-24 of the terms it is formed from: each product
and sum rounds once, a row's sum over at most 1024 threads of 8 values is a chain of 8 and
two butterflies of 5, and rsqrt is good to 2 units.  64 roundings cover the longest chain
(two norms in the backward); the weight gradients add one rounding per row that a block
takes in turn (at most T / 152 + 1 rows, fewer where a block takes several side by side),
per row side by side (15) and per block (152, in eight chains: 19 + 8)."""

import pytest
import torch

from tests import dense_ref as ref
from tests.dense_ref import U32, floor_of, half_step, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def make(T, H, dtype, stream, gate, seed=0, post=True, nxt=True, residual=True, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0, dt=dtype: (torch.randn(*s, generator=g, device=dev) * std + mean).to(dt)  # noqa: E731
    kinds = {"none": lambda: None, "feature": lambda: r(H, std=0.3, mean=0.5),
             "token": lambda: r(T, 1, dt=torch.float32), "full": lambda: r(T, H, std=0.5)}
    return dict(z=r(T, H), r=r(T, H, std=2.0, dt=stream) if residual else None, w=r(H, std=0.25, mean=1.0) if post else None,
                g=kinds[gate](), v=r(H, std=0.25, mean=1.0) if nxt else None, ds=r(T, H, dt=stream), dy=r(T, H) if nxt else None)


def d64(t):
    return None if t is None else t.double()


def forward(m, a, **kw):
    import mxfp4_expert_layer_gb300 as pkg
    return pkg.block_norm(m["z"], m["r"], norm_weight=m["w"], gate=m["g"], residual_scale=a, next_weight=m["v"], eps=EPS, **kw)


def check_forward(m, a, s, y):
    z, r, w, g, v = (d64(m[k]) for k in "zrwgv")
    want, _ = ref.block_norm(z, r, w, g, a, None, EPS)
    branch, _ = ref.block_norm(z.abs(), None if r is None else r.abs(), None if w is None else w.abs(),
                               None if g is None else g.abs(), abs(a), None, EPS)
    within(s, want, half_step(s.dtype) * want.abs() + 32 * U32 * branch + floor_of(s.dtype))
    if m["v"] is not None:  # the next norm is taken of the stored stream
        kept = s.double()
        out = kept / ref.rms(kept, EPS) * v
        within(y, out, (half_step(y.dtype) + 32 * U32) * out.abs() + floor_of(y.dtype))
    else:
        assert y is None


def check_backward(m, a, s, grads):
    z, w, g, v, ds, dy = (d64(m[k]) for k in ("z", "w", "g", "v", "ds", "dy"))
    want, mag = ref.block_norm_grads(ds, dy, z, s.double(), w, g, a, v, EPS)
    T = z.shape[0]
    for name, t in grads._asdict().items():
        if name not in want:
            assert t is None, name
            continue
        chain = 64 + (T / 152 + 43 if name.endswith("weight") or (name == "gate" and m["g"].dim() == 1) else 0)
        within(t, want[name], half_step(t.dtype) * want[name].abs() + chain * U32 * mag[name] + floor_of(t.dtype))


def both(m, a):
    import mxfp4_expert_layer_gb300 as pkg
    s, y = forward(m, a)
    check_forward(m, a, s, y)
    grads = pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"], residual_scale=a,
                                    next_weight=m["v"], eps=EPS, has_residual=m["r"] is not None)
    check_backward(m, a, s, grads) if m["r"] is not None else check_backward(m, a, s, grads._replace(
        residual=(a * ref_ds(m, s)).to(s.dtype)))
    return s, y, grads


def ref_ds(m, s):
    want, _ = ref.block_norm_grads(d64(m["ds"]), d64(m["dy"]), d64(m["z"]), s.double(), d64(m["w"]), d64(m["g"]), 1.0, d64(m["v"]), EPS)
    return want["residual"]


@pytest.mark.parametrize("gate", ["none", "feature", "token", "full"])
@pytest.mark.parametrize("dtype,stream", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                          (torch.bfloat16, torch.float32), (torch.float16, torch.float32)])
@pytest.mark.parametrize("T,H", [(1, 2880), (5, 8), (37, 264), (700, 72)])
def test_shapes_types_gates(T, H, dtype, stream, gate):
    both(make(T, H, dtype, stream, gate, seed=T + H), 0.7)


@pytest.mark.parametrize("T,H", [(1, 8192), (3, 8192), (2, 4104), (1000, 2880), (1, 8), (641, 4096)])
def test_widths_and_row_counts(T, H):
    both(make(T, H, torch.bfloat16, torch.bfloat16, "feature", seed=H), 1.0)


@pytest.mark.parametrize("gate", ["none", "feature", "token", "full"])
@pytest.mark.parametrize("T,H", [(2001, 2880), (1300, 4096), (10007, 264), (18301, 8), (9800, 512)])
def test_many_rows(T, H, gate):
    """Row counts at which the forward's persistent blocks take over (four rows for each
    group of threads on the GPU)."""
    stream = torch.float32 if H == 4096 else torch.bfloat16
    both(make(T, H, torch.bfloat16, stream, gate, seed=T), 0.7)


@pytest.mark.parametrize("T,H,dtype,stream", [(300, 8192, torch.bfloat16, torch.float32), (7, 6000, torch.float16, torch.float16),
                                              (1200, 4104, torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("gate", ["none", "feature", "full"])
def test_rows_wider_than_a_blocks_registers(T, H, dtype, stream, gate):
    both(make(T, H, dtype, stream, gate, seed=H), 0.7)


@pytest.mark.parametrize("post,nxt,residual,gate", [(False, True, True, "none"), (False, True, True, "token"),
                                                    (True, False, True, "full"), (True, True, False, "feature"),
                                                    (False, False, True, "feature"), (False, False, True, "none"),
                                                    (True, False, False, "token")])
def test_absent_arguments(post, nxt, residual, gate):
    both(make(19, 320, torch.bfloat16, torch.bfloat16, gate, seed=3, post=post, nxt=nxt, residual=residual), 0.5)


def test_only_one_incoming_gradient():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(21, 96, torch.float16, torch.float16, "full", seed=5)
    s, _ = forward(m, 1.0)
    m["ds"] = None
    check_backward(m, 1.0, s, pkg.block_norm_backward(None, m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"],
                                                      next_weight=m["v"], eps=EPS))


def test_rows_of_zeros_and_large_values():
    """A zero row has n = 0 and, with a zero residual, y = 0; rows of large and of tiny
    values stay finite and right (their squares stay inside f32)."""
    m = make(6, 512, torch.bfloat16, torch.bfloat16, "feature", seed=6)
    m["z"][0] = 0
    m["r"][0] = 0
    m["z"][1] *= 2.0 ** 50
    m["z"][2] *= 2.0 ** -40
    m["r"][3] *= 2.0 ** 40
    s, y, _ = both(m, 1.0)
    assert not s[0].any() and not y[0].any()


def test_an_infinity_stays_in_its_row():
    m = make(4, 256, torch.bfloat16, torch.bfloat16, "none", seed=7)
    clean = forward(m, 1.0)
    m["z"][2, 5] = float("inf")
    s, y = forward(m, 1.0)
    rows = [0, 1, 3]
    assert torch.equal(s[rows], clean[0][rows]) and torch.equal(y[rows], clean[1][rows])
    assert not torch.isfinite(y[2, 5])


def test_in_place_and_into_given_buffers():
    import mxfp4_expert_layer_gb300 as pkg
    # H / 8 odd: neighbouring rows share a 32-byte sector
    m = make(900, 200, torch.bfloat16, torch.bfloat16, "token", seed=8)
    s, y = forward(m, 0.5)
    r2, z2 = m["r"].clone(), m["z"].clone()
    s2, y2 = pkg.block_norm(z2, r2, norm_weight=m["w"], gate=m["g"], residual_scale=0.5, next_weight=m["v"], eps=EPS,
                            residual_out=r2, out=z2)
    assert s2 is r2 and y2 is z2
    assert torch.equal(s2, s) and torch.equal(y2, y)


def test_rows_behind_the_last_are_left():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(7, 328, torch.bfloat16, torch.bfloat16, "full", seed=9)
    so, yo = (torch.full((9, 328), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkg.block_norm(m["z"], m["r"], norm_weight=m["w"], gate=m["g"], next_weight=m["v"], residual_out=so[:7], out=yo[:7])
    assert (so[7:] == 7).all() and (yo[7:] == 7).all()


def test_backward_repeats_bit_for_bit():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(1500, 512, torch.bfloat16, torch.bfloat16, "feature", seed=10)
    s, _ = forward(m, 1.0)
    runs = [pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"], next_weight=m["v"])
            for _ in range(2)]
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """The kernel's gradients projected on a direction against a central difference of the
    64-bit forward: rounding of the gradients is the only error left (half a step of each
    term; the difference itself is good to 1e-7)."""
    import mxfp4_expert_layer_gb300 as pkg
    m = make(12, 64, torch.float16, torch.float32, "feature", seed=11)
    a = 0.7
    s, _ = forward(m, a)
    z, r, w, g, v, ds, dy = (d64(m[k]) for k in ("z", "r", "w", "g", "v", "ds", "dy"))
    grads = pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"], residual_scale=a,
                                    next_weight=m["v"], eps=EPS)

    def loss(z, r, w, g, v):
        s, y = ref.block_norm(z, r, w, g, a, v, EPS)
        return ((ds * s).sum() + (dy * y).sum()).item()

    args = [z, r, w, g, v]
    for i, grad in enumerate((grads.block, grads.residual, grads.norm_weight, grads.gate, grads.next_weight)):
        direction = torch.randn(args[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                                dtype=torch.float64)
        h = 1e-4
        up, down = (loss(*[t + sign * h * direction if j == i else t for j, t in enumerate(args)]) for sign in (1, -1))
        got = (grad.double() * direction).sum().item()
        tol = (half_step(grad.dtype) + 200 * U32) * (grad.double().abs() * direction.abs()).sum().item() + 1e-5
        assert abs(got - (up - down) / (2 * h)) <= tol, i


def test_captured_and_on_a_side_stream():
    import mxfp4_expert_layer_gb300 as pkg
    m = make(300, 1024, torch.bfloat16, torch.bfloat16, "full", seed=12)
    s, y = forward(m, 1.0)
    call = lambda: pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"],  # noqa: E731
                                           next_weight=m["v"])
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2 = forward(m, 1.0)
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out2[0], s) and torch.equal(out2[1], y)
    graphs = []
    for _ in range(2):  # two graphs replayed together: each holds its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = forward(m, 1.0), call()
        graphs.append((graph, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for (graph, _), st in zip(graphs, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for _, ((s2, y2), got) in graphs:
        assert torch.equal(s2, s) and torch.equal(y2, y)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
