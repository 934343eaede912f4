"""The dense operators as a decoder uses them, each stage against the 64-bit statement on
its own inputs: a decode step's half layer (norms around a block, MoE layer and shared
feed-forward block side by side, MXFP4 projection), and a training step through two norms
and a feed-forward block.  Further: calls in place, from several threads and in captured
graphs, and what the Python entry points refuse."""

import threading

import pytest
import torch

from synthetic import make_layer
from tests import test_gpu_block_norm as norm
from tests import test_gpu_ffn as ffn
from tests import test_gpu_matvec as matvec
from tests.dense_ref import half_step, within
from tests.gpu_helpers import build_layer

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.mark.parametrize("T", [1, 6, 24, 64])
def test_half_layer_of_a_decode_step(T):
    """y = norm of the stream after attention; experts and a shared block of y; the stream
    after both; its norm through an MXFP4 projection, and through a gated one.  Eager and
    captured runs give the same bits."""
    import mxfp4_expert_layer_gb300 as pkg
    H, I = 512, 384
    a = norm.make(T, H, BF16, BF16, "feature", seed=T)
    b = norm.make(T, H, BF16, BF16, "token", seed=T + 1)
    w = ffn.make(T, H, I, BF16, seed=T + 2)
    layer = build_layer(make_layer(T=T, H=H, I=256, E=8, k=2, seed=T))
    head = matvec.make(T, 1000, H, BF16, seed=T + 3)
    lm = pkg.MatvecMXFP4(head["codes"], head["scales"], bias=head["bias"])
    gated = pkg.MatvecMXFP4(head["codes"], head["scales"], kind=pkg.MOE_WEIGHTS_GATEUP, bias=head["bias"])

    def step():
        s0, y0 = pkg.block_norm(a["z"], a["r"], norm_weight=a["w"], gate=a["g"], residual_scale=0.7, next_weight=a["v"],
                                eps=norm.EPS)
        both = layer(y0) + pkg.ffn_forward(y0, w["wgu"], w["wd"])
        s1, y1 = pkg.block_norm(both, s0, norm_weight=b["w"], gate=b["g"], residual_scale=1.0, next_weight=b["v"],
                                eps=norm.EPS)
        return s0, y0, both, s1, y1, lm(y1), gated(y1)

    s0, y0, both, s1, y1, logits, h = got = step()
    norm.check_forward(a, 0.7, s0, y0)
    ffn.check(dict(w, x=y0), backward=False)
    norm.check_forward(dict(b, z=both, r=s0), 1.0, s1, y1)
    within(logits, *matvec.expect(dict(head, x=y1), False))
    within(h, *matvec.expect(dict(head, x=y1), True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, again):
        assert torch.equal(x, y)
    assert pkg.dense_status() == 0


@pytest.mark.parametrize("T,dtype,stream", [(9, torch.float16, torch.float16), (150, BF16, torch.float32),
                                            (1300, BF16, BF16)])
def test_training_step(T, dtype, stream):
    """norm -> feed-forward -> norm, and the gradients back through all three: each operator
    gets what the one before it gave, and is held to its own bound on that."""
    import mxfp4_expert_layer_gb300 as pkg
    H, I = 264, 520
    one, two = (norm.make(T, H, dtype, stream, gate, seed=i) for i, gate in ((1, "full"), (2, "feature")))
    w = ffn.make(T, H, I, dtype, seed=3)
    s1, y1 = norm.forward(one, 0.7)
    out, gu = pkg.ffn_forward(y1, w["wgu"], w["wd"], save=True)
    two = dict(two, z=out, r=s1)
    s2, _ = norm.forward(two, 1.0)
    g2 = pkg.block_norm_backward(two["ds"], two["dy"], out, s2, norm_weight=two["w"], gate=two["g"], residual_scale=1.0,
                                 next_weight=two["v"], eps=norm.EPS)
    norm.check_backward(two, 1.0, s2, g2)
    ffn.check(dict(w, x=y1, dy=g2.block))
    gf = pkg.ffn_backward(g2.block, y1, gu, w["wgu"], w["wd"])
    one = dict(one, ds=g2.residual, dy=gf.x)
    g1 = pkg.block_norm_backward(one["ds"], one["dy"], one["z"], s1, norm_weight=one["w"], gate=one["g"],
                                 residual_scale=0.7, next_weight=one["v"], eps=norm.EPS)
    norm.check_backward(one, 0.7, s1, g1)
    assert pkg.dense_status() == 0


@pytest.mark.parametrize("T,H,I", [(1040, 264, 520),    # 2 I = T: one class of products
                                   (2000, 520, 136),    # the weights' products have the longer sums
                                   (20, 2880, 2880), (300, 2048, 1000), (700, 4104, 72)])
def test_gradient_products_of_one_launch(T, H, I):
    """Sizes at which the three products of the backward differ in which is longest, how
    many tiles each has and how its last round fills; and any of them left out."""
    import mxfp4_expert_layer_gb300 as pkg
    m = ffn.make(T, H, I, BF16, seed=T + I)
    _, gu = ffn.check(m)
    every = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"])
    for need_x, need_w in ((True, False), (False, True)):
        some = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"], need_x=need_x, need_weights=need_w)
        for got, want, asked in zip(some, every, (need_x, need_w, need_w)):
            assert (got is not None) == asked
            if asked:  # the sums' order may differ by the split of K: two roundings of the f32 sum's bound
                got, want = got.double(), want.double()
                assert (got - want).norm() <= 2 * half_step(BF16) * want.norm()


@pytest.mark.parametrize("T,H,gate", [(2001, 2880, "feature"), (1300, 4096, "full"), (10007, 264, "token"), (40, 8192, "none")])
def test_norms_in_place(T, H, gate):
    """The persistent kernels bring rows in ahead of the ones they write: in place, forward
    and backward, they give the same bits."""
    import mxfp4_expert_layer_gb300 as pkg
    from mxfp4_expert_layer_gb300 import _lib as L
    m = norm.make(T, H, BF16, BF16, gate, seed=T)
    s, y = norm.forward(m, 0.7)
    z, r = m["z"].clone(), m["r"].clone()
    s2, y2 = pkg.block_norm(z, r, norm_weight=m["w"], gate=m["g"], residual_scale=0.7, next_weight=m["v"], eps=norm.EPS,
                            residual_out=r, out=z)
    assert s2 is r and y2 is z and torch.equal(r, s) and torch.equal(z, y)
    want = pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"], residual_scale=0.7,
                                   next_weight=m["v"], eps=norm.EPS)
    z, ds = m["z"].clone(), m["ds"].clone()
    dw, dv = (torch.empty(H, device="cuda") for _ in range(2))
    dg = None if m["g"] is None else torch.empty(m["g"].shape, device="cuda",
                                                 dtype=BF16 if gate == "full" else torch.float32)
    nbytes = L.moe_block_norm_workspace_bytes(T, H)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    kind = {"none": L.MOE_GATE_NONE, "feature": L.MOE_GATE_FEATURE, "token": L.MOE_GATE_TOKEN, "full": L.MOE_GATE_FULL}[gate]
    L.check("moe_block_norm_backward", L.moe_block_norm_backward(
        p(ds), p(m["dy"]), p(z), p(m["w"]), p(m["g"]), kind, p(s), 0.7, p(m["v"]), norm.EPS, T, H, L.MOE_DTYPE_BF16,
        L.MOE_DTYPE_BF16, p(z), p(ds), p(dw), p(dg), p(dv), p(ws), nbytes, torch.cuda.current_stream().cuda_stream))
    for got, exp in zip((z, ds, dw, dg, dv), want):
        assert (got is None and exp is None) or torch.equal(got, exp)


def test_calls_from_two_threads():
    """Two threads, each on its own stream, call every operator at once on its own data."""
    import mxfp4_expert_layer_gb300 as pkg
    jobs = []
    for i in range(2):
        n = norm.make(300, 520, BF16, BF16, "feature", seed=i)
        f = ffn.make(200, 520, 328, BF16, seed=i)
        v = matvec.make(20, 500, 1024, BF16, seed=i)
        jobs.append((n, f, v, pkg.MatvecMXFP4(v["codes"], v["scales"], bias=v["bias"])))

    def run(job):
        n, f, v, lin = job
        s, y = norm.forward(n, 0.7)
        g = pkg.block_norm_backward(n["ds"], n["dy"], n["z"], s, norm_weight=n["w"], gate=n["g"], residual_scale=0.7,
                                    next_weight=n["v"], eps=norm.EPS)
        out, gu = pkg.ffn_forward(f["x"], f["wgu"], f["wd"], save=True)
        return (s, y, *g, out, *pkg.ffn_backward(f["dy"], f["x"], gu, f["wgu"], f["wd"]), lin(v["x"]))

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = run(jobs[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert pkg.dense_status() == 0


@pytest.mark.parametrize("T", [3, 20, 64])
def test_projection_captured_twice(T):
    """Two graphs of one handle replay at once: each holds its own workspace."""
    import mxfp4_expert_layer_gb300 as pkg
    m = matvec.make(T, 2000, 2880, BF16, seed=T)
    w = pkg.MatvecMXFP4(m["codes"], m["scales"], bias=m["bias"])
    xs = [m["x"], m["x"].flip(0).contiguous()]
    want = [w(x) for x in xs]
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = w(x)
        graphs.append((graph, y, torch.cuda.Stream()))
    for graph, _, s in graphs:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                graph.replay()
    torch.cuda.synchronize()
    for (_, y, _), exp in zip(graphs, want):
        assert torch.equal(y, exp)


def test_inputs_away_from_their_storage_start():
    """Rows further into an allocation (16-byte aligned, not 32) and odd row pitches in
    sectors: the wide accesses fall back where they have to."""
    import mxfp4_expert_layer_gb300 as pkg

    def shifted(t):
        flat = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
        at = 16 // t.element_size()
        view = flat[at:at + t.numel()].view(t.shape)
        view.copy_(t)
        return view

    n = {k: shifted(v) for k, v in norm.make(33, 1000, BF16, BF16, "full", seed=1).items()}
    norm.both(n, 0.7)
    for T in (5, 40, 400):
        m = {k: shifted(v) for k, v in ffn.make(T, 264, 136, BF16, seed=T).items()}
        plain = {k: v.clone() for k, v in m.items()}
        gu = shifted(torch.empty(T, 272, device="cuda"))
        out, gu0 = ffn.check(m)
        gu.copy_(gu0)
        a = pkg.ffn_backward(m["dy"], m["x"], gu, m["wgu"], m["wd"])
        b = pkg.ffn_backward(plain["dy"], plain["x"], gu0, plain["wgu"], plain["wd"])
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    v = matvec.make(12, 400, 512, BF16, seed=2)
    v.update(codes=shifted(v["codes"]), x=shifted(v["x"]))
    matvec.check(v, False)


def test_refusals():
    """What an entry point cannot take is refused before anything is launched."""
    import mxfp4_expert_layer_gb300 as pkg
    n = norm.make(4, 64, BF16, BF16, "feature", seed=1)
    s, _ = norm.forward(n, 1.0)
    call = dict(norm_weight=n["w"], gate=n["g"], next_weight=n["v"])
    wide = torch.randn(4, 128, device="cuda", dtype=BF16)
    for bad, kw in ((dict(block=n["z"][:, :63]), {}), (dict(block=wide[:, ::2]), {}), (dict(block=n["z"].float()), {}),
                    (dict(block=n["z"].cpu()), {}), (dict(block=n["z"][0]), {}), (dict(residual=n["r"][:3]), {}),
                    (dict(residual=n["r"].half()), {}), ({}, dict(norm_weight=n["w"][:32])), ({}, dict(gate=n["g"].float())),
                    ({}, dict(gate=torch.ones(4, 1, device="cuda", dtype=BF16))), ({}, dict(residual_out=s.float())),
                    ({}, dict(out=s[:2])), ({}, dict(next_weight=None, out=s))):
        args = dict(block=n["z"], residual=n["r"])
        args.update(bad)
        with pytest.raises(ValueError):
            pkg.block_norm(args["block"], args["residual"], **dict(call, **kw))
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(residual_scale=float("inf"))):
        with pytest.raises(pkg._lib.MoEError):
            pkg.block_norm(n["z"], n["r"], **dict(call, **kw))
    with pytest.raises(pkg._lib.MoEError):   # rows of more than 8192 values, and of a count that is no multiple of 8
        pkg.block_norm(torch.zeros(1, 8200, device="cuda", dtype=BF16))
    with pytest.raises(pkg._lib.MoEError):
        pkg.block_norm(torch.zeros(1, 12, device="cuda", dtype=BF16))
    with pytest.raises(pkg._lib.MoEError):   # no tokens
        pkg.block_norm(n["z"][:0], n["r"][:0], **call)
    with pytest.raises(TypeError):
        pkg.block_norm([1.0], None)
    back = dict(norm_weight=n["w"], gate=n["g"], next_weight=n["v"])
    with pytest.raises(pkg._lib.MoEError):   # nothing flows back
        pkg.block_norm_backward(None, None, n["z"], s, norm_weight=n["w"])
    with pytest.raises(pkg._lib.MoEError):   # the stream is needed for its norm's gradient
        pkg.block_norm_backward(n["ds"], n["dy"], n["z"], None, **back)
    with pytest.raises(ValueError):
        pkg.block_norm_backward(n["ds"].float(), n["dy"], n["z"], s, **back)
    f = ffn.make(4, 64, 72, BF16, seed=1)
    out, gu = pkg.ffn_forward(f["x"], f["wgu"], f["wd"], save=True)
    for bad in (dict(x=f["x"].half()), dict(wgu=f["wgu"][:143]), dict(wd=f["wd"].t().contiguous()), dict(wd=f["wd"].cpu()),
                dict(x=f["x"][:, :56])):
        m = dict(f, **bad)
        with pytest.raises(ValueError):
            pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    with pytest.raises(ValueError):
        pkg.ffn_backward(f["dy"], f["x"], gu.half(), f["wgu"], f["wd"])
    with pytest.raises(pkg._lib.MoEError):
        pkg.ffn_backward(f["dy"], f["x"], gu, f["wgu"], f["wd"], need_x=False, need_weights=False)
    for act in (2, -1):
        with pytest.raises(pkg._lib.MoEError):
            pkg.ffn_forward(f["x"], f["wgu"], f["wd"], act=act)
    with pytest.raises((ValueError, OverflowError)):
        pkg.ffn_forward(f["x"], f["wgu"], f["wd"], act=1 << 32)
    v = matvec.make(4, 64, 128, BF16, seed=1)
    w = pkg.MatvecMXFP4(v["codes"], v["scales"], bias=v["bias"])
    for x in (v["x"].float(), v["x"][:, :64], v["x"].cpu(), v["x"].t()):
        with pytest.raises(ValueError):
            w(x)
    for T in (0, 65):
        with pytest.raises(pkg._lib.MoEError):
            w(torch.zeros(T, 128, device="cuda", dtype=BF16))
    with pytest.raises(ValueError):
        pkg.MatvecMXFP4(v["codes"], v["scales"][:, :2])
    with pytest.raises(pkg._lib.MoEError):   # gate and up rows come in pairs
        pkg.MatvecMXFP4(v["codes"][:63], v["scales"][:63], kind=pkg.MOE_WEIGHTS_GATEUP)
    assert pkg.dense_status() == 0
