"""GPU checks of the moves between token and expert order and of their gradients against
plain statements: the order and the moved rows exactly, the sums in 64 bits.

Bounds.  Moved rows and whole numbers are equal.  out and d_x are one rounding to their type
of an f32 sum of at most k products, k + 1 roundings of 2^-24 on the sum of magnitudes; d_y is
one rounding of one f32 product.  d_topk_w is an f32 sum of H products by at least 32 threads,
each a chain of at most H / 32, joined by a butterfly of 5 and at most 31 warps: H / 32 + 40
roundings of the sum of magnitudes.  The logits' gradient has sums of at most 32 terms or of
8 and a butterfly (5), exp to 1 unit (2 roundings) and a handful of products: 64 cover it."""

import pytest
import torch

from tests.dense_ref import U32, floor_of, half_step, within

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def routing(T, k, E, drop=0.0, seed=0, skew=0.5, dev="cuda"):
    """Distinct experts per token by a skewed router; the last tokens, and some single
    assignments, go to no expert (by indices on either side of the range)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device=dev) + skew * torch.randn(E, generator=g, device=dev)
    idx = torch.topk(logits, k, 1).indices.int()
    if drop:
        gone = torch.rand(T, k, generator=g, device=dev) < drop / 2
        gone[T - int(T * drop / 2):] = True
        bad = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device=dev)
        idx = torch.where(gone, bad[torch.randint(0, 4, (T, k), generator=g, device=dev)], idx)
    return idx.contiguous()


def order(idx, E):
    """offsets, perm, inv_perm by a stable sort."""
    T, k = idx.shape
    key = torch.where((idx >= 0) & (idx < E), idx, E).flatten().long()
    perm = torch.sort(key, stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=idx.device)
    counts = torch.bincount(key, minlength=E + 1)
    return ((counts.cumsum(0) - counts).int(), torch.where(key[perm] < E, perm, -1 - perm).int(),
            torch.where(key < E, inv, -1 - inv).int().view(T, k))


def moved(x, perm, k):
    """The rows that belong at each place, as bytes."""
    b = x.contiguous().view(torch.uint8).view(x.shape[0], -1)
    kept = perm >= 0
    return torch.where(kept[:, None], b[torch.where(kept, perm, 0).long() // k], 0)


def rows_of(T, H, dtype, seed, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    if dtype.itemsize == 1:
        return torch.randint(0, 256, (T, H), generator=g, device=dev, dtype=torch.uint8).view(dtype)
    return torch.randn(T, H, generator=g, device=dev).to(dtype)


def bytes_of(t):
    return t.contiguous().view(torch.uint8).view(t.shape[0], -1)


def check_sort(s, x, idx, E, scales=None):
    offsets, perm, inv = order(idx, E)
    k = idx.shape[1]
    assert torch.equal(s.offsets, offsets) and torch.equal(s.perm, perm) and torch.equal(s.inv_perm, inv)
    assert s.rows.dtype == x.dtype and torch.equal(bytes_of(s.rows), moved(x, perm, k))
    if scales is None:
        assert s.scales is None
    else:
        assert s.scales.dtype == scales.dtype and torch.equal(bytes_of(s.scales), moved(scales, perm, k))


def picked(y, inv):
    on = inv >= 0
    return torch.where(on[:, :, None], y[torch.where(on, inv, 0).long()].double(), 0.0)


def check_unsort(out, y, inv, w):
    rows = picked(y, inv)
    w = torch.ones(inv.shape, dtype=torch.float64, device=y.device) if w is None else torch.where(inv >= 0, w.double(), 0.0)
    want, mag = (rows * w[:, :, None]).sum(1), (rows.abs() * w.abs()[:, :, None]).sum(1)
    assert out.dtype == y.dtype
    within(out, want, half_step(out.dtype) * want.abs() + (inv.shape[1] + 1) * U32 * mag + floor_of(out.dtype))


def check_unsort_grads(grads, d_out, y, inv, w):
    T, k = inv.shape
    H = d_out.shape[1]
    if grads.topk_w is not None:
        rows = picked(y, inv)
        want, mag = (rows * d_out.double()[:, None]).sum(2), (rows * d_out.double()[:, None]).abs().sum(2)
        within(grads.topk_w, want, (H / 32 + 40) * U32 * mag + floor_of(F32))
    if grads.y is not None:
        at = torch.where(inv >= 0, inv, -1 - inv).flatten().long()
        w = torch.ones(inv.shape, dtype=torch.float64, device=d_out.device) if w is None else w.double()
        w = torch.where(inv >= 0, w, 0.0)
        want = torch.empty(T * k, H, dtype=torch.float64, device=d_out.device)
        want[at] = (w[:, :, None] * d_out.double()[:, None]).view(T * k, H)
        within(grads.y, want, (half_step(grads.y.dtype) + U32) * want.abs() + floor_of(grads.y.dtype))


def all_of(T, k, E, H, dtype, drop, seed=0, weighted=True):
    import mxfp4_expert_layer_gb300 as pkg
    idx = routing(T, k, E, drop, seed)
    x, y = rows_of(T, H, dtype, seed + 1), rows_of(T * k, H, dtype, seed + 2)
    d_out, d_rows = rows_of(T, H, dtype, seed + 3), rows_of(T * k, H, dtype, seed + 4)
    w = torch.softmax(rows_of(T, k, F32, seed + 5), 1) if weighted else None
    s = pkg.sort_tokens(x, idx, E)
    check_sort(s, x, idx, E)
    check_unsort(pkg.unsort_tokens(y, s.inv_perm, w), y, s.inv_perm, w)
    check_unsort(pkg.sort_tokens_backward(d_rows, s.inv_perm), d_rows, s.inv_perm, None)
    check_unsort_grads(pkg.unsort_tokens_backward(d_out, y, s.inv_perm, w), d_out, y, s.inv_perm, w)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,E,H,drop", [
    (1, 1, 1, 8, 0.0), (1, 4, 32, 2880, 0.0), (2, 32, 256, 72, 0.3), (7, 1, 256, 264, 0.5), (64, 4, 128, 2880, 0.0),
    (64, 4, 128, 16, 0.2), (100, 8, 8, 520, 0.1), (333, 4, 32, 2880, 0.1), (1000, 8, 256, 64, 0.3),
    (1025, 1, 3, 4096, 0.0), (5000, 2, 8, 1024, 0.0), (2049, 5, 61, 328, 0.02)])
def test_shapes_and_types(T, k, E, H, dtype, drop):
    all_of(T, k, E, H, dtype, drop, seed=T + H)


@pytest.mark.parametrize("T,k,E,H", [(40000, 8, 256, 16), (70001, 1, 100, 8), (9000, 32, 200, 24), (524288, 2, 8, 8)])
def test_many_assignments(T, k, E, H):
    all_of(T, k, E, H, BF16, 0.05, seed=T)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,E,H", [(2500, 9, 32, 2888), (2000, 2, 8, 8192), (2000, 17, 32, 16384), (3000, 4, 128, 2880),
                                     (15000, 3, 7, 40), (5000, 8, 64, 4096), (2000, 32, 40, 4104), (1000, 4, 16, 2880)])
def test_many_tokens_of_wide_rows(T, k, E, H, dtype):
    """Rows in several column chunks, more than eight rows a token, and both at once, where
    persistent blocks take the tokens in turn."""
    all_of(T, k, E, H, dtype, 0.05, seed=H + k)


@pytest.mark.parametrize("H", [8192, 16384, 32768])
def test_widest_rows(H):
    all_of(37, 3, 16, H, BF16, 0.1, seed=H)
    if H <= 16384:
        all_of(13, 2, 16, H, F32, 0.1, seed=H)


@pytest.mark.parametrize("T,k,E,drop", [(512, 4, 128, 0.0), (2048, 1, 9, 0.2), (683, 3, 7, 0.1), (2049, 1, 256, 0.0), (128, 16, 16, 0.3),
                                        (8192, 8, 32, 0.0), (8193, 8, 31, 0.01)])
def test_where_the_ways_to_the_order_meet(T, k, E, drop):
    """2048 assignments and the next: one launch and two; 65536 and more: runs in registers and not."""
    all_of(T, k, E, 48, BF16, drop, seed=T)


@pytest.mark.parametrize("dtype", [torch.float64, torch.int32, torch.int64, torch.bool, torch.float8_e5m2, torch.complex64])
def test_rows_of_any_type(dtype):
    import mxfp4_expert_layer_gb300 as pkg
    for T in (7, 3000):
        x = torch.randint(0, 256, (T, 80), device="cuda", dtype=torch.uint8)
        x = (x & 1 if dtype == torch.bool else x).view(dtype)
        idx = routing(T, 2, 16, 0.2, seed=T)
        check_sort(pkg.sort_tokens(x, idx, 16), x, idx, 16)


def test_without_weights():
    all_of(77, 4, 16, 136, F16, 0.1, weighted=False)


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 4, 32), (64, 4, 128, 2880), (1000, 4, 128, 2880), (4096, 8, 64, 256)])
@pytest.mark.parametrize("scales", ["mx", "row", "odd", "wide"])
def test_eight_bit_rows_with_scales(T, k, E, H, scales):
    import mxfp4_expert_layer_gb300 as pkg
    x = rows_of(T, H, torch.float8_e4m3fn, T)
    sc = {"mx": lambda: rows_of(T, H // 32, torch.uint8, 1), "row": lambda: rows_of(T, 1, F32, 1),
          "odd": lambda: rows_of(T, 7, torch.uint8, 1), "wide": lambda: rows_of(T, 300, BF16, 1)}[scales]()
    idx = routing(T, k, E, 0.2, seed=T)
    check_sort(pkg.sort_tokens(x, idx, E, scales=sc), x, idx, E, sc)


@pytest.mark.parametrize("T,k,E", [(1, 1, 8), (64, 4, 128), (3000, 4, 32)])
def test_nothing_kept_and_all_on_one_expert(T, k, E):
    """Every assignment dropped; and every one on the first, or on the last, expert (the
    same index k times in a token)."""
    import mxfp4_expert_layer_gb300 as pkg
    x, y, w = rows_of(T, 64, BF16, 1), rows_of(T * k, 64, BF16, 2), torch.rand(T, k, device="cuda")
    for e in (-1, E, 0, E - 1):
        idx = torch.full((T, k), e, dtype=torch.int32, device="cuda")
        s = pkg.sort_tokens(x, idx, E)
        check_sort(s, x, idx, E)
        out = pkg.unsort_tokens(y, s.inv_perm, w)
        check_unsort(out, y, s.inv_perm, w)
        g = pkg.unsort_tokens_backward(x, y, s.inv_perm, w)
        check_unsort_grads(g, x, y, s.inv_perm, w)
        if not 0 <= e < E:
            assert int(s.offsets[E]) == 0 and not s.rows.any() and not out.any() and not g.y.any() and not g.topk_w.any()


@pytest.mark.parametrize("T,k,E", [(1, 4, 32), (64, 4, 128), (4096, 4, 128), (300, 2, 8)])
def test_order_of_the_layers_tile_table(T, k, E):
    """Where nothing is dropped the order is that of moe_build_tile_table."""
    import mxfp4_expert_layer_gb300 as pkg
    idx = routing(T, k, E, seed=T)
    s, table = pkg.sort_tokens(rows_of(T, 32, BF16, 0), idx, E), pkg.build_tile_table(idx, E)
    for a, b in ((s.offsets, table["offsets"]), (s.perm, table["perm"]), (s.inv_perm.flatten(), table["inv_perm"])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(5, 64), (300, 2880)])
def test_what_is_not_finite_stays_where_it_is(T, H):
    """NaN and infinities in rows and weights of dropped assignments reach nothing; in a
    live row they reach that token alone."""
    import mxfp4_expert_layer_gb300 as pkg
    idx = routing(T, 4, 16, 0.4, seed=T)
    y, w, d_out = rows_of(4 * T, H, BF16, 1), torch.rand(T, 4, device="cuda"), rows_of(T, H, BF16, 3)
    s = pkg.sort_tokens(d_out, idx, 16)
    gone = s.inv_perm < 0
    y[int(s.offsets[16]):] = float("nan")
    w[gone] = float("inf")
    check_unsort(pkg.unsort_tokens(y, s.inv_perm, w), y, s.inv_perm, w)
    g = pkg.unsort_tokens_backward(d_out, y, s.inv_perm, w)
    check_unsort_grads(g, d_out, y, s.inv_perm, w)
    assert torch.isfinite(g.y.float()).all() and torch.isfinite(g.topk_w).all()
    live = int((~gone).any(1).nonzero()[0])
    j = int((~gone[live]).nonzero()[0])
    y[int(s.inv_perm[live, j]), 3] = float("inf")
    out = pkg.unsort_tokens(y, s.inv_perm, w)
    assert int((~torch.isfinite(out.float())).sum()) == 1 and out[live, 3] == float("inf")
    d_out[live, 5] = float("nan")
    g = pkg.unsort_tokens_backward(d_out, y, s.inv_perm, w)
    bad = ~torch.isfinite(g.y.float())
    assert int(bad.sum()) == int((~gone[live]).sum()) and bad[int(s.inv_perm[live, j]), 5]


def test_places_outside_the_rows_are_not_read():
    """inv_perm is the caller's: entries beyond the rows count as dropped."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k, H = 9, 3, 40
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k).clone()
    inv[0, 0], inv[4, 1], inv[8, 2] = T * k, 2 ** 31 - 1, -2 ** 31
    y, w, d_out = rows_of(T * k, H, F32, 1), torch.rand(T, k, device="cuda"), rows_of(T, H, F32, 2)
    clean = torch.where((inv >= 0) & (inv < T * k), inv, -1)
    check_unsort(pkg.unsort_tokens(y, inv, w), y, clean, w)
    g = pkg.unsort_tokens_backward(d_out, y, inv, w)
    check_unsort_grads(g._replace(y=None), d_out, y, clean, w)


def test_gradients_one_at_a_time_and_against_differences():
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 6, 3, 5, 16
    idx = routing(T, k, E, 0.3, seed=3)
    y, w, d_out = rows_of(T * k, H, F32, 1), torch.rand(T, k, device="cuda"), rows_of(T, H, F32, 2)
    inv = pkg.sort_tokens(d_out, idx, E).inv_perm
    both = pkg.unsort_tokens_backward(d_out, y, inv, w)
    one = pkg.unsort_tokens_backward(d_out, y, inv, w, need_w=False)
    assert one.topk_w is None and torch.equal(one.y, both.y)
    assert torch.equal(pkg.unsort_tokens_backward(d_out, None, inv, w, need_w=False).y, both.y)
    one = pkg.unsort_tokens_backward(d_out, y, inv, w, need_y=False)
    assert one.y is None and torch.equal(one.topk_w, both.topk_w)

    def f(y, w):
        return (picked(y, inv) * torch.where(inv >= 0, w.double(), 0.0)[:, :, None]).sum(1).mul(d_out.double()).sum()
    y, w, h = y.double(), w.double(), 1e-5
    for t, g in ((y, both.y), (w, both.topk_w)):  # bilinear: central differences are exact to rounding
        for i in range(0, t.numel(), 7):
            keep = t.view(-1)[i].item()
            t.view(-1)[i] = keep + h
            up = f(y, w)
            t.view(-1)[i] = keep - h
            down = f(y, w)
            t.view(-1)[i] = keep
            # f is below 1000 and rounds at 2^-53 of it, over 2 h: 1e-8; the gradient is off by
            # (H / 32 + 40) 2^-24 of terms of at most 20 together: 5e-5
            assert abs(float((up - down) / (2 * h)) - g.view(-1)[i].item()) < 5e-5 + 1e-8


# ------------------------------------------------------------------ the logits' gradient
GATINGS = {"topk": 0, "all": 2, "sigmoid": 4}


def weights64(logits, idx, gating):
    chosen = logits.gather(1, idx.long())
    if gating == "topk":
        return torch.softmax(chosen, 1)
    if gating == "all":
        return torch.softmax(logits, 1).gather(1, idx.long())
    s = torch.sigmoid(chosen)
    return s / s.sum(1, keepdim=True)


def logits_grad(d_w, logits, idx, w, gating):
    """Values and magnitudes from the formulas."""
    g, l, w = d_w.double(), logits.double(), w.double()
    on = (idx >= 0) & (idx < logits.shape[1])
    at = torch.where(on, idx, 0).long()
    S, M = (w * g).sum(1, keepdim=True), (w * g).abs().sum(1, keepdim=True)
    zero = torch.zeros_like(l)
    if gating == "all":
        p = torch.softmax(l, 1)
        return (p * (zero.scatter_add(1, at, torch.where(on, g, 0.0)) - S),
                p * (zero.scatter_add(1, at, torch.where(on, g, 0.0).abs()) + M))
    part, mag = w * (g - S), w * (g.abs() + M)
    if gating == "sigmoid":
        part, mag = part * torch.sigmoid(-l.gather(1, at)), mag * torch.sigmoid(-l.gather(1, at))
    return zero.scatter_add(1, at, torch.where(on, part, 0.0)), zero.scatter_add(1, at, torch.where(on, mag, 0.0))


@pytest.mark.parametrize("gating", list(GATINGS))
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 4, 32), (9, 32, 256), (333, 4, 32), (4097, 8, 100), (20, 1, 33)])
def test_logits_gradient(T, k, E, gating):
    import mxfp4_expert_layer_gb300 as pkg
    logits = 3 * rows_of(T, E, F32, T)
    logits, idx, w = pkg.route(None, None, k, logits=logits, from_logits=True, gating=GATINGS[gating])
    d_w = rows_of(T, k, F32, T + 1)
    got = pkg.route_backward(d_w, logits, idx, w, gating=GATINGS[gating])
    want, mag = logits_grad(d_w, logits, idx, w, gating)
    # (the exponential of l - max rounds its argument: another |l - max| <= 64 roundings)
    within(got, want, 128 * U32 * mag + floor_of(F32))
    l = logits.double().requires_grad_()
    (ref,) = torch.autograd.grad(weights64(l, idx, gating), l, d_w.double())
    # against the definition: w is an input here, itself rounded by the routing (its tests hold it to 1e-5)
    within(got, ref, 128 * U32 * mag + 2e-5 * mag + floor_of(F32))


@pytest.mark.parametrize("lowest", [float("-inf"), torch.finfo(F32).min])
@pytest.mark.parametrize("gating", list(GATINGS))
def test_logits_gradient_of_masked_experts(gating, lowest):
    """Experts masked by -inf or the type's lowest value get no gradient, and give no NaN, also
    where fewer experts than k are left."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E = 40, 4, 48
    logits = rows_of(T, E, F32, 1)
    logits[:, 5:] = lowest
    logits[::2, 2:] = lowest
    logits, idx, w = pkg.route(None, None, k, logits=logits, from_logits=True, gating=GATINGS[gating])
    d_w = rows_of(T, k, F32, 2)
    got = pkg.route_backward(d_w, logits, idx, w, gating=GATINGS[gating])
    want, mag = logits_grad(d_w, logits, idx, w, gating)
    within(got, want, 128 * U32 * mag + floor_of(F32))
    assert not got[:, 5:].any() and not got[::2, 2:].any()


@pytest.mark.parametrize("gating", list(GATINGS))
def test_logits_gradient_of_listed_twice_and_of_none(gating):
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E = 12, 4, 8
    logits, d_w = rows_of(T, E, F32, 1), rows_of(T, k, F32, 2)
    idx = torch.randint(-1, E + 1, (T, k), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(3))
    idx[0] = 5
    idx[1] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    w = torch.rand(T, k, device="cuda")
    got = pkg.route_backward(d_w, logits, idx, w, gating=GATINGS[gating])
    want, mag = logits_grad(d_w, logits, idx, w, gating)
    within(got, want, 128 * U32 * mag + floor_of(F32))
    if gating != "all":
        assert not got[1].any()


# ------------------------------------------------------------------ as programs call them
def test_captured_other_streams_and_repeats():
    """Captured and replayed on new inputs, on a stream of its own, and eagerly: the same
    bits; and run to run the same."""
    import mxfp4_expert_layer_gb300 as pkg
    for T, k, E, H in ((64, 4, 128, 2880), (3000, 4, 32, 512)):
        def inputs(seed):
            return (rows_of(T, H, BF16, seed), routing(T, k, E, 0.1, seed), rows_of(T * k, H, BF16, seed + 1),
                    torch.rand(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))

        def step(x, idx, y, w):
            s = pkg.sort_tokens(x, idx, E)
            return tuple(s._replace(scales=s.rows)) + (pkg.unsort_tokens(y, s.inv_perm, w),
                                                       pkg.sort_tokens_backward(y, s.inv_perm)) + \
                tuple(pkg.unsort_tokens_backward(x, y, s.inv_perm, w))
        held = [t.clone() for t in inputs(1)]
        step(*held)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step(*held)
        side = torch.cuda.Stream()
        for seed in (1, 2, 3):
            new = inputs(seed)
            for a, b in zip(held, new):
                a.copy_(b)
            graph.replay()
            eager = step(*new)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                other = step(*new)
            torch.cuda.current_stream().wait_stream(side)
            for a, b, c in zip(captured, eager, other):
                assert torch.equal(a, b) and torch.equal(a, c)


def test_results_given():
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 50, 4, 16, 96
    idx, y, w = routing(T, k, E, 0.1), rows_of(T * k, H, F16, 1), torch.rand(T, k, device="cuda")
    inv = pkg.sort_tokens(rows_of(T, H, F16, 2), idx, E).inv_perm
    out = torch.full((T + 2, H), 7.0, dtype=F16, device="cuda")
    assert pkg.unsort_tokens(y, inv, w, out=out[1:T + 1]).data_ptr() == out[1].data_ptr()
    check_unsort(out[1:T + 1], y, inv, w)
    pkg.sort_tokens_backward(y, inv, out=out[1:T + 1])
    check_unsort(out[1:T + 1], y, inv, None)
    assert (out[0] == 7).all() and (out[T + 1] == 7).all()


def test_parts_of_a_batch():
    """Index and weight arrays that begin at any element: slices of a larger routing."""
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 61, 3, 16, 96
    idx, w, x = routing(T, k, E, 0.1, seed=1), torch.rand(T, k, device="cuda"), rows_of(T, H, BF16, 2)
    for part in (slice(1, 20), slice(20, 61), slice(3, 4)):
        n = part.stop - part.start
        s = pkg.sort_tokens(x[part], idx[part], E)
        check_sort(s, x[part], idx[part], E)
        y, inv = rows_of(n * k, H, BF16, 3), torch.empty(n * k + 1, dtype=torch.int32, device="cuda")[1:].view(n, k)
        inv.copy_(s.inv_perm)
        check_unsort(pkg.unsort_tokens(y, inv, w[part]), y, s.inv_perm, w[part])
        check_unsort_grads(pkg.unsort_tokens_backward(x[part], y, inv, w[part]), x[part], y, s.inv_perm, w[part])
        logits = torch.randn(T, E, device="cuda")[part]
        got = pkg.route_backward(w[part], logits, idx[part], w[part])
        want, mag = logits_grad(w[part], logits, idx[part], w[part], "topk")
        within(got, want, 128 * U32 * mag + floor_of(F32))


def test_refusals():
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 6, 2, 8, 32
    x, idx, y = rows_of(T, H, BF16, 1), routing(T, k, E), rows_of(T * k, H, BF16, 2)
    s, w = pkg.sort_tokens(x, idx, E), torch.rand(T, k, device="cuda")
    for call in (lambda: pkg.sort_tokens(x, idx.long(), E), lambda: pkg.sort_tokens(x, idx[:5], E),
                 lambda: pkg.sort_tokens(x, idx.t().contiguous().t(), E), lambda: pkg.sort_tokens(x.t(), idx, E),
                 lambda: pkg.sort_tokens(x.cpu(), idx.cpu(), E), lambda: pkg.sort_tokens(x, idx.cpu(), E),
                 lambda: pkg.sort_tokens(x, idx, E, scales=w[:5]), lambda: pkg.sort_tokens(x[0], idx, E),
                 lambda: pkg.unsort_tokens(y[:-1], s.inv_perm, w), lambda: pkg.unsort_tokens(y, s.inv_perm.flatten(), w),
                 lambda: pkg.unsort_tokens(y, s.inv_perm, w.to(BF16)), lambda: pkg.unsort_tokens(y.double(), s.inv_perm, w),
                 lambda: pkg.unsort_tokens(y, s.inv_perm, w, out=x.half()),
                 lambda: pkg.unsort_tokens_backward(x, y.half(), s.inv_perm, w),
                 lambda: pkg.unsort_tokens_backward(x[:5], y, s.inv_perm, w),
                 lambda: pkg.route_backward(w, torch.zeros(T, E, device="cuda", dtype=BF16), idx, w),
                 lambda: pkg.route_backward(w[:, :1], torch.zeros(T, E, device="cuda"), idx, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pkg.sort_tokens(x, idx, 0), lambda: pkg.sort_tokens(x, idx, 257), lambda: pkg.sort_tokens(x, idx, 1),
                 lambda: pkg.sort_tokens(x[:0], idx[:0], E), lambda: pkg.sort_tokens(rows_of(T, 12, BF16, 1), idx, E),
                 lambda: pkg.unsort_tokens(rows_of(T * k, 12, BF16, 1), s.inv_perm, w),
                 lambda: pkg.unsort_tokens(y, s.inv_perm, w, out=y[:T]),
                 lambda: pkg.unsort_tokens_backward(x, None, s.inv_perm, w),
                 lambda: pkg.unsort_tokens_backward(x, y, s.inv_perm, w, need_y=False, need_w=False),
                 lambda: pkg.route_backward(w, torch.zeros(T, E, device="cuda"), idx, w, gating=6),
                 lambda: pkg.route_backward(w, torch.zeros(T, E, device="cuda"), idx, w, gating=1)):
        with pytest.raises(pkg._lib.MoEError):
            call()
    check_sort(pkg.sort_tokens(x, idx, E), x, idx, E)  # and the device is as it was


@pytest.mark.parametrize("T,k,H", [(70000, 8, 4096)])
def test_more_than_2_31_elements(T, k, H):
    """Rows whose element offsets pass 2^31 and whose byte offsets pass 2^32."""
    import mxfp4_expert_layer_gb300 as pkg
    E = 64
    idx, x = routing(T, k, E, 0.01, seed=1), rows_of(T, H, BF16, 1)
    s = pkg.sort_tokens(x, idx, E)
    offsets, perm, inv = order(idx, E)
    assert torch.equal(s.offsets, offsets) and torch.equal(s.perm, perm) and torch.equal(s.inv_perm, inv)
    for part in (slice(0, 2000), slice(T * k // 2, T * k // 2 + 2000), slice(T * k - 8000, T * k)):
        assert torch.equal(bytes_of(s.rows[part]), moved(x, perm[part], k))
    w = torch.rand(T, k, device="cuda")
    out = pkg.unsort_tokens(s.rows, inv, w)
    g = pkg.unsort_tokens_backward(x, s.rows, inv, w)
    for part in (slice(0, 500), slice(T // 2, T // 2 + 500), slice(T - 500, T)):
        check_unsort(out[part], s.rows, inv[part], w[part])
        rows = picked(s.rows, inv[part])
        terms = rows * x[part].double()[:, None]
        within(g.topk_w[part], terms.sum(2), (H / 32 + 40) * U32 * terms.abs().sum(2) + floor_of(F32))
        on = inv[part] >= 0
        want = w[part].double()[:, :, None] * x[part].double()[:, None]
        within(g.y[inv[part][on].long()], want[on], (half_step(BF16) + U32) * want[on].abs() + floor_of(BF16))
