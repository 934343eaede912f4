"""Measured cases of the operators around experts of one's own: tokens sorted by expert and
back with their gradients and the router's, projections with bias, activation and residual
(forward and training step), and the norm around a block with an 8-bit output.

``run`` makes the calls a user makes where ``own`` is true; elsewhere it computes the
same operators from elementary torch operations in 32 bits.  ``exact`` restates each
operator in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = {"silu": 0, "gelu": 1, "none": 2}
GATINGS = {"topk": 0, "all": 2, "sigmoid": 4}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch of 64 before its experts
        dict(name="sort_decode", op="sort", T=64, k=4, E=128, H=2880, dtype="bf16", dropped=0.0),
        # a prefill chunk dispatched in 8 bits with a scale per 32 values, its last tokens padding
        dict(name="sort_prefill_8bit", op="sort", T=4096, k=4, E=128, H=2880, dtype="e4m3", dropped=0.06),
        # one generated token behind its experts
        dict(name="unsort_decode", op="unsort", T=1, k=4, E=32, H=2880, dtype="bf16", dropped=0.0),
        # a large prefill behind eight wide experts
        dict(name="unsort_prefill", op="unsort", T=8192, k=2, E=8, H=4096, dtype="f16", dropped=0.0),
        # a ragged, padded micro-batch: both moves, all their gradients and the router's
        dict(name="dispatch_train_ragged", op="dispatch_train", T=333, k=4, E=32, H=2880, dtype="f16", dropped=0.1,
             gating="topk"),
        # a large training batch with eight experts
        dict(name="dispatch_train_large", op="dispatch_train", T=8192, k=2, E=8, H=4096, dtype="bf16", dropped=0.0,
             gating="all"),
        # one token through an output projection onto the residual stream
        dict(name="linear_decode", op="linear", T=1, K=4096, N=2880, dtype="bf16", act="none", bias=True,
             residual=True, out="bf16"),
        # a prefill chunk through a square projection onto a residual stream kept in 32 bits
        dict(name="linear_prefill", op="linear", T=2048, K=4096, N=4096, dtype="bf16", act="none", bias=True,
             residual=True, out="f32"),
        # a ragged training step of one layer of a plain (not gated) feed-forward block
        dict(name="linear_train_ragged", op="linear_train", T=1001, K=2880, N=2880, dtype="f16", act="gelu", bias=True,
             residual=False, out="f16"),
        # a large training step of the same
        dict(name="linear_train_large", op="linear_train", T=4096, K=4096, N=14336, dtype="bf16", act="gelu", bias=True,
             residual=False, out="bf16"),
        # one generated token through the norm pair, for 8-bit experts
        dict(name="norm8_decode", op="norm8", T=1, H=2880, dtype="bf16", stream="bf16", gate="none", scales="mx"),
        # a prefill chunk, one scale per token
        dict(name="norm8_prefill", op="norm8", T=4096, H=2880, dtype="bf16", stream="bf16", gate="token", scales="row"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "unsort", "dispatch_train", "linear", "linear_train", "norm8"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("sort", "unsort", "dispatch_train"):
        k = rng.randint(1, 8)
        case = dict(op=op, T=_log_int(rng, 1, 8192), k=k, E=_log_int(rng, k, 256), H=16 * _log_int(rng, 4, 256),
                    dtype=rng.choice([dtype, "e4m3"]) if op == "sort" else rng.choice([dtype, "f32"]),
                    dropped=rng.choice([0.0, 0.05, 0.5]))
        if op == "dispatch_train":
            case["gating"] = rng.choice(["topk", "all", "sigmoid"])
        return case
    if op in ("linear", "linear_train"):
        return dict(op=op, T=_log_int(rng, 1, 2048), K=8 * _log_int(rng, 8, 512), N=8 * _log_int(rng, 4, 1792),
                    dtype=dtype, act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, out=rng.choice([dtype, "f32"]))
    scales = rng.choice(["mx", "row"])
    return dict(op=op, T=_log_int(rng, 1, 8192), H=32 * _log_int(rng, 2, 128) if scales == "mx" else
                8 * _log_int(rng, 8, 512), dtype=dtype, stream=rng.choice([dtype, "f32"]),
                gate=rng.choice(["none", "feature", "token", "full"]), scales=scales)


def work(case):
    op, T = case["op"], case["T"]
    if op in ("sort", "unsort", "dispatch_train"):
        k, E, H = case["k"], case["E"], case["H"]
        n, size = T * k, {"e4m3": 1, "f32": 4}.get(case["dtype"], 2)
        row = H * size + (H // 32 if case["dtype"] == "e4m3" else 0)
        sort = T * row + n * row + 12 * n + 4 * (E + 1)
        if op == "sort":
            return {"bytes": sort, "flops": 0}
        unsort = n * row + T * row + 8 * n
        if op == "unsort":
            return {"bytes": unsort, "flops": 2 * n * H}
        # both moves; then d_out and y read again, d_y and d_w written; d_rows summed into d_x; the logits' gradient
        unsort_bwd = T * row + n * row + 8 * n + n * row + 4 * n
        sort_bwd = n * row + T * row + 4 * n
        route_bwd = (8 if case["gating"] == "all" else 4) * T * E + 12 * n
        return {"bytes": sort + unsort + unsort_bwd + sort_bwd + route_bwd, "flops": 6 * n * H}
    if op in ("linear", "linear_train"):
        K, N = case["K"], case["N"]
        o = 4 if case["out"] == "f32" else 2
        fwd = 2 * (T * K + N * K) + o * T * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        if op == "linear":
            return {"bytes": fwd, "flops": 2 * T * N * K}
        return {"bytes": fwd + o * T * N + 2 * (T * K + N * K) + (4 * N if case["bias"] else 0), "flops": 6 * T * N * K}
    H, s = case["H"], 4 if case["stream"] == "f32" else 2
    gate = {"none": 0, "feature": 2 * H, "token": 4 * T, "full": 2 * T * H}[case["gate"]]
    scales = 4 * T if case["scales"] == "row" else T * H // 32
    return {"bytes": T * H * (2 + 2 * s + 1) + 4 * H + gate + scales, "flops": 14 * T * H}


# ------------------------------------------------------------------ inputs
def _weights(logits, idx, gating):
    chosen = logits.gather(1, idx.long())
    if gating == "topk":
        return torch.softmax(chosen, 1)
    if gating == "all":
        return torch.softmax(logits, 1).gather(1, idx.long())
    s = torch.sigmoid(chosen)
    return s / s.sum(1, keepdim=True)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T, op = case["T"], case["op"]
    dt = DTYPES.get(case["dtype"])

    def rand(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dtype)

    st = dict(case=case)
    if op in ("sort", "unsort", "dispatch_train"):
        k, E, H = case["k"], case["E"], case["H"]
        # experts of unequal popularity, as a router leaves them
        logits = rand(T, E, dtype=torch.float32) + 0.5 * rand(E, dtype=torch.float32)
        routed = torch.topk(logits, k, 1).indices.int()
        st["idx"] = routed.clone()
        # the last tokens are padding: they go to no expert
        st["idx"][T - int(T * case["dropped"]):] = -1
        st["w"] = _weights(logits, routed, case.get("gating", "topk"))
        if op == "sort":
            if case["dtype"] == "e4m3":
                st["x"] = rand(T, H, std=100.0, dtype=torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn)
                st["scales"] = torch.randint(110, 125, (T, H // 32), generator=g, device=dev, dtype=torch.uint8)
            else:
                st["x"] = rand(T, H)
            return st
        st["y"] = rand(T * k, H)
        if op == "unsort":
            # what the sort before the experts left behind
            st["inv_perm"] = _sort_order(st["idx"], E)[2]
            return st
        st["x"], st["d_out"], st["d_rows"] = rand(T, H), rand(T, H), rand(T * k, H)
        st["logits"], st["routed"] = logits, routed
        return st
    if op in ("linear", "linear_train"):
        K, N, odt = case["K"], case["N"], DTYPES[case["out"]]
        st["x"] = rand(T, K)
        st["weight"] = rand(N, K, std=1.0 / math.sqrt(K))
        st["bias"] = rand(N, std=0.5, dtype=torch.float32) if case["bias"] else None
        st["residual"] = rand(T, N, std=2.0, dtype=odt) if case["residual"] else None
        if op == "linear_train":
            st["d_out"] = rand(T, N, dtype=odt)
        return st
    H, sdt = case["H"], DTYPES[case["stream"]]
    st["block"], st["residual"] = rand(T, H), rand(T, H, std=2.0, dtype=sdt)
    st["norm_weight"], st["next_weight"] = rand(H, std=0.25, mean=1.0), rand(H, std=0.25, mean=1.0)
    kind = case["gate"]
    st["gate"] = (rand(H, std=0.3, mean=0.5) if kind == "feature" else
                  torch.sigmoid(rand(T, 1, dtype=torch.float32)) if kind == "token" else
                  rand(T, H, std=0.5) if kind == "full" else None)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import mxfp4_expert_layer_gb300 as moe
        return _own(moe, op, state)
    return {"sort": _sort, "unsort": _unsort, "dispatch_train": _dispatch_train, "linear": _linear,
            "linear_train": _linear_train, "norm8": _norm8}[op](state)


def _own(moe, op, st):
    case = st["case"]
    if op == "sort":
        s = moe.sort_tokens(st["x"], st["idx"], case["E"], scales=st.get("scales"))
        return s.rows, s.scales, s.offsets, s.perm, s.inv_perm
    if op == "unsort":
        return moe.unsort_tokens(st["y"], st["inv_perm"], st["w"])
    if op == "dispatch_train":
        s = moe.sort_tokens(st["x"], st["idx"], case["E"])
        out = moe.unsort_tokens(st["y"], s.inv_perm, st["w"])
        d_y, d_w = moe.unsort_tokens_backward(st["d_out"], st["y"], s.inv_perm, st["w"])
        d_x = moe.sort_tokens_backward(st["d_rows"], s.inv_perm)
        d_logits = moe.route_backward(d_w, st["logits"], st["routed"], st["w"], gating=GATINGS[case["gating"]])
        return s.rows, s.offsets, s.perm, s.inv_perm, out, d_y, d_w, d_x, d_logits
    act = ACTS[case["act"]] if "act" in case else None
    if op == "linear":
        return moe.linear_forward(st["x"], st["weight"], st["bias"], st["residual"], act=act,
                                  out_dtype=DTYPES[case["out"]])
    if op == "linear_train":
        out, pre = moe.linear_forward(st["x"], st["weight"], st["bias"], st["residual"], act=act,
                                      out_dtype=DTYPES[case["out"]], save=True)
        return (out,) + tuple(moe.linear_backward(st["d_out"], st["x"], st["weight"], pre, act=act,
                                                  need_bias=case["bias"]))
    s = moe.block_norm_8bit(st["block"], st["residual"], norm_weight=st["norm_weight"], gate=st["gate"],
                            residual_scale=0.5, next_weight=st["next_weight"], eps=EPS, scales=case["scales"])
    return s.residual, s.codes, s.scales


# ------------------------------------------------------------------ plain forms
def _sort_order(idx, E):
    """offsets, perm, inv_perm of a routing: sorted by expert, then by place; what names no expert comes last, its
    entries as -1 - entry."""
    T, k = idx.shape
    key = torch.where((idx >= 0) & (idx < E), idx, E).view(-1)
    perm = torch.argsort(key, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=idx.device)
    offsets = torch.searchsorted(key[perm], torch.arange(E + 1, device=idx.device, dtype=key.dtype))
    perm = torch.where(key[perm] < E, perm, -1 - perm)
    inv = torch.where(key < E, inv, -1 - inv)
    return offsets.int(), perm.int(), inv.int().view(T, k)


def _gathered(x, perm, k):
    rows = x[torch.where(perm >= 0, perm, 0).long() // k]
    return torch.where((perm >= 0)[:, None], rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _sort(st):
    case, x = st["case"], st["x"]
    offsets, perm, inv = _sort_order(st["idx"], case["E"])
    scales = None
    if case["dtype"] == "e4m3":
        rows = _gathered(x.view(torch.uint8), perm, case["k"]).view(x.dtype)
        scales = _gathered(st["scales"], perm, case["k"])
    else:
        rows = _gathered(x, perm, case["k"])
    return rows, scales, offsets, perm, inv


def _summed(y, inv, w):
    picked = y[torch.where(inv >= 0, inv, 0).long()].float()
    picked = torch.where((inv >= 0)[:, :, None], picked, 0.0)
    return (picked * w[:, :, None]).sum(1).to(y.dtype)


def _unsort(st):
    return _summed(st["y"], st["inv_perm"], st["w"])


def _dispatch_train(st):
    case, idx, w, y = st["case"], st["idx"], st["w"], st["y"]
    T, k, E = case["T"], case["k"], case["E"]
    offsets, perm, inv = _sort_order(idx, E)
    rows = _gathered(st["x"], perm, k)
    out = _summed(y, inv, w)
    on = inv >= 0
    at = torch.where(on, inv, 0).long()
    d_out = st["d_out"].float()
    d_w = torch.where(on, (y[at].float() * d_out[:, None]).sum(2), 0.0)
    a = torch.where(perm >= 0, perm, 0).long()
    d_y = torch.where((perm >= 0)[:, None], d_out[a // k] * w.view(-1)[a][:, None], 0.0).to(y.dtype)
    d_x = _summed(st["d_rows"], inv, torch.ones_like(w))
    chosen = st["routed"].long()
    total = (w * d_w).sum(1, keepdim=True)
    if case["gating"] == "all":
        p = torch.exp(st["logits"] - st["logits"].max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        d_logits = p * (torch.zeros_like(p).scatter_add_(1, chosen, d_w) - total)
    else:
        part = w * (d_w - total)
        if case["gating"] == "sigmoid":
            part = part / (1.0 + torch.exp(st["logits"].gather(1, chosen)))
        d_logits = torch.zeros_like(st["logits"]).scatter_add_(1, chosen, part)
    return rows, offsets, perm, inv, out, d_y, d_w, d_x, d_logits


def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    return v


def _act_grad(v, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 + v * (1.0 - s))
    t = torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v))
    return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * (0.7978845608028654 * (1.0 + 3 * 0.044715 * v * v))


def _linear_pre(st):
    pre = st["x"].float() @ st["weight"].float().t()
    return pre if st["bias"] is None else pre + st["bias"]


def _linear_out(st, pre):
    out = _act(pre, st["case"]["act"])
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return out.to(DTYPES[st["case"]["out"]])


def _linear(st):
    return _linear_out(st, _linear_pre(st))


def _linear_train(st):
    dt, act = st["x"].dtype, st["case"]["act"]
    pre = _linear_pre(st)
    out = _linear_out(st, pre)
    dp = st["d_out"].float()
    if act != "none":
        dp = dp * _act_grad(pre, act)
    d_x = dp @ st["weight"].float()
    d_w = dp.t() @ st["x"].float()
    return out, d_x.to(dt), d_w.to(dt), dp.sum(0) if st["bias"] is not None else None


def _norm8(st):
    case, f = st["case"], torch.Tensor.float
    z, r = f(st["block"]), f(st["residual"])
    p = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * f(st["norm_weight"])
    if st["gate"] is not None:
        p = p * f(st["gate"])
    s = (0.5 * r + p).to(st["residual"].dtype)
    sf = f(s)
    y = sf * torch.rsqrt(sf.square().mean(1, keepdim=True) + EPS) * f(st["next_weight"])
    if case["scales"] == "row":
        scale = (y.abs().amax(1, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
        return s, (y / scale).to(torch.float8_e4m3fn), scale
    T, H = y.shape
    y = y.view(T, H // 32, 32)
    m, e = torch.frexp(y.abs().amax(2, keepdim=True))
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    codes = (y * torch.exp2(-e.float())).to(torch.float8_e4m3fn).view(T, H)
    return s, codes, (e + 127).to(torch.uint8).view(T, H // 32).view(torch.float8_e8m0fnu)


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in st.items()}
    if op in ("sort", "unsort", "dispatch_train"):
        k, E = case["k"], case["E"]
        # an assignment's place is the number of those before it in the order of (expert, place)
        key = st["idx"].long().reshape(-1)
        key[(key < 0) | (key >= E)] = E
        order = (key * (T * k) + torch.arange(T * k, device=key.device)).sort().indices
        place = torch.empty_like(order)
        place.scatter_(0, order, torch.arange(T * k, device=key.device))
        kept = key < E
        counts = torch.bincount(key, minlength=E + 1)
        offsets = (torch.cumsum(counts, 0) - counts).int()
        perm = torch.where(kept[order], order, -1 - order).int()
        inv = torch.where(kept, place, -1 - place).int().view(T, k)
        if op != "unsort":
            x = d["x"] if case["dtype"] != "e4m3" else st["x"].float().double()
            rows = x[order // k] * kept[order][:, None]
        if op == "sort":
            scales = st["scales"][order // k] * kept[order][:, None] if "scales" in st else None
            return rows, scales, offsets, perm, inv
        y, w = d["y"], d["w"]
        out = torch.zeros(T, case["H"], dtype=torch.float64, device=y.device)
        place = place.view(T, k)
        alive = kept.view(T, k).double()
        for j in range(k):
            out += (w[:, j] * alive[:, j])[:, None] * y[place[:, j]]
        if op == "unsort":
            return out
        d_out, d_rows = d["d_out"], d["d_rows"]
        d_w, d_x = torch.zeros_like(w), torch.zeros_like(d_out)
        d_y = torch.zeros_like(y)
        for j in range(k):
            at = place[:, j]
            d_w[:, j] = torch.einsum("th,th->t", d_out, y[at]) * alive[:, j]
            d_x += alive[:, j][:, None] * d_rows[at]
            d_y[at] = (w[:, j] * alive[:, j])[:, None] * d_out
        logits = d["logits"].requires_grad_()
        (d_logits,) = torch.autograd.grad(_weights(logits, st["routed"], case["gating"]), logits, d_w)
        return rows, offsets, perm, inv, out, d_y, d_w, d_x, d_logits
    if op in ("linear", "linear_train"):
        def act64(v):
            if case["act"] == "silu":
                return v * torch.sigmoid(v)
            if case["act"] == "gelu":
                return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
            return v * 1.0
        pre = torch.matmul(d["x"], d["weight"].t())
        if d["bias"] is not None:
            pre = pre + d["bias"]
        pre.requires_grad_()
        branch = act64(pre)
        out = branch.detach() if d["residual"] is None else branch.detach() + d["residual"]
        if op == "linear":
            return out
        (dp,) = torch.autograd.grad(branch, pre, d["d_out"])
        d_bias = dp.sum(0) if d["bias"] is not None else None
        return out, torch.matmul(dp, d["weight"]), torch.matmul(dp.t(), d["x"]), d_bias
    z = d["block"]
    branch = z / torch.sqrt((z * z).sum(1, keepdim=True) / case["H"] + EPS) * d["norm_weight"]
    if d["gate"] is not None:
        branch = branch * d["gate"]
    s = 0.5 * d["residual"] + branch
    kept = s.to(st["residual"].dtype).double()  # the next norm is taken of the stored stream
    y = kept / torch.sqrt((kept * kept).sum(1, keepdim=True) / case["H"] + EPS) * d["next_weight"]
    if case["scales"] == "row":
        scale = torch.maximum(y.abs().max(1, keepdim=True).values / 448, torch.tensor(2.0 ** -126, device=y.device).double())
        return s, y / scale, scale
    groups = y.view(T, -1, 32)
    largest = groups.abs().max(2).values
    e = torch.ceil(torch.log2(largest / 448)).clamp(min=-126)
    return s, (groups / torch.exp2(e)[:, :, None]).view(T, -1), torch.exp2(e)
