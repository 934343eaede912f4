"""Measured cases of the operators around the expert layer: the norms before and after a
block with its gate and residual scale, the dense gated feed-forward block (forward and
training step), and products of a few tokens with MXFP4 weights.

``run`` makes the calls a user makes where ``own`` is true; elsewhere it computes the
same operators from elementary torch operations in 32 bits.  ``exact`` restates each
operator in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = {"silu": 0, "gelu": 1}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token through the norm pair of a 2880-wide decoder layer
        dict(name="norm_decode", op="norm", T=1, H=2880, dtype="bf16", stream="bf16", gate="feature", scale=1.0),
        # a 4096-token prefill: per-token gate, scaled residual
        dict(name="norm_prefill", op="norm", T=4096, H=2880, dtype="bf16", stream="bf16", gate="token", scale=0.5),
        # a ragged training micro-batch in fp16 with a full gate
        dict(name="norm_bwd_ragged", op="norm_bwd", T=333, H=2880, dtype="f16", stream="f16", gate="full", scale=1.0),
        # a large training batch that keeps its residual stream in 32 bits
        dict(name="norm_bwd_large", op="norm_bwd", T=8192, H=4096, dtype="bf16", stream="f32", gate="feature",
             scale=0.7),
        # one generated token through a dense (shared) expert
        dict(name="ffn_decode", op="ffn", T=1, H=2880, I=2880, dtype="bf16", act="silu"),
        # a decode batch through a Mixtral-sized dense layer
        dict(name="ffn_batch", op="ffn", T=64, H=4096, I=14336, dtype="f16", act="silu"),
        # a prefill chunk through the same layer
        dict(name="ffn_prefill", op="ffn", T=2048, H=4096, I=14336, dtype="bf16", act="silu"),
        # a ragged training step: forward, then every gradient
        dict(name="ffn_train_ragged", op="ffn_train", T=1001, H=2880, I=2880, dtype="f16", act="gelu"),
        # a large training step
        dict(name="ffn_train_large", op="ffn_train", T=4096, H=4096, I=14336, dtype="bf16", act="silu"),
        # one token, one square MXFP4 projection
        dict(name="matvec_decode", op="matvec", T=1, N=2880, K=2880, dtype="bf16", kind="plain", act="silu"),
        # a decode batch of 16 through gate and up rows in MXFP4
        dict(name="matvec_gated", op="matvec", T=16, N=14336, K=4096, dtype="f16", kind="gated", act="silu"),
        # one token through a very tall MXFP4 projection
        dict(name="matvec_tall", op="matvec", T=1, N=131072, K=4096, dtype="bf16", kind="plain", act="silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ffn", "ffn_train", "matvec"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("norm", "norm_bwd"):
        return dict(op=op, T=_log_int(rng, 1, 8192), H=8 * _log_int(rng, 8, 512), dtype=dtype,
                    stream=rng.choice([dtype, "f32"]), gate=rng.choice(["none", "feature", "token", "full"]),
                    scale=rng.choice([1.0, 0.5, 0.7]))
    if op in ("ffn", "ffn_train"):
        return dict(op=op, T=_log_int(rng, 1, 2048), H=8 * _log_int(rng, 8, 512), I=8 * _log_int(rng, 8, 1792),
                    dtype=dtype, act=rng.choice(["silu", "gelu"]))
    return dict(op=op, T=_log_int(rng, 1, 64), N=_log_int(rng, 32, 32768), K=32 * _log_int(rng, 1, 256), dtype=dtype,
                kind=rng.choice(["plain", "gated"]), act=rng.choice(["silu", "gelu"]))


def work(case):
    T = case["T"]
    if case["op"] in ("norm", "norm_bwd"):
        H, a = case["H"], 2
        s = 4 if case["stream"] == "f32" else 2
        gate = {"none": 0, "feature": a * H, "token": 4 * T, "full": a * T * H}[case["gate"]]
        if case["op"] == "norm":
            return {"bytes": T * H * (2 * a + 2 * s) + 2 * a * H + gate, "flops": 12 * T * H}
        gate += {"none": 0, "feature": 4 * H, "token": 4 * T, "full": a * T * H}[case["gate"]]
        return {"bytes": T * H * (3 * a + 3 * s) + 2 * a * H + 8 * H + gate, "flops": 30 * T * H}
    if case["op"] in ("ffn", "ffn_train"):
        H, I = case["H"], case["I"]
        fwd = {"bytes": 2 * (3 * H * I + 2 * T * H), "flops": 6 * T * H * I}
        if case["op"] == "ffn":
            return fwd
        # out, then d_x and both weight gradients; x, d_out and the weights read once
        return {"bytes": 2 * (6 * H * I + 4 * T * H), "flops": 18 * T * H * I}
    N, K = case["N"], case["K"]
    rows = 2 * N if case["kind"] == "gated" else N
    return {"bytes": rows * (K // 2 + K // 32) + 4 * rows + 2 * T * (K + N), "flops": 2 * T * rows * K}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T = case["T"]

    def rand(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dtype)

    st = dict(case=case)
    if case["op"] in ("norm", "norm_bwd"):
        H, sdt = case["H"], DTYPES[case["stream"]]
        st["block"] = rand(T, H)
        st["residual"] = rand(T, H, std=2.0, dtype=sdt)
        st["norm_weight"] = rand(H, std=0.25, mean=1.0)
        st["next_weight"] = rand(H, std=0.25, mean=1.0)
        kind = case["gate"]
        st["gate"] = None
        if kind == "feature":
            st["gate"] = rand(H, std=0.3, mean=0.5)
        elif kind == "token":
            st["gate"] = torch.sigmoid(rand(T, 1, dtype=torch.float32))
        elif kind == "full":
            st["gate"] = rand(T, H, std=0.5)
        if case["op"] == "norm_bwd":
            # the stream that the forward left behind, and both gradients
            st["stream"] = rand(T, H, std=2.0, dtype=sdt)
            st["d_stream"] = rand(T, H, std=1.0, dtype=sdt)
            st["d_out"] = rand(T, H)
        return st
    if case["op"] in ("ffn", "ffn_train"):
        H, I = case["H"], case["I"]
        st["x"] = rand(T, H)
        st["w_gateup"] = rand(2 * I, H, std=1.0 / math.sqrt(H))
        st["w_down"] = rand(H, I, std=1.0 / math.sqrt(I))
        if case["op"] == "ffn_train":
            st["d_out"] = rand(T, H)
        return st
    N, K = case["N"], case["K"]
    rows = 2 * N if case["kind"] == "gated" else N
    st["x"] = rand(T, K)
    st["codes"] = torch.randint(0, 256, (rows, K // 2), generator=g, device=dev, dtype=torch.uint8)
    st["scales"] = torch.randint(120, 125, (rows, K // 32), generator=g, device=dev, dtype=torch.uint8)
    st["bias"] = rand(rows, dtype=torch.float32)
    if own:
        import mxfp4_expert_layer_gb300 as moe
        kind = moe.MOE_WEIGHTS_GATEUP if case["kind"] == "gated" else moe.MOE_WEIGHTS_DOWN
        # laid out once, as a program that decodes with these weights does at load
        st["weight"] = moe.MatvecMXFP4(st["codes"], st["scales"], kind=kind, bias=st["bias"], act=ACTS[case["act"]])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import mxfp4_expert_layer_gb300 as moe
        return _own(moe, op, state)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "ffn": _ffn, "ffn_train": _ffn_train, "matvec": _matvec}[op](state)


def _own(moe, op, st):
    case = st["case"]
    if op == "norm":
        return moe.block_norm(st["block"], st["residual"], norm_weight=st["norm_weight"], gate=st["gate"],
                              residual_scale=case["scale"], next_weight=st["next_weight"], eps=EPS)
    if op == "norm_bwd":
        g = moe.block_norm_backward(st["d_stream"], st["d_out"], st["block"], st["stream"],
                                    norm_weight=st["norm_weight"], gate=st["gate"], residual_scale=case["scale"],
                                    next_weight=st["next_weight"], eps=EPS)
        return g.block, g.residual, g.norm_weight, g.gate, g.next_weight
    if op == "ffn":
        return moe.ffn_forward(st["x"], st["w_gateup"], st["w_down"], act=ACTS[case["act"]])
    if op == "ffn_train":
        out, gateup = moe.ffn_forward(st["x"], st["w_gateup"], st["w_down"], act=ACTS[case["act"]], save=True)
        return (out,) + tuple(moe.ffn_backward(st["d_out"], st["x"], gateup, st["w_gateup"], st["w_down"],
                                               act=ACTS[case["act"]]))
    return st["weight"](st["x"])


# ------------------------------------------------------------------ plain forms
def _norm(st):
    f = torch.Tensor.float
    z, r = f(st["block"]), f(st["residual"])
    p = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * f(st["norm_weight"])
    if st["gate"] is not None:
        p = p * f(st["gate"])
    s = (st["case"]["scale"] * r + p).to(st["residual"].dtype)
    sf = f(s)
    y = sf * torch.rsqrt(sf.square().mean(1, keepdim=True) + EPS) * f(st["next_weight"])
    return s, y.to(st["block"].dtype)


def _norm_bwd(st):
    f = torch.Tensor.float
    z, s, ds, dy = f(st["block"]), f(st["stream"]), f(st["d_stream"]), f(st["d_out"])
    wp, wn, gate = f(st["norm_weight"]), f(st["next_weight"]), st["gate"]
    rs = torch.rsqrt(s.square().mean(1, keepdim=True) + EPS)
    rz = torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
    u = dy * wn
    ds = ds + rs * u - s * (rs * rs * rs * (u * s).mean(1, keepdim=True))
    d_next = (dy * s * rs).sum(0)
    zn = z * rz
    n = zn * wp
    d_gate, p = None, ds
    if gate is not None:
        p = ds * f(gate)
        d_gate = ds * n
        if gate.dim() == 1:
            d_gate = d_gate.sum(0)
        elif gate.shape[1] == 1:
            d_gate = d_gate.sum(1, keepdim=True)
        else:
            d_gate = d_gate.to(gate.dtype)
    d_norm = (p * zn).sum(0)
    v = p * wp
    dz = rz * v - z * (rz * rz * rz * (v * z).mean(1, keepdim=True))
    return dz.to(st["block"].dtype), (st["case"]["scale"] * ds).to(st["stream"].dtype), d_norm, d_gate, d_next


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    t = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * (0.7978845608028654 * (1.0 + 3 * 0.044715 * g * g))


def _ffn(st):
    I = st["case"]["I"]
    gu = st["x"].float() @ st["w_gateup"].float().t()
    h = _act(gu[:, :I], st["case"]["act"]) * gu[:, I:]
    return (h @ st["w_down"].float().t()).to(st["x"].dtype)


def _ffn_train(st):
    I, act, dt = st["case"]["I"], st["case"]["act"], st["x"].dtype
    x, wgu, wd, d_out = (st[k].float() for k in ("x", "w_gateup", "w_down", "d_out"))
    gu = x @ wgu.t()
    g, u = gu[:, :I], gu[:, I:]
    a = _act(g, act)
    h = a * u
    out = h @ wd.t()
    dh = d_out @ wd
    dgu = torch.cat((dh * u * _act_grad(g, act), dh * a), 1)
    return out.to(dt), (dgu @ wgu).to(dt), (dgu.t() @ x).to(dt), (d_out.t() @ h).to(dt)


def _dequantised(codes, scales, dtype):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device, dtype=dtype)
    rows, half = codes.shape
    idx = torch.stack((codes & 15, codes >> 4), -1).view(-1).int()
    w = table.index_select(0, idx).view(rows, half // 16, 32)
    return (w * torch.exp2(scales.to(dtype) - 127.0).unsqueeze(-1)).view(rows, 2 * half)


def _matvec(st):
    case = st["case"]
    y = st["x"].float() @ _dequantised(st["codes"], st["scales"], torch.float32).t() + st["bias"]
    if case["kind"] == "gated":
        N = case["N"]
        y = _act(y[:, :N], case["act"]) * y[:, N:]
    return y.to(st["x"].dtype)


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in st.items()}
    op = case["op"]
    if op == "norm":
        z = d["block"]
        branch = z / torch.sqrt((z * z).sum(1, keepdim=True) / case["H"] + EPS) * d["norm_weight"]
        if d["gate"] is not None:
            branch = branch * d["gate"]
        s = case["scale"] * d["residual"] + branch
        kept = s.to(st["residual"].dtype).double()  # the next norm is taken of the stored stream
        return s, kept / torch.sqrt((kept * kept).sum(1, keepdim=True) / case["H"] + EPS) * d["next_weight"]
    if op == "norm_bwd":
        def rms_norm(v, w):
            return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w
        # autograd of the definition, the stream taken as an input of its own norm
        z = d["block"].requires_grad_()
        wp, wn = d["norm_weight"].requires_grad_(), d["next_weight"].requires_grad_()
        s = d["stream"].requires_grad_()
        (ds_norm, d_next) = torch.autograd.grad(rms_norm(s, wn), (s, wn), d["d_out"])
        ds = d["d_stream"] + ds_norm
        gate = d["gate"]
        if gate is None:
            dz, dwp = torch.autograd.grad(rms_norm(z, wp), (z, wp), ds)
            return dz, case["scale"] * ds, dwp, None, d_next
        gate.requires_grad_()
        dz, dwp, dg = torch.autograd.grad(gate * rms_norm(z, wp), (z, wp, gate), ds)
        return dz, case["scale"] * ds, dwp, dg, d_next

    def act64(v, name):
        if name == "silu":
            return v * torch.sigmoid(v)
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))

    if op in ("ffn", "ffn_train"):
        I, x, wgu, wd = case["I"], d["x"], d["w_gateup"], d["w_down"]
        g, u = torch.matmul(x, wgu[:I].t()), torch.matmul(x, wgu[I:].t())
        if op == "ffn":
            return torch.matmul(act64(g, case["act"]) * u, wd.t())
        g.requires_grad_()
        u.requires_grad_()
        h = act64(g, case["act"]) * u
        dh = torch.matmul(d["d_out"], wd)
        dg, du = torch.autograd.grad(h, (g, u), dh)
        dx = torch.matmul(dg, wgu[:I]) + torch.matmul(du, wgu[I:])
        dwgu = torch.cat((torch.matmul(dg.t(), x), torch.matmul(du.t(), x)))
        h = h.detach()
        return torch.matmul(h, wd.t()), dx, dwgu, torch.matmul(d["d_out"].t(), h)
    # MXFP4: value = sign * E2M1 magnitude * 2^(scale - 127), the even column in the low nibble
    rows, K = st["codes"].shape[0], case["K"]
    y = torch.empty(case["T"], rows, dtype=torch.float64, device=d["x"].device)
    magnitude = torch.tensor(E2M1, dtype=torch.float64, device=d["x"].device)
    for r0 in range(0, rows, 16384):
        c = st["codes"][r0:r0 + 16384].long()
        w = torch.empty(c.shape[0], K, dtype=torch.float64, device=c.device)
        for odd in (0, 1):
            code = (c >> (4 * odd)) & 15
            w[:, odd::2] = magnitude[code & 7] * (1 - 2 * (code >> 3)).double()
        e = st["scales"][r0:r0 + 16384].double().repeat_interleave(32, 1)
        y[:, r0:r0 + 16384] = torch.matmul(d["x"], (w * torch.pow(2.0, e - 127)).t())
    y = y + d["bias"]
    if case["kind"] == "gated":
        return act64(y[:, :case["N"]], case["act"]) * y[:, case["N"]:]
    return y
