"""The operators of a W8A8 Mamba-2 layer around the SSD scan, as measured calls.

Four kinds of pass over one layer's data (H heads of P features, G groups of N state channels):

* ``add_norm``  residual addition + RMSNorm + INT8 codes with one scale per token
* ``gate_norm`` y * silu(z) + RMSNorm + INT8 codes with one scale per token
* ``matmul``    INT8 matrix product with a scale per token and per output channel
* ``conv``      causal depthwise convolution + SiLU of the scan's x, B, C and softplus of dt, for
                prompts (padded batches, a state to continue from); ``step`` is its one-token form

``run`` computes them with elementary torch operations, or with ``own`` set through
int8_quant_b200.  INT8 codes come back as the values they stand for (code * scale, bf16).
"""
import torch

own = False

P, N, W = 64, 128, 4          # head size, state size, convolution taps of every Mamba-2 layer here
EPS = 1e-5


def listed():
    return [
        # a decode batch of 8 on the 2.7B layer: latency is everything
        {"name": "add-norm-2.7b-decode", "op": "add_norm", "tokens": 8, "d": 2560, "residual": "fp32"},
        # an ordinary prompt of odd length on the 1.3B layer, residual stream in bf16
        {"name": "add-norm-1.3b-odd", "op": "add_norm", "tokens": 2047, "d": 2048, "residual": "bf16"},
        # the 2.7B prompt batch, 8 x 8192 tokens, residual stream in fp32
        {"name": "add-norm-2.7b", "op": "add_norm", "tokens": 65536, "d": 2560, "residual": "fp32"},
        # a large decode batch after the one-token scan step
        {"name": "gate-norm-2.7b-decode", "op": "gate_norm", "tokens": 128, "d": 5120},
        # the 16K-token prompt after its scan
        {"name": "gate-norm-2.7b-16k", "op": "gate_norm", "tokens": 16384, "d": 5120},
        # in_proj of a decode batch of 8: the weights' bytes bound it
        {"name": "in-proj-2.7b-decode", "op": "matmul", "tokens": 8, "k": 2560, "n": 10576, "bias": False},
        # out_proj of the 8B layer on a prompt of odd length
        {"name": "out-proj-8b-odd", "op": "matmul", "tokens": 1001, "k": 8192, "n": 4096, "bias": True},
        # in_proj of the 2.7B prompt batch: the tensor pipe bounds it
        {"name": "in-proj-2.7b", "op": "matmul", "tokens": 65536, "k": 2560, "n": 10576, "bias": False},
        # a padded batch of the 8B layer (8 groups) that continues from earlier segments
        {"name": "conv-8b-padded", "op": "conv", "batch": 4, "seqlen": 1001, "heads": 128, "groups": 8,
         "padded": True, "from_state": True},
        # the 2.7B prompt batch
        {"name": "conv-2.7b", "op": "conv", "batch": 8, "seqlen": 8192, "heads": 80, "groups": 1,
         "padded": False, "from_state": False},
        # one token of a small and of a large serving batch
        {"name": "conv-step-2.7b", "op": "step", "batch": 8, "heads": 80, "groups": 1},
        {"name": "conv-step-8b", "op": "step", "batch": 128, "heads": 128, "groups": 8},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["add_norm", "gate_norm", "matmul", "conv", "step"])
    if op == "add_norm":
        return {"op": op, "tokens": _log_int(rng, 1, 65536), "d": 16 * _log_int(rng, 8, 160),
                "residual": rng.choice(["fp32", "bf16", "none"])}
    if op == "gate_norm":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "d": 16 * _log_int(rng, 16, 512)}
    if op == "matmul":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "k": 16 * _log_int(rng, 16, 512),
                "n": _log_int(rng, 64, 18560), "bias": rng.random() < 0.5}
    heads = rng.choice([2, 8, 20, 40, 64, 80, 128])
    groups = rng.choice([g for g in (1, 2, 8) if heads % g == 0])
    if op == "step":
        return {"op": op, "batch": _log_int(rng, 1, 256), "heads": heads, "groups": groups}
    batch = _log_int(rng, 1, 8)
    return {"op": op, "batch": batch, "seqlen": _log_int(rng, 1, 32768 // batch), "heads": heads, "groups": groups,
            "padded": rng.random() < 0.5, "from_state": rng.random() < 0.5}


def _channels(case):
    return case["heads"] * P + 2 * case["groups"] * N


def _inputs(case, seed):
    """What the operator reads, made on the GPU from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    op, s = case["op"], {}
    if op == "add_norm":
        T, d = case["tokens"], case["d"]
        outliers = torch.where(torch.rand(d, generator=g, device=dev) < 0.005, 20.0, 1.0)
        s["x"] = (normal(T, d) * outliers).bfloat16()
        res = {"fp32": torch.float32, "bf16": torch.bfloat16, "none": None}[case["residual"]]
        s["residual"] = None if res is None else normal(T, d).mul_(3.0).to(res)
        s["weight"] = 1.0 + 0.2 * normal(d)
    elif op == "gate_norm":
        T, d = case["tokens"], case["d"]
        s["y"] = (normal(T, d) * torch.rand(T, 1, generator=g, device=dev).add_(0.5)).bfloat16()
        # z is the first d columns of in_proj's output rows
        s["zx"] = normal(T, 2 * d + 2 * N + d // P // 8 * 8).mul_(1.5).bfloat16()
        s["z"] = s["zx"][:, :d]
        s["weight"] = 1.0 + 0.2 * normal(d)
    elif op == "matmul":
        T, k, n = case["tokens"], case["k"], case["n"]
        s["q"] = normal(T, k).mul_(35.0).round_().clamp_(-127, 127).to(torch.int8)
        s["s_t"] = torch.rand(T, generator=g, device=dev).mul_(0.03).add_(0.01)
        s["Wq"] = normal(n, k).mul_(30.0).round_().clamp_(-127, 127).to(torch.int8)
        s["s_w"] = torch.rand(n, generator=g, device=dev).mul_(1e-3).add_(5e-4)
        s["bias"] = normal(n) if case["bias"] else None
    else:
        b, L = case["batch"], case.get("seqlen", 1)
        H, C = case["heads"], _channels(case)
        d = H * P
        rows = normal(b, L, d + C + (H + 7) // 8 * 8).bfloat16()         # in_proj's output: z | xBC | dt
        s["rows"], s["xbc"], s["dt_raw"] = rows, rows[:, :, d:d + C], rows[:, :, d + C:d + C + H]
        s["weight"] = 0.5 * normal(W, C)
        s["bias"] = 0.2 * normal(C)
        dt0 = torch.exp(torch.rand(H, generator=g, device=dev) * 4.605170186 - 6.907755279)
        s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))               # softplus(dt_bias) in [1e-3, 1e-1]
        s["lengths"] = None
        if case.get("padded"):
            s["lengths"] = torch.randint(0, L + 1, (b,), generator=g, device=dev, dtype=torch.int32)
        s["state"] = normal(b, W - 1, C).bfloat16() if op == "step" or case["from_state"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    new = lambda *shape, t=torch.bfloat16: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    op = case["op"]
    if op in ("add_norm", "gate_norm"):
        T, d = case["tokens"], case["d"]
        s["codes"], s["scale"], s["value"] = new(T, d, t=torch.int8), new(T, t=torch.float32), new(T, d)
        if op == "add_norm":
            s["residual_out"] = torch.empty_like(s["x"] if s["residual"] is None else s["residual"])
    elif op == "matmul":
        s["out"] = new(case["tokens"], case["n"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        b, L, H, G = case["batch"], case.get("seqlen", 1), case["heads"], case["groups"]
        lead = (b, L) if op == "conv" else (b,)
        s["x"], s["B"], s["C"] = new(*lead, H, P), new(*lead, G, N), new(*lead, G, N)
        s["dt"] = new(*lead, H, t=torch.float32)
        s["final"] = new(b, W - 1, _channels(case)) if op == "conv" else None
    return s


# ---------------------------------------------------------------- plain forms

def _codes(v, weight):
    """RMSNorm of the rows of v, quantised to 8 bits with one scale per row: (values, scales)."""
    p = v * weight
    top = p.abs().amax(-1)
    r = torch.rsqrt((v * v).mean(-1) + EPS)
    inv = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    codes = torch.round(p * inv[:, None])
    scale = torch.where(top > 0, top * r / 127.0, torch.ones_like(top))
    return (codes * scale[:, None]).bfloat16(), scale


def _plain_add_norm(s):
    v = s["x"].float()
    kept = torch.bfloat16
    if s["residual"] is not None:
        v, kept = v + s["residual"].float(), s["residual"].dtype
    stored = v.to(kept)
    value, scale = _codes(stored.float(), s["weight"])
    return {"value": value, "scale": scale, "residual": stored}


def _plain_gate_norm(s):
    z = s["z"].float()
    value, scale = _codes(s["y"].float() * (z / (1.0 + torch.exp(-z))), s["weight"])
    return {"value": value, "scale": scale}


def _plain_matmul(s):
    out = (s["q"].float() @ s["Wq"].float().T) * (s["s_t"][:, None] * s["s_w"])
    if s["bias"] is not None:
        out = out + s["bias"]
    return {"out": out.bfloat16()}


def _plain_conv(s, xbc, dt_raw, before):
    """xbc [b, L, C], dt_raw [b, L, H], before: the W - 1 inputs ahead of the first token."""
    b, L, C = xbc.shape
    c = s["case"]
    H, G = c["heads"], c["groups"]
    full = torch.cat([before, xbc], 1).float()
    w = s["weight"]
    u = full[:, :L] * w[0] + full[:, 1:L + 1] * w[1] + full[:, 2:L + 2] * w[2] + full[:, 3:] * w[3] + s["bias"]
    u = u / (1.0 + torch.exp(-u))
    v = dt_raw.float() + s["dt_bias"]
    dt = torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))
    end = torch.full((b,), L, device=u.device)
    if s["lengths"] is not None:
        end = s["lengths"].long()
        real = (torch.arange(L, device=u.device) < end[:, None])[:, :, None]
        u, dt = torch.where(real, u, torch.zeros_like(u)), torch.where(real, dt, torch.zeros_like(dt))
    at = end[:, None] + torch.arange(W - 1, device=u.device)
    final = torch.cat([before, xbc], 1).gather(1, at[:, :, None].expand(-1, -1, C))
    u = u.bfloat16()
    return {"x": u[..., :H * P].reshape(b, L, H, P), "dt": dt,
            "B": u[..., H * P:H * P + G * N].reshape(b, L, G, N),
            "C": u[..., H * P + G * N:].reshape(b, L, G, N), "state": final}


def _plain(s):
    op = s["case"]["op"]
    if op == "add_norm":
        return _plain_add_norm(s)
    if op == "gate_norm":
        return _plain_gate_norm(s)
    if op == "matmul":
        return _plain_matmul(s)
    if op == "step":
        r = _plain_conv(s, s["xbc"], s["dt_raw"], s["state"])
        s["state"].copy_(r["state"])                                  # the step updates the state it is given
        return {k: s["state"] if k == "state" else v[:, 0] for k, v in r.items()}
    before = s["state"]
    if before is None:
        before = torch.zeros_like(s["xbc"][:, :1]).expand(-1, W - 1, -1)
    return _plain_conv(s, s["xbc"], s["dt_raw"], before)


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import int8_quant_b200 as iq
    op = s["case"]["op"]
    if op == "add_norm":
        iq.ssd_add_rmsnorm_i8(s["x"], s["residual"], s["weight"], EPS, s["residual_out"], s["codes"], s["scale"],
                              s["value"])
        return {"value": s["value"], "scale": s["scale"], "residual": s["residual_out"]}
    if op == "gate_norm":
        iq.ssd_gated_rmsnorm_i8(s["y"], s["z"], s["weight"], EPS, s["codes"], s["scale"], s["value"])
        return {"value": s["value"], "scale": s["scale"]}
    if op == "matmul":
        iq.ssd_matmul_i8(s["q"], s["s_t"], s["Wq"], s["s_w"], s["bias"], s["out"], s["status"])
        return {"out": s["out"]}
    if op == "step":
        iq.ssd_conv_step_bf16(s["xbc"][:, 0], s["dt_raw"][:, 0], s["weight"], s["bias"], s["dt_bias"], s["state"],
                              s["x"], s["dt"], s["B"], s["C"])
        return {"x": s["x"], "dt": s["dt"], "B": s["B"], "C": s["C"], "state": s["state"]}
    iq.ssd_conv_fwd_bf16(s["xbc"], s["dt_raw"], s["weight"], s["bias"], s["dt_bias"], s["lengths"], s["state"],
                         s["x"], s["dt"], s["B"], s["C"], s["final"])
    return {"x": s["x"], "dt": s["dt"], "B": s["B"], "C": s["C"], "state": s["final"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- definitions in 64 bits

def _norm64(v, weight):
    p = v * weight.double()
    step = p.abs().max(dim=1, keepdim=True).values / 127
    codes = torch.where(step > 0, (p / step).round(), torch.zeros_like(p))
    scale = torch.where(step > 0, step / (v.square().mean(1, keepdim=True) + EPS).sqrt(), torch.ones_like(step))
    return codes * scale, scale[:, 0]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "add_norm":
        total = s["x"].double()
        kept = torch.bfloat16
        if s["residual"] is not None:
            total, kept = total + s["residual"].double(), s["residual"].dtype
        value, scale = _norm64(total.to(kept).double(), s["weight"])     # the norm is of the residual as stored
        return {"value": value, "scale": scale, "residual": total}
    if op == "gate_norm":
        z = s["z"].double()
        value, scale = _norm64(s["y"].double() * z * torch.sigmoid(z), s["weight"])
        return {"value": value, "scale": scale}
    if op == "matmul":
        out = torch.mm(s["q"].double(), s["Wq"].double().t())
        out *= s["s_t"].double()[:, None]
        out *= s["s_w"].double()
        if s["bias"] is not None:
            out += s["bias"].double()
        return {"out": out}
    b, L, C = s["xbc"].shape
    H, G = case["heads"], case["groups"]
    line = torch.zeros(b, W - 1 + L, C, dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        line[:, :W - 1] = s["state"].double()
    line[:, W - 1:] = s["xbc"].double()
    u = s["bias"].double().repeat(b, L, 1)
    for i in range(W):
        u.addcmul_(line[:, i:i + L], s["weight"][i].double())
    u *= torch.sigmoid(u)
    dt = torch.logaddexp(s["dt_raw"].double() + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    final = line[:, L:].clone()
    if s["lengths"] is not None:
        for row, n in enumerate(s["lengths"].tolist()):
            u[row, n:] = 0
            dt[row, n:] = 0
            final[row] = line[row, n:n + W - 1]
    d = H * P
    r = {"x": u[..., :d].reshape(b, L, H, P), "dt": dt, "B": u[..., d:d + G * N].reshape(b, L, G, N),
         "C": u[..., d + G * N:].reshape(b, L, G, N)}
    r = {k: v[:, 0] for k, v in r.items()} if op == "step" else r
    return {**r, "state": final}


def work(case):
    """Inputs read once, outputs written once (codes as 8 bits); two operations a product and sum."""
    op = case["op"]
    if op == "add_norm":
        T, d = case["tokens"], case["d"]
        res = {"fp32": 8, "bf16": 4, "none": 2}[case["residual"]]
        return {"bytes": T * d * (2 + res + 1) + 4 * T + 4 * d, "flops": 8 * T * d}
    if op == "gate_norm":
        T, d = case["tokens"], case["d"]
        return {"bytes": T * d * 5 + 4 * T + 4 * d, "flops": 12 * T * d}
    if op == "matmul":
        T, k, n = case["tokens"], case["k"], case["n"]
        return {"bytes": T * k + n * k + 2 * T * n + 4 * T + 8 * n, "flops": 2 * T * k * n}
    b, L, H, C = case["batch"], case.get("seqlen", 1), case["heads"], _channels(case)
    states = 2 if op == "step" or case.get("from_state") else 1
    return {"bytes": b * L * (4 * C + 6 * H) + states * 2 * b * (W - 1) * C + 4 * (W + 1) * C + 4 * H,
            "flops": b * L * (2 * W * C + 6 * C)}
