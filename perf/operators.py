"""Measured cases of the operators around the SSD core: what a Mamba-2 layer runs before and after
``ssd_forward`` and ``ssd_step``.

Four operators: the root-mean-square norm with the residual's addition or the gate, also with an
8-bit output and one scale per row; the matrix product with scales, bias, activation and residual in
its epilogue (the layer's in- and out-projection); the short causal convolution that turns the
in-projection's rows into the SSD core's x, B, C and dt; and its form for single tokens.

``run`` computes them in their plain form, elementary torch operations in fp32 rounded once at the
end, or, with ``own`` true, through the package's entry points. Layer sizes are those of the 2.7B-
and 370M-shaped layers (H heads of P channels, G groups of N state columns): d_inner = H*P, a model
width of d_inner / 2, an in-projection of 2*d_inner + 2*G*N + H channels laid out as [z | x B C | dt].
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126  # smallest normal fp32: a row of zeros keeps a scale it can be divided by

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "none": 0}


def listed():
    return [
        # The norm before the in-projection of one decode step of 64 sequences: the residual stream
        # in fp32, the norm's output in 8 bits for the projection. The smallest norm: latency.
        dict(name="norm residual decode", op="norm", M=64, D=2560, mode="residual", dtype="bf16",
             residual="f32", quantize=True, groups=1),
        # The gated norm after the SSD core of the 2.7B-shaped layer (4 x 4096 tokens), the gate read
        # in place from the in-projection's rows, 8-bit output for the out-projection. The largest.
        dict(name="norm gate prefill", op="norm", M=16384, D=5120, mode="gate", dtype="bf16",
             residual="none", quantize=True, groups=1),
        # A ragged batch at an odd width with fp32 activations, and a residual: the general path.
        dict(name="norm residual odd f32", op="norm", M=1531, D=1237, mode="residual", dtype="f32",
             residual="f32", quantize=False, groups=1),
        # Single-sequence decode of the 370M-shaped layer's out-projection with 8-bit operands, the
        # residual added: the smallest product, latency.
        dict(name="product e4m3 one token", op="linear", M=1, K=2048, N=1024, dtype="e4m3",
             out="bf16", bias=False, act="none", residual=True),
        # The in-projection of a decode step of 64 sequences, 2.7B-shaped layer: one read of the weights.
        dict(name="product bf16 decode", op="linear", M=64, K=2560, N=10576, dtype="bf16",
             out="bf16", bias=False, act="none", residual=False),
        # A ragged prompt through an MLP-like product with bias and activation: no size a tile fits.
        dict(name="product bf16 bias gelu ragged", op="linear", M=1003, K=1000, N=1777, dtype="bf16",
             out="bf16", bias=True, act="gelu", residual=False),
        # The out-projection of the 2.7B-shaped layer's prefill, residual added in fp32.
        dict(name="product bf16 residual prefill", op="linear", M=16384, K=5120, N=2560, dtype="bf16",
             out="f32", bias=False, act="none", residual=True),
        # The in-projection of the same prefill with 8-bit operands: the largest product.
        dict(name="product e4m3 prefill", op="linear", M=16384, K=2560, N=10576, dtype="e4m3",
             out="bf16", bias=False, act="none", residual=False),
        # The convolution of the 2.7B-shaped layer's prefill, read in place from the in-projection.
        dict(name="conv prefill", op="conv", B=4, L=4096, H=80, P=64, G=1, N=128, W=4, dtype="bf16"),
        # A short ragged prompt in fp32, a window of three, several groups.
        dict(name="conv ragged f32", op="conv", B=3, L=517, H=12, P=48, G=3, N=24, W=3, dtype="f32"),
        # The convolution of one decode step: 64 sequences of the 2.7B-shaped layer, and one sequence
        # of the 370M-shaped layer.
        dict(name="conv step decode", op="conv_step", B=64, H=80, P=64, G=1, N=128, W=4, dtype="bf16"),
        dict(name="conv step one token", op="conv_step", B=1, H=32, P=64, G=1, N=128, W=4, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "conv", "conv_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm":
        M = _log_int(rng, 1, 16384)
        D = _log_int(rng, 64, 8192)
        D = min(D, 16384 * 5120 // M)
        if rng.random() < 0.7:
            D = max(64, D // 64 * 64)
        mode = rng.choice(["none", "residual", "gate"])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if D % g == 0])
        residual = rng.choice([dtype, "f32"]) if mode == "residual" else "none"
        return dict(op=op, M=M, D=D, mode=mode, dtype=dtype, residual=residual,
                    quantize=rng.random() < 0.5, groups=groups)
    if op == "linear":
        dtype = rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "e4m3", "f32"])
        M = _log_int(rng, 1, 16384)
        N = _log_int(rng, 64, 10576)
        K = _log_int(rng, 128, 5120)
        K = min(K, 16384 * 2560 * 10576 // (M * N))
        grain = rng.choice([64, 64, 64, 64, 16, 16, 16, 1])
        K = max(64, K // grain * grain)
        if rng.random() < 0.7:
            N = N // 16 * 16
        out = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, M=M, K=K, N=N, dtype=dtype, out=out, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "none", "silu", "gelu"]), residual=rng.random() < 0.5)
    H = _log_int(rng, 2, 80)
    G = rng.choice([g for g in (1, 1, 2, 3, 8) if H % g == 0])
    P = rng.choice([64, 64, 64, 128, 48, 33])
    P = P if H * P <= 5120 else 64
    N = rng.choice([128, 128, 64, 16, 24, 37])
    W = rng.choice([4, 4, 3, 2])
    if op == "conv_step":
        return dict(op=op, B=_log_int(rng, 1, 256), H=H, P=P, G=G, N=N, W=W, dtype=dtype)
    tokens = _log_int(rng, 1, 16384 if dtype == "bf16" else 8192)
    B = min(tokens, _log_int(rng, 1, 16))
    return dict(op=op, B=B, L=max(1, tokens // B), H=H, P=P, G=G, N=N, W=W, dtype=dtype)


def _widths(c):
    d_inner = c["H"] * c["P"]
    conv = d_inner + 2 * c["G"] * c["N"]
    return d_inner, conv, d_inner + conv + c["H"]  # x, [x B C], the in-projection's row


def _rows_e4m3(v):
    """fp32 rows as 8-bit values and one scale per row."""
    scale = (v.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": dict(c)}
    dtype = _TYPES[c["dtype"]]
    if c["op"] == "norm":
        M, D = c["M"], c["D"]
        s["weight"] = 1 + 0.1 * normal(D)
        # rows of different sizes, as tokens have them
        s["x"] = (normal(M, D) * torch.exp(0.5 * normal(M, 1))).to(dtype)
        if c["mode"] == "residual":
            s["residual"] = (2 * normal(M, D)).to(_TYPES[c["residual"]])
        if c["mode"] == "gate":
            # z is the head of the in-projection's rows [z | x B C | dt]
            row = normal(M, 2 * D + 64).to(dtype)
            s["gate"] = row[:, :D]
    elif c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        x, w = normal(M, K), normal(N, K) / math.sqrt(K)
        if c["dtype"] == "e4m3":
            s["x"], s["x_scale"] = _rows_e4m3(x)
            s["w"], s["w_scale"] = _rows_e4m3(w)
        else:
            s["x"], s["w"] = x.to(dtype), w.to(dtype)
        s["bias"] = normal(N) if c["bias"] else None
        s["residual"] = normal(M, N).to(_TYPES[c["out"]]) if c["residual"] else None
    else:
        d_inner, conv, row = _widths(c)
        L = c["L"] if c["op"] == "conv" else 1
        proj = normal(c["B"], L, row).to(dtype)
        if c["op"] == "conv_step":
            proj = proj[:, 0]
        s["u"] = proj[..., d_inner:d_inner + conv]
        s["dt"] = proj[..., d_inner + conv:]
        s["weight"] = (torch.rand(conv, c["W"], generator=g, device="cuda") * 2 - 1) / math.sqrt(c["W"])
        s["bias"] = 0.1 * normal(conv)
        # softplus(dt_bias) spread over [1e-3, 1e-1], as the SSD core's step sizes are
        step = torch.exp(torch.rand(c["H"], generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["state"] = normal(c["B"], c["W"] - 1, conv).to(dtype)
    return s


def _plain_norm(s, c):
    v = s["x"].float()
    out = {}
    if c["mode"] == "residual":
        v = v + s["residual"].float()
        out["residual"] = v.to(_TYPES[c["residual"]])
    if c["mode"] == "gate":
        z = s["gate"].float()
        v = v * (z * torch.sigmoid(z))
    group = v.reshape(c["M"], c["groups"], -1)
    group = group * torch.rsqrt((group * group).mean(-1, keepdim=True) + EPS)
    y = group.reshape(c["M"], c["D"]) * s["weight"]
    if c["quantize"]:
        out["y"], out["scale"] = _rows_e4m3(y)
    else:
        out["y"] = y.to(_TYPES[c["dtype"]])
    return out


def _plain_linear(s, c):
    y = s["x"].float() @ s["w"].float().t()
    if c["dtype"] == "e4m3":
        y = y * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(_TYPES[c["out"]])


def _plain_conv(s, c):
    dtype = _TYPES[c["dtype"]]
    u = s["u"] if c["op"] == "conv" else s["u"][:, None]
    window = torch.cat([s["state"], u], 1)
    L, W = u.shape[1], c["W"]
    v = s["bias"] + sum(window[:, k:k + L].float() * s["weight"][:, k] for k in range(W))
    v = (v * torch.sigmoid(v)).to(dtype)
    d_inner, conv, _ = _widths(c)
    gn = c["G"] * c["N"]
    lead = u.shape[:2] if c["op"] == "conv" else u.shape[:1]
    raw = s["dt"].float() + s["dt_bias"]
    dt = torch.log1p(torch.exp(-raw.abs())) + raw.clamp_min(0)
    out = {"x": v[..., :d_inner].reshape(*lead, c["H"], c["P"]),
           "B": v[..., d_inner:d_inner + gn].reshape(*lead, c["G"], c["N"]),
           "C": v[..., d_inner + gn:].reshape(*lead, c["G"], c["N"]), "dt": dt}
    last = window[:, L:].clone()
    if c["op"] == "conv_step":
        s["state"].copy_(last)
        last = s["state"]
    return dict(out, state=last)


def _own(s, c):
    import selective_state_space_17_b200 as ssd
    if c["op"] == "norm":
        y, scale, residual = ssd.rms_norm(s["x"], s["weight"], residual=s.get("residual"),
                                          gate=s.get("gate"), eps=EPS, groups=c["groups"],
                                          quantize=c["quantize"])
        out = {"y": y}
        if scale is not None:
            out["scale"] = scale
        if residual is not None:
            out["residual"] = residual
        return out
    if c["op"] == "linear":
        return ssd.linear(s["x"], s["w"], bias=s["bias"], activation=c["act"],
                          residual=s["residual"], x_scale=s.get("x_scale"),
                          w_scale=s.get("w_scale"), out_dtype=_TYPES[c["out"]])
    sizes = (c["H"], c["P"], c["G"], c["N"])
    if c["op"] == "conv":
        x, Bm, Cm, dt, state = ssd.conv(s["u"], s["weight"], s["bias"], *sizes, dt=s["dt"],
                                        dt_bias=s["dt_bias"], initial_state=s["state"])
        return {"x": x, "B": Bm, "C": Cm, "dt": dt, "state": state}
    x, Bm, Cm, dt = ssd.conv_step(s["u"], s["weight"], s["bias"], s["state"], *sizes, dt=s["dt"],
                                  dt_bias=s["dt_bias"])
    return {"x": x, "B": Bm, "C": Cm, "dt": dt, "state": s["state"]}


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "norm":
        return _plain_norm(state, c)
    if c["op"] == "linear":
        return _plain_linear(state, c)
    return _plain_conv(state, c)


def work(case):
    c = case
    size = _BYTES[c["dtype"]]
    if c["op"] == "norm":
        n = c["M"] * c["D"]
        total = n * size + 4 * c["D"]
        total += 2 * n * _BYTES[c["residual"]] + (n * size if c["mode"] == "gate" else 0)
        total += n + 4 * c["M"] if c["quantize"] else n * size
        return {"bytes": total, "flops": n * (4 + 6 * (c["mode"] == "gate") + 3 * c["quantize"])}
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        out = _BYTES[c["out"]]
        total = (M + N) * K * size + M * N * out * (2 if c["residual"] else 1)
        total += 4 * N * c["bias"] + (4 * (M + N) if c["dtype"] == "e4m3" else 0)
        return {"bytes": total, "flops": 2 * M * N * K}
    _, conv, _ = _widths(c)
    tokens = c["B"] * (c["L"] if c["op"] == "conv" else 1)
    total = 2 * tokens * conv * size + tokens * c["H"] * (size + 4)
    total += 2 * c["B"] * (c["W"] - 1) * conv * size + 4 * conv * (c["W"] + 1) + 4 * c["H"]
    return {"bytes": total, "flops": tokens * conv * (2 * c["W"] + 5)}


def _exact_e4m3(v):
    """64-bit rows rounded to the nearest e4m3 value of their row's scale (ties to even): one sign,
    four exponent bits of bias 7, three mantissa bits, no infinity, largest value 448."""
    scale = torch.maximum(v.abs().max(1).values / E4M3_MAX, torch.full_like(v[:, 0], SCALE_MIN))
    q = v / scale.unsqueeze(1)
    exponent = torch.frexp(q)[1].clamp(min=-5) - 1  # 2^exponent <= |q|, subnormals below 2^-6
    step = torch.ldexp(torch.ones_like(q), exponent - 3)
    return torch.round(q / step) * step, scale


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        v = s["x"].double()
        out = {}
        if "residual" in s:
            v = s["residual"].double() + v
            out["residual"] = v
        if "gate" in s:
            z = s["gate"].double()
            v = v * z / (torch.exp(-z) + 1)
        parts = []
        for part in v.chunk(c["groups"], dim=1):
            parts.append(part / (part.pow(2).sum(1, keepdim=True) / part.shape[1] + EPS).sqrt())
        y = torch.cat(parts, 1) * s["weight"].double()
        if c["quantize"]:
            out["y"], out["scale"] = _exact_e4m3(y)
        else:
            out["y"] = y
        return out
    if c["op"] == "linear":
        x, w = s["x"].double(), s["w"].double()
        if c["dtype"] == "e4m3":
            x *= s["x_scale"].double().unsqueeze(1)
            w *= s["w_scale"].double().unsqueeze(1)
        y = torch.einsum("mk,nk->mn", x, w)
        if c["bias"]:
            y += s["bias"].double()
        if c["act"] == "silu":
            y = y / (1 + torch.exp(-y))
        if c["act"] == "gelu":
            y = y * torch.special.erfc(y / -math.sqrt(2.0)) / 2
        if c["residual"]:
            y += s["residual"].double()
        return y
    u = s["u"].double()
    u = u if c["op"] == "conv" else u.unsqueeze(1)
    line = torch.cat((s["state"].double(), u), dim=1)
    v = torch.einsum("blcw,cw->blc", line.unfold(1, c["W"], 1), s["weight"].double()) + s["bias"].double()
    v = v / (1 + torch.exp(-v))
    d_inner, conv, _ = _widths(c)
    x, Bm, Cm = v.split([d_inner, c["G"] * c["N"], c["G"] * c["N"]], dim=2)
    raw = s["dt"].double() + s["dt_bias"].double()
    return {"x": x, "B": Bm, "C": Cm, "dt": torch.logaddexp(raw, torch.zeros_like(raw)),
            "state": line[:, line.shape[1] - (c["W"] - 1):]}
