"""The operators around the SSD core (rms_norm, linear, conv, conv_step) against
their formulas in 64 bits, at the sizes, strides and values where they can go
wrong, and a run of them together with the SSD core.

Tolerances. U = 2^-24 bounds an fp32 rounding relative to its result and
HALF[t] the rounding to the output's type; a sum of n terms in fp32, in any
order, is off by at most n U times the sum of their magnitudes. Each test adds
up the roundings of its formula.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, E4M3)}
E4M3_SUBNORMAL_HALF = 2.0 ** -10  # half the distance of e4m3 values below 2^-6


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_17_b200 as _ssd
    return _ssd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def check(name, got, want, tol):
    """|got - want| <= tol everywhere, NaN where and only where the formula has NaN."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, name
    assert torch.equal(got.isnan(), want.isnan()), f"{name}: NaN in other places"
    same = got.isinf() & (got == want)
    bad = ((got - want).abs() > tol) & ~same & ~want.isnan()
    if bad.any():
        at = bad.nonzero()[0].tolist()
        tol = torch.as_tensor(tol, device=got.device).expand(got.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{got[tuple(at)]} for {want[tuple(at)]}, tolerance {tol[tuple(at)]}")


# ---------------------------------------------------------------- rms_norm

def norm64(x, weight, residual, gate, eps, groups):
    v = x.double()
    if residual is not None:
        v = v + residual.double()
    if gate is not None:
        v = v * torch.nn.functional.silu(gate.double())
    parts = v.reshape(*v.shape[:-1], groups, -1)
    y = parts / torch.sqrt((parts ** 2).mean(-1, keepdim=True) + eps)
    return v, y.reshape(v.shape) * weight.double()


def norm_rel(D, groups):
    """Relative error of y in fp32: v has one rounding, silu of |z| < 8 its
    exponential's (2 + 1.45 |z| <= 14 units) and the division's (4), a square
    and the sum of at most D / 32 + 42 terms in a lane, a warp and a CTA (the
    square root halves it), mean, eps, root (4), and the products (4)."""
    return (1 + 20 + (D / groups / 32 + 44) / 2 + 8 + 4) * U


def check_norm(ssd, x, weight, residual=None, gate=None, groups=1, eps=1e-5, quantize=False, **kw):
    r0 = None if residual is None else residual.clone()
    x0 = x.clone()
    y, s, ro = ssd.rms_norm(x, weight, residual=residual, gate=gate, eps=eps, groups=groups,
                            quantize=quantize, **kw)
    v, want = norm64(x0, weight, r0, gate, eps, groups)
    rel = norm_rel(x.shape[-1], groups)
    if residual is not None:
        check("residual", ro, v, v.abs() * HALF[ro.dtype] * 1.01)
    else:
        assert ro is None
    if quantize:
        top = want.abs().amax(-1)
        scale = torch.where(top.isnan(), top, (top / 448).clamp_min(2.0 ** -126))
        check("scale", s, scale, scale.abs() * (rel + 2 * U))
        got = y.double() * s.double()[..., None]
        # two more products, then the rounding to e4m3 (and below its normal range)
        tol = want.abs() * (rel + 4 * U) * 1.1 + want.abs() * HALF[E4M3] + scale[..., None] * E4M3_SUBNORMAL_HALF
        check("y", got, want, tol * (1 + 2.0 ** -20))
    else:
        assert s is None and y.dtype == x.dtype
        check("y", y, want, want.abs() * (rel + HALF[x.dtype]) * (1 + 2.0 ** -20))


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("mode", ["plain", "residual", "residual_f32", "gate"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D,groups", [
    (1, 1, 1), (3, 8, 1), (5, 7, 7), (1, 64, 1), (7, 256, 1), (9, 264, 1), (33, 1000, 1), (3, 1237, 1),
    (17, 2560, 8), (2, 5120, 1), (600, 512, 4), (3, 10240, 32), (4, 4100, 1), (700, 5120, 8), (650, 2570, 1), (2500, 77, 1), (2, 16392, 1), (1, 20001, 3),
])
def test_norm(ssd, rows, D, groups, dtype, mode, quantize):
    g = gen(rows * 31 + D)
    x = randn(g, rows, D, dtype=dtype) * torch.exp(randn(g, rows, 1)).to(dtype)
    weight = 1 + 0.2 * randn(g, D)
    kw = {}
    if mode.startswith("residual"):
        kw["residual"] = randn(g, rows, D, dtype=F32 if mode.endswith("f32") else dtype, scale=3.0)
    if mode == "gate":
        kw["gate"] = randn(g, rows, D, dtype=dtype)
    check_norm(ssd, x, weight, groups=groups, quantize=quantize, **kw)


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("offset,pitch", [(0, 640), (8, 648), (3, 517), (1, 513)])
def test_norm_gate_is_read_from_a_wider_row(ssd, offset, pitch, quantize):
    g = gen(5)
    row = randn(g, 4, 6, pitch, dtype=BF16)
    check_norm(ssd, randn(g, 4, 6, 512, dtype=BF16), 1 + 0.1 * randn(g, 512),
               gate=row[..., offset:offset + 512], quantize=quantize)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [96, 97, 4104, 40000])
def test_norm_in_place(ssd, D, dtype):
    """y over x and residual_out over the residual, kept rows and rows read twice."""
    g = gen(D)
    x, r = randn(g, 5, D, dtype=dtype), randn(g, 5, D)
    check_norm(ssd, x, 1 + 0.1 * randn(g, D), residual=r, residual_out=r, y=x)


@pytest.mark.parametrize("D,groups", [(64, 1), (4096, 1), (1028, 2), (70000, 1)])
def test_norm_rows_of_zeros_infinities_and_nans(ssd, D, groups):
    g = gen(9)
    x = randn(g, 6, D)
    x[0] = 0                      # zeros: y = 0, the smallest scale
    x[1, D // 2] = float("nan")
    x[2, 1] = float("inf")        # sum of squares inf: 0, and NaN in the place itself
    x[3] *= 1e-30                 # below eps
    x[4] *= 1e15                  # squares stay finite
    weight = torch.ones(D, device="cuda")
    v, want = norm64(x, weight, None, None, 1e-5, groups)
    y, _, _ = ssd.rms_norm(x, weight, groups=groups)
    check("y", y, want, want.abs() * (norm_rel(D, groups) + HALF[F32]))
    q, s, _ = ssd.rms_norm(x, weight, groups=groups, quantize=True)
    assert (q[0].float() == 0).all() and s[0] == 2.0 ** -126
    assert s[1].isnan() and s[2].isnan()
    assert q[1].float().isnan().all() and q[2].float().isnan().all()
    ok = [0, 3, 4, 5]
    check("q", (q.double() * s.double()[:, None])[ok], want[ok],
          want[ok].abs() * (HALF[E4M3] + norm_rel(D, groups) + 8 * U) + s[ok].double()[:, None] * E4M3_SUBNORMAL_HALF * 1.001)


def test_norm_many_rows_and_no_rows(ssd):
    g = gen(3)
    check_norm(ssd, randn(g, 70001, 64, dtype=BF16), 1 + 0.1 * randn(g, 64), quantize=True)
    y, s, r = ssd.rms_norm(torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), quantize=True)
    assert y.shape == (0, 64) and s.shape == (0,) and r is None


# ------------------------------------------------------------------- linear

def quantize_rows(v):
    scale = (v.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    return (v / scale[:, None]).clamp(-448, 448).to(E4M3), scale


ACT64 = {"none": lambda v: v, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}


def operands(g, M, N, K, dtype):
    x, w = randn(g, M, K), randn(g, N, K, scale=1 / math.sqrt(K))
    if dtype is E4M3:
        (xq, xs), (wq, ws) = quantize_rows(x), quantize_rows(w)
        return xq, wq, dict(x_scale=xs, w_scale=ws)
    return x.to(dtype), w.to(dtype), {}


def linear_tol(x, w, scales, bias, act, want, out, K):
    """K products in fp32, truncated rather than rounded where the tensor cores
    add (2 U a step), the scales' two products, the bias, an activation of slope
    at most 1.13 with twenty units of its own, the residual, the output."""
    size = x.double().abs() @ w.double().abs().t()
    if scales:
        size = size * scales["x_scale"].double()[:, None] * scales["w_scale"].double()
    if bias is not None:
        size = size + bias.double().abs()
    slope = 1.0 if act == "none" else 1.13
    return size * (2 * K + 8) * U * slope + want.abs() * (HALF[out] * 1.01 + 4 * U) + size * 20 * U * (act != "none")


def check_linear(ssd, M, N, K, dtype, out, bias=False, act="none", residual=False, seed=0, x=None):
    g = gen(seed + M + 7 * N + 13 * K)
    x0, w, scales = operands(g, M, N, K, dtype)
    x = x0 if x is None else x(x0)
    b = randn(g, N) if bias else None
    r = randn(g, M, N, dtype=out) if residual else None
    y = ssd.linear(x, w, bias=b, activation=act, residual=r, out_dtype=out, **scales)
    acc = x.double() @ w.double().t()
    if scales:
        acc = acc * scales["x_scale"].double()[:, None] * scales["w_scale"].double()
    if bias:
        acc = acc + b.double()
    want = ACT64[act](acc)
    tol = linear_tol(x, w, scales, b, act, want, out, K)
    if residual:
        want = want + r.double()
        tol = tol + (want.abs() + r.double().abs()) * (HALF[out] * 1.01)
    assert y.dtype == out
    check("y", y, want, tol)


@pytest.mark.parametrize("dtype", [F32, BF16, E4M3])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 64, 16), (2, 8, 64), (3, 130, 32), (1, 1024, 2048), (5, 777, 1000), (16, 128, 48),
    (17, 256, 2560), (64, 200, 80), (64, 2576, 512), (65, 64, 65), (100, 129, 4096), (128, 128, 128),
    (129, 300, 272), (200, 1777, 1000), (256, 264, 160), (257, 513, 96), (333, 100, 333), (520, 1040, 1040),
])
def test_linear_sizes(ssd, M, N, K, dtype):
    out = F32 if (M + N) % 2 or dtype is F32 else BF16
    check_linear(ssd, M, N, K, dtype, out)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bias,residual", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (E4M3, BF16), (E4M3, F32)])
@pytest.mark.parametrize("M,N,K", [(3, 72, 96), (70, 333, 640), (300, 784, 2048)])
def test_linear_epilogue(ssd, M, N, K, dtype, out, bias, residual, act):
    check_linear(ssd, M, N, K, dtype, out, bias, act, residual)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("M,N,K", [(2048, 2560, 512), (2051, 1784, 1040), (4096, 4384, 256), (1100, 5000, 768)])
def test_linear_many_rows(ssd, M, N, K, dtype):
    check_linear(ssd, M, N, K, dtype, BF16, bias=True, act="silu", residual=True)


@pytest.mark.parametrize("variant", [1, 2, 3])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32), (E4M3, BF16), (E4M3, F32)])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (7, 100, 208), (130, 264, 1040), (300, 520, 77), (513, 1000, 640)])
def test_linear_kernels(ssd, M, N, K, dtype, out, variant):
    """Each kernel on the same products, whatever the automatic choice."""
    ssd.layer.set_linear_variant(variant)
    try:
        check_linear(ssd, M, N, K, dtype, out, bias=True, act="gelu", residual=True)
        check_linear(ssd, M, N, K, dtype, out, residual=True)
    finally:
        ssd.layer.set_linear_variant(0)


@pytest.mark.parametrize("M", [3, 70, 1100])
def test_linear_fp32_beyond_bf16(ssd, M):
    """fp32 operands that three bf16 parts cannot hold: the products of
    infinities, NaN and the largest values are those of fp32; and scales at the
    ends of the range keep their 24 bits."""
    g = gen(8)
    x, w = randn(g, M, 96), randn(g, 72, 96)
    w[5] = 0.5  # a row that one bf16 part holds: its other parts are zeros
    bad = x.clone()
    bad[0, 3], bad[1, 4], bad[2, 5] = float("inf"), float("nan"), 3.4e38
    small = w * 2.0 ** -20
    got = ssd.linear(bad, small)
    want = bad.double() @ small.double().t()
    size = bad.double().abs() @ small.double().abs().t()
    check("y", got, want, torch.where(size.isfinite(), size * 220 * U, torch.zeros_like(size)))
    again = ssd.linear(x, w)
    check("y", again, x.double() @ w.double().t(), (x.double().abs() @ w.double().abs().t()) * 220 * U)
    for sx, sw in ((2.0 ** 90, 2.0 ** -60), (2.0 ** -90, 2.0 ** 60)):
        got = ssd.linear(x * sx, w * sw)
        check("y", got, (x.double() * sx) @ (w.double() * sw).t(),
              ((x.double() * sx).abs() @ (w.double() * sw).abs().t()) * 220 * U)


def test_linear_fp32_captured_and_replayed(ssd):
    """The copies of one graph's call are its own: two graphs replayed in turn,
    and an eager call between, with a value that does not split in one of them."""
    g = gen(9)
    x, w = randn(g, 100, 130), randn(g, 90, 130)
    graphs = []
    ssd.linear(x, w)
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        xi = x.clone()
        with torch.cuda.graph(graph):
            y = ssd.linear(xi, w)
        graphs.append((graph, xi, y))
    want = ssd.linear(x, w)
    graphs[0][1][7, 7] = float("inf")
    for _ in range(3):
        for graph, _, _ in graphs:
            graph.replay()
        assert torch.equal(ssd.linear(x, w), want)
        assert torch.equal(graphs[1][2], want)
        y = graphs[0][2]
        assert not y[7].isfinite().any()
        rest = [m for m in range(100) if m != 7]
        size = x.double().abs() @ w.double().abs().t()
        check("y", y[rest], (x.double() @ w.double().t())[rest], (size * 300 * U)[rest])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,pitch", [(0, 320), (8, 328), (3, 301), (1, 298)])
@pytest.mark.parametrize("M", [1, 40, 700])
def test_linear_reads_rows_of_a_wider_buffer(ssd, M, offset, pitch, dtype):
    def view(x):
        row = torch.full((M, pitch), float("nan"), dtype=dtype, device="cuda")
        row[:, offset:offset + 296] = x
        return row[:, offset:offset + 296]
    check_linear(ssd, M, 136, 296, dtype, dtype, x=view)


def test_linear_keeps_the_shape_of_its_rows_and_adds_in_place(ssd):
    g = gen(1)
    x, w = randn(g, 2, 3, 64, dtype=BF16), randn(g, 24, 64, dtype=BF16, scale=0.125)
    y = randn(g, 2, 3, 24, dtype=BF16)
    before = y.double().clone()
    out = ssd.linear(x, w, residual=y, y=y)
    assert out is y
    prod = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().t().abs()
    check("y", y, prod + before, size * 140 * U + (prod + before).abs() * HALF[BF16] * 1.01)


def test_linear_infinities_and_nans_stay_in_their_rows(ssd):
    g = gen(2)
    for M in (8, 300):
        x, w = randn(g, M, 256, dtype=BF16), randn(g, 200, 256, dtype=BF16)
        x[3, 5], x[5, 7] = float("nan"), float("inf")
        y = ssd.linear(x, w, out_dtype=F32)
        assert y[3].isnan().all() and not y[5].isfinite().any()
        rest = [m for m in range(M) if m not in (3, 5)]
        assert y[rest].isfinite().all()


def test_linear_writes_nothing_but_its_output(ssd):
    """Odd sizes: what lies around the output keeps its values."""
    g = gen(3)
    for M, N, K in ((1, 17, 64), (37, 65, 64), (130, 200, 128), (515, 333, 64), (2055, 1112, 64)):
        buf = torch.full((M * N + 512,), 7.0, dtype=BF16, device="cuda")
        y = buf[256:256 + M * N].view(M, N)
        x, w = randn(g, M, K, dtype=BF16), randn(g, N, K, dtype=BF16)
        ssd.linear(x, w, y=y)
        assert (buf[:256] == 7).all() and (buf[256 + M * N:] == 7).all(), (M, N, K)
        want = x.double() @ w.double().t()
        check("y", y, want, want.abs() * HALF[BF16] * 1.01 + (x.double().abs() @ w.double().t().abs()) * (2 * K + 8) * U)


# ---------------------------------------------------------- conv, conv_step

def conv64(u, weight, bias, state, silu):
    W = weight.shape[1]
    line = torch.cat([state.double(), u.double()], 1)
    terms = line.unfold(1, W, 1) * weight.double()
    v = terms.sum(-1) + (0 if bias is None else bias.double())
    size = terms.abs().sum(-1) + (0 if bias is None else bias.double().abs())
    return (torch.nn.functional.silu(v) if silu else v), size, line[:, u.shape[1]:]


def conv_case(B, L, H, P, G, N, W, dtype, seed=0, pad=0):
    """u and dt as views of the in-projection's rows [z | x B C | dt | pad]."""
    g = gen(seed + B + 5 * L + H)
    C = H * P + 2 * G * N
    proj = randn(g, B, L, H * P + C + H + pad, dtype=dtype)
    return dict(u=proj[..., H * P:H * P + C], dt=proj[..., H * P + C:H * P + C + H],
                weight=randn(g, C, W, scale=0.5), bias=0.3 * randn(g, C), dt_bias=randn(g, H) - 3,
                state=randn(g, B, W - 1, C, dtype=dtype))


def check_conv(case, sizes, got, state, silu=True, bias=True):
    H, P, G, N = sizes
    x, Bm, Cm, dt, fs = got
    u, lead = case["u"], case["u"].shape[:2]
    W = case["weight"].shape[1]
    want, size, last = conv64(u, case["weight"], case["bias"] if bias else None, state, silu)
    # W + 1 roundings, silu's slope of at most 1.1 and its own twenty-five units
    # (exponential of |v| < 12: 20 units), then the output
    tol = (W + 2) * U * size * 1.1 + want.abs() * (25 * U + HALF[u.dtype]) * 1.01
    out = torch.cat([x.reshape(*lead, -1), Bm.reshape(*lead, -1), Cm.reshape(*lead, -1)], -1)
    assert x.shape == (*lead, H, P) and Bm.shape == Cm.shape == (*lead, G, N)
    check("x|B|C", out, want, tol)
    if dt is not None:
        raw = case["dt"].double() + case["dt_bias"].double()
        step = torch.nn.functional.softplus(raw, threshold=1e9)
        # the sum's rounding moves softplus by at most |raw| U of itself below 0
        # and |raw| U above; exp, log1p and the sum of both: eight units
        check("dt", dt, step, (raw.abs() + 8) * U * 2 * step.clamp_min(raw.abs() * U) + 1e-37)
    if fs is not None:
        assert torch.equal(fs, last.to(fs.dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,L,H,P,G,N", [
    (1, 1, 1, 64, 1, 16), (2, 2, 2, 64, 1, 16), (1, 3, 4, 64, 2, 128), (3, 5, 3, 33, 1, 37), (2, 64, 2, 8, 2, 8),
    (1, 65, 5, 64, 5, 24), (2, 300, 4, 48, 2, 20), (1, 2051, 3, 64, 1, 128),
])
def test_conv(ssd, B, L, H, P, G, N, W, dtype):
    c = conv_case(B, L, H, P, G, N, W, dtype)
    got = ssd.conv(c["u"], c["weight"], c["bias"], H, P, G, N, dt=c["dt"], dt_bias=c["dt_bias"],
                   initial_state=c["state"])
    check_conv(c, (H, P, G, N), got, c["state"])


@pytest.mark.parametrize("pad", [0, 1, 5])
def test_conv_without_state_bias_activation_or_dt(ssd, pad):
    H, P, G, N = 3, 64, 1, 16
    c = conv_case(2, 37, H, P, G, N, 4, BF16, pad=pad)
    zero = torch.zeros_like(c["state"])
    got = ssd.conv(c["u"], c["weight"], None, H, P, G, N, activation="none", return_final_state=False)
    assert got[3] is None and got[4] is None
    check_conv(c, (H, P, G, N), got, zero, silu=False, bias=False)
    got = ssd.conv(c["u"], c["weight"], c["bias"], H, P, G, N, dt=c["dt"])
    check_conv(dict(c, dt_bias=torch.zeros_like(c["dt_bias"])), (H, P, G, N), got, zero)


def test_conv_in_pieces_and_token_by_token_is_the_same(ssd):
    """A prompt cut at any place, and token by token, gives the same bits."""
    H, P, G, N = 4, 64, 2, 24
    sizes = (H, P, G, N)
    c = conv_case(3, 41, H, P, G, N, 4, BF16)
    w = (c["weight"], c["bias"], *sizes)
    whole = ssd.conv(c["u"], *w, dt=c["dt"], dt_bias=c["dt_bias"], initial_state=c["state"])
    for cut in (1, 2, 3, 17, 40):
        a = ssd.conv(c["u"][:, :cut], *w, dt=c["dt"][:, :cut], dt_bias=c["dt_bias"], initial_state=c["state"])
        b = ssd.conv(c["u"][:, cut:], *w, dt=c["dt"][:, cut:], dt_bias=c["dt_bias"], initial_state=a[4])
        for i in range(4):
            assert torch.equal(torch.cat([a[i], b[i]], 1), whole[i]), (cut, i)
        assert torch.equal(b[4], whole[4])
    state = c["state"].clone()
    for t in range(41):
        got = ssd.conv_step(c["u"][:, t], c["weight"], c["bias"], state, *sizes, dt=c["dt"][:, t],
                            dt_bias=c["dt_bias"])
        for i in range(4):
            assert torch.equal(got[i], whole[i][:, t]), (t, i)
    assert torch.equal(state, whole[4])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,P,G,N,W", [(1, 1, 1, 1, 1, 2), (64, 80, 64, 1, 128, 4), (300, 2, 33, 1, 37, 3)])
def test_conv_step(ssd, B, H, P, G, N, W, dtype):
    c = conv_case(B, 1, H, P, G, N, W, dtype)
    state = c["state"].clone()
    got = ssd.conv_step(c["u"][:, 0], c["weight"], c["bias"], state, H, P, G, N, dt=c["dt"][:, 0],
                        dt_bias=c["dt_bias"])
    check_conv(c, (H, P, G, N), [t.unsqueeze(1) for t in got] + [state], c["state"])


def test_conv_of_extreme_values(ssd):
    """Inputs at which exp overflows or nothing is left, and no tokens at all."""
    H, P, G, N = 1, 8, 1, 8
    c = conv_case(1, 6, H, P, G, N, 2, F32)
    u = c["u"].clone()
    u[0, :, 0] = torch.tensor([1e30, -1e30, 100.0, -100.0, -1e4, 0.0])
    c["u"], c["weight"][0] = u, torch.tensor([0.0, 1.0])
    c["bias"][0] = 0
    raw = torch.tensor([-200.0, -80.0, -20.0, 20.0, 80.0, 1e4], device="cuda").reshape(1, 6, 1)
    got = ssd.conv(u, c["weight"], c["bias"], H, P, G, N, dt=raw, initial_state=c["state"])
    x = got[0][0, :, 0, 0].tolist()
    assert x[0] == pytest.approx(1e30) and x[1] == 0 and x[2] == 100 and abs(x[3]) < 1e-40 and x[5] == 0
    step = torch.nn.functional.softplus(raw.double(), threshold=1e9)
    check("dt", got[3], step, step * (raw.abs() + 8) * 2 * U + 2.0 ** -126)
    none = ssd.conv(u[:, :0], c["weight"], c["bias"], H, P, G, N, initial_state=c["state"])
    assert none[0].shape == (1, 0, H, P) and torch.equal(none[4], c["state"])
    none = ssd.conv(u[:, :0], c["weight"], c["bias"], H, P, G, N)
    assert (none[4] == 0).all()


# ------------------------------------------------------- streams and graphs

def layer_weights(g, H, P, G, N, W, d, dtype):
    d_inner, C = H * P, H * P + 2 * G * N
    row = d_inner + C + H
    return dict(norm=1 + 0.1 * randn(g, d), w_in=randn(g, row, d, dtype=dtype, scale=d ** -0.5),
                conv=randn(g, C, W, scale=0.5), conv_bias=0.1 * randn(g, C), dt_bias=randn(g, H) - 3,
                A=-torch.exp(randn(g, H)), D=randn(g, H), gate_norm=1 + 0.1 * randn(g, d_inner),
                w_out=randn(g, d, d_inner, dtype=dtype, scale=d_inner ** -0.5))


def split(row, H, P, G, N):
    C = H * P + 2 * G * N
    return row[..., :H * P], row[..., H * P:H * P + C], row[..., H * P + C:]


def project(ssd, x, w, quantize, out_dtype, residual=None):
    """x is rms_norm's (y, scale, ...); w a matrix or its (values, scales)."""
    if quantize:
        return ssd.linear(x[0], w[0], x_scale=x[1], w_scale=w[1], residual=residual, out_dtype=out_dtype)
    return ssd.linear(x[0], w, residual=residual, out_dtype=out_dtype)


def layer_prefill(ssd, p, h, sizes, quantize, conv_state=None, ssm_state=None):
    """One Mamba-2 layer on the residual stream h [B, L, d] fp32; every operator's output."""
    H, P, G, N = sizes
    dtype = torch.bfloat16 if quantize else p["w_in"].dtype
    n = ssd.rms_norm(h.to(dtype), p["norm"], quantize=quantize)
    row = project(ssd, n, p["w_in"], quantize, dtype)
    z, u, dt_raw = split(row, *sizes)
    x, Bm, Cm, dt, cs = ssd.conv(u, p["conv"], p["conv_bias"], *sizes, dt=dt_raw, dt_bias=p["dt_bias"],
                                 initial_state=conv_state)
    y, fs = ssd.forward(x, dt, p["A"], Bm, Cm, p["D"], chunk=64, initial_state=ssm_state)
    g = ssd.rms_norm(y.flatten(-2), p["gate_norm"], gate=z, quantize=quantize)
    out = project(ssd, g, p["w_out"], quantize, F32, residual=h)
    return dict(n=n, row=row, conv=(x, Bm, Cm, dt, cs), y=y, fs=fs, g=g, out=out)


def layer_step(ssd, p, h, sizes, quantize, conv_state, ssm_state):
    dtype = torch.bfloat16 if quantize else p["w_in"].dtype
    n = ssd.rms_norm(h.to(dtype), p["norm"], quantize=quantize)
    row = project(ssd, n, p["w_in"], quantize, dtype)
    z, u, dt_raw = split(row, *sizes)
    x, Bm, Cm, dt = ssd.conv_step(u, p["conv"], p["conv_bias"], conv_state, *sizes, dt=dt_raw,
                                  dt_bias=p["dt_bias"])
    y = ssd.step(x, dt, p["A"], Bm, Cm, p["D"], ssm_state)
    g = ssd.rms_norm(y.flatten(-2), p["gate_norm"], gate=z, quantize=quantize)
    return project(ssd, g, p["w_out"], quantize, F32, residual=h)


def layer64(p, h, sizes):
    """The layer in 64 bits, token by token, from the formulas."""
    H, P, G, N = sizes
    d = {k: v.double() for k, v in p.items()}
    _, n = norm64(h, d["norm"], None, None, 1e-5, 1)
    z, u, dt_raw = split(n @ d["w_in"].t(), *sizes)
    B, L, C = u.shape
    W = d["conv"].shape[1]
    v, _, _ = conv64(u, d["conv"], d["conv_bias"], torch.zeros(B, W - 1, C, device=h.device), True)
    x = v[..., :H * P].reshape(B, L, H, P)
    Bm, Cm = (t.reshape(B, L, G, N).repeat_interleave(H // G, 2) for t in v[..., H * P:].split(G * N, -1))
    dt = torch.nn.functional.softplus(dt_raw + d["dt_bias"])
    s = torch.zeros(B, H, P, N, dtype=torch.double, device=h.device)
    ys = []
    for t in range(L):
        a = torch.exp(dt[:, t] * d["A"])
        s = a[..., None, None] * s + dt[:, t, :, None, None] * x[:, t, :, :, None] * Bm[:, t, :, None, :]
        ys.append((s * Cm[:, t, :, None, :]).sum(-1) + d["D"][:, None] * x[:, t])
    _, g = norm64(torch.stack(ys, 1).flatten(-2), d["gate_norm"], None, z, 1e-5, 1)
    return g @ d["w_out"].t() + h.double(), s


def test_layer_fp32_against_64_bits(ssd):
    """The whole layer in fp32, prefill and then token by token, against 64
    bits. Its longest sums have d_inner + d + N = 400 terms and every operator's
    output is of order one: 400 U x 6 operators = 1.4e-4 of the largest output."""
    sizes, d = (4, 48, 2, 24), 128
    g = gen(11)
    p = layer_weights(g, *sizes, 4, d, F32)
    h = randn(g, 2, 50, d)
    want, state = layer64(p, h, sizes)
    whole = layer_prefill(ssd, p, h, sizes, False)
    tol = 1.5e-4 * want.abs().max()
    check("prefill", whole["out"], want, tol)
    check("state", whole["fs"], state, 1.5e-4 * state.abs().max())
    first = layer_prefill(ssd, p, h[:, :30].contiguous(), sizes, False)
    cs, ss = first["conv"][4], first["fs"]
    for t in range(30, 50):
        out = layer_step(ssd, p, h[:, t].contiguous(), sizes, False, cs, ss)
        check(f"step {t}", out, want[:, t], tol)
    check("state", ss, state, 1.5e-4 * state.abs().max())


@pytest.mark.parametrize("quantize", [False, True])
def test_layer_operators_in_a_row(ssd, quantize):
    """bf16 and 8-bit layer on the tensor-core sizes: every operator's output
    against 64 bits on the very inputs it was given."""
    sizes, d = (8, 64, 1, 128), 256
    H, P, G, N = sizes
    g = gen(12)
    p = layer_weights(g, *sizes, 4, d, BF16)
    w = {k: p[k] for k in ("w_in", "w_out")}
    if quantize:
        for k in w:
            p[k] = quantize_rows(w[k].float())
    h = randn(g, 2, 200, d)
    r = layer_prefill(ssd, p, h, sizes, quantize)

    def check_norm_out(got, want, D):
        y, s, _ = got
        rel = norm_rel(D, 1) + 8 * U
        if quantize:
            check("norm", y.double() * s.double()[..., None], want,
                  want.abs() * (rel + HALF[E4M3]) + s.double()[..., None] * E4M3_SUBNORMAL_HALF * 1.001)
        else:
            check("norm", y, want, want.abs() * (rel + HALF[BF16]))

    def check_product(x, k, got, out, residual=None):
        a, b = (x[0].double(), p[k][0].double()) if quantize else (x[0].double(), p[k].double())
        if quantize:
            a, b = a * x[1].double()[..., None], b * p[k][1].double()[:, None]
        want = a @ b.t()
        size = a.abs() @ b.abs().t()
        tol = size * (2 * a.shape[-1] + 8) * U + want.abs() * HALF[out] * 1.01
        if residual is not None:
            want = want + residual.double()
            tol = tol + want.abs() * HALF[out] * 1.01
        check(k, got, want, tol)

    check_norm_out(r["n"], norm64(h.bfloat16(), p["norm"], None, None, 1e-5, 1)[1], d)
    check_product(r["n"], "w_in", r["row"], BF16)
    z, u, dt_raw = split(r["row"], *sizes)
    zero = torch.zeros(2, 3, u.shape[-1], device="cuda", dtype=BF16)
    check_conv(dict(u=u, dt=dt_raw, weight=p["conv"], bias=p["conv_bias"], dt_bias=p["dt_bias"]), sizes,
               r["conv"], zero)
    check_norm_out(r["g"], norm64(r["y"].flatten(-2), p["gate_norm"], None, z, 1e-5, 1)[1], H * P)
    check_product(r["g"], "w_out", r["out"], F32, residual=h)


def test_layer_step_captured_and_replayed(ssd):
    """A decode step captured into a graph and replayed on new inputs gives the
    bits of the eager step, twice, also with another graph of the same step."""
    sizes, d = (8, 64, 1, 128), 256
    g = gen(13)
    p = layer_weights(g, *sizes, 4, d, BF16)
    for k in ("w_in", "w_out"):
        p[k] = quantize_rows(p[k].float())
    B, C = 5, 8 * 64 + 256
    hs = [randn(g, B, d) for _ in range(4)]
    cs0, ss0 = randn(g, B, 3, C, dtype=BF16), randn(g, B, 8, 64, 128)
    cs, ss = cs0.clone(), ss0.clone()
    want = [layer_step(ssd, p, h, sizes, True, cs, ss) for h in hs]
    want_state = (cs.clone(), ss.clone())
    graphs = []
    h_in, cs, ss = torch.empty(B, d, device="cuda"), cs0.clone(), ss0.clone()
    h_in.copy_(hs[0])
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer_step(ssd, p, h_in, sizes, True, cs, ss)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer_step(ssd, p, h_in, sizes, True, cs, ss)
        graphs.append((graph, out))
    cs.copy_(cs0)
    ss.copy_(ss0)
    for i, h in enumerate(hs):
        h_in.copy_(h)
        graph, out = graphs[i % 2]
        graph.replay()
        assert torch.equal(out, want[i]), i
    assert torch.equal(cs, want_state[0]) and torch.equal(ss, want_state[1])


def test_calls_on_two_streams_at_once(ssd):
    """The same operators on two streams, given as an argument or as the current
    one, interleaved and repeated: the bits of a single call."""
    g = gen(14)
    x, w = randn(g, 300, 512, dtype=BF16), randn(g, 640, 512, dtype=BF16, scale=0.05)
    x1, r = x[:9].contiguous(), randn(g, 300, 640, dtype=BF16)
    wn = 1 + 0.1 * randn(g, 512)
    want = (ssd.linear(x, w, residual=r), ssd.linear(x1, w), ssd.rms_norm(x, wn, quantize=True)[0])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((ssd.linear(x, w, residual=r, stream=a), ssd.linear(x1, w, stream=b),
                    ssd.rms_norm(x, wn, quantize=True, stream=a)[0]))
        with torch.cuda.stream(b):
            got.append((ssd.linear(x, w, residual=r), ssd.linear(x1, w, stream=a),
                        ssd.rms_norm(x, wn, quantize=True)[0]))
    torch.cuda.synchronize()
    for one in got:
        for i in range(3):
            assert torch.equal(one[i].view(torch.uint8), want[i].view(torch.uint8)), i


def test_repeated_calls_give_the_same_bits(ssd):
    g = gen(15)
    for M, N, K in ((1, 1024, 2048), (64, 2576, 2560), (700, 640, 1040), (2048, 2560, 512)):
        x, w = randn(g, M, K, dtype=BF16), randn(g, N, K, dtype=BF16)
        want = ssd.linear(x, w, out_dtype=F32)
        for _ in range(30):
            assert torch.equal(ssd.linear(x, w, out_dtype=F32), want), (M, N, K)


def test_refusals_on_the_device(ssd):
    x, w = torch.zeros(4, 64, device="cuda", dtype=BF16), torch.zeros(8, 64, device="cuda", dtype=BF16)
    f = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="columns"):
        ssd.linear(x, w[:, :32].contiguous())
    with pytest.raises(TypeError, match="w must be torch.bfloat16"):
        ssd.linear(x, w.float())
    with pytest.raises(ValueError, match="w must be contiguous"):
        ssd.linear(x, torch.zeros(64, 8, device="cuda", dtype=BF16).t())
    with pytest.raises(ValueError, match="contiguous"):
        ssd.linear(torch.zeros(64, 4, device="cuda", dtype=BF16).t(), w)
    with pytest.raises(ValueError, match="activation"):
        ssd.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="x_scale"):
        ssd.linear(x, w, x_scale=f[:4])
    with pytest.raises(ValueError, match="x_scale"):
        ssd.linear(x.to(E4M3), w.to(E4M3), x_scale=f[:4].contiguous())
    with pytest.raises(TypeError, match="residual must be"):
        ssd.linear(x, w, residual=torch.zeros(4, 8, device="cuda"), out_dtype=BF16)
    with pytest.raises(TypeError, match="float32, bfloat16 or float8"):
        ssd.linear(x.half(), w.half())
    with pytest.raises(ValueError, match="y must have shape"):
        ssd.linear(x, w, y=torch.zeros(4, 9, device="cuda", dtype=BF16))
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.linear(x, torch.zeros(64, 64, device="cuda", dtype=BF16), y=x)
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.linear(x[:1].expand(4, 64), w)  # rows on top of one another
    with pytest.raises(ValueError, match="cannot be combined"):
        ssd.rms_norm(x, f, residual=x, gate=x)
    with pytest.raises(ValueError, match="residual_out needs"):
        ssd.rms_norm(x, f, residual_out=x)
    with pytest.raises(ValueError, match="scale needs"):
        ssd.rms_norm(x, f, scale=f)
    with pytest.raises(TypeError, match="residual must be"):
        ssd.rms_norm(x, f, residual=x.half())
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.rms_norm(x, f, groups=3)
    with pytest.raises(ValueError, match="weight must have shape"):
        ssd.rms_norm(x, f[:32].contiguous())
    u = torch.zeros(1, 4, 160, device="cuda", dtype=BF16)
    cw, st = torch.zeros(160, 4, device="cuda"), torch.zeros(1, 3, 160, device="cuda", dtype=BF16)
    with pytest.raises(ssd.SSDError, match="INVALID_ARG"):
        ssd.conv(u, cw, None, 2, 64, 1, 16, initial_state=st, final_state=st)
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.conv(u, torch.zeros(160, 5, device="cuda"), None, 2, 64, 1, 16)
    with pytest.raises(ValueError, match="u must be"):
        ssd.conv(u, cw, None, 2, 64, 1, 8)
    with pytest.raises(ValueError, match="dt_bias needs dt"):
        ssd.conv(u, cw, None, 2, 64, 1, 16, dt_bias=f[:2].contiguous())
    with pytest.raises(ValueError, match="state is required"):
        ssd.conv_step(u[:, 0], cw, None, None, 2, 64, 1, 16)


def test_offsets_beyond_32_bits(ssd):
    """The last rows of operands and outputs of more than 2^31 elements."""
    g = gen(16)
    M, D = 4_200_000, 512
    x, w = randn(g, M, D, dtype=BF16), 1 + 0.1 * randn(g, D)
    last = slice(M - 100, M)
    y, s, _ = ssd.rms_norm(x, w, quantize=True)
    _, want = norm64(x[last], w, None, None, 1e-5, 1)
    check("norm", y[last].double() * s[last].double()[:, None], want,
          want.abs() * (norm_rel(D, 1) + 8 * U + HALF[E4M3]) + s[last].double()[:, None] * E4M3_SUBNORMAL_HALF * 1.001)
    del x, y
    M, K = 2_000_000, 1088
    x = randn(g, M, K, dtype=BF16)
    for N in (1088, 1089):
        w = randn(g, N, K, dtype=BF16, scale=0.03)
        y = ssd.linear(x, w)
        last = slice(M - 100, M)
        want = x[last].double() @ w.double().t()
        size = x[last].double().abs() @ w.double().abs().t()
        check("linear", y[last], want, size * (2 * K + 8) * U + want.abs() * HALF[BF16] * 1.01)
        del y
    del x
    L, sizes = 1_000_000, (32, 64, 1, 128)
    C = 32 * 64 + 256
    u, w = randn(g, 1, L, C, dtype=BF16), randn(g, C, 4, scale=0.5)
    got = ssd.conv(u, w, None, *sizes)
    tail = u[:, L - 40:]
    c = dict(u=tail, weight=w)
    check_conv(c, sizes, [t[:, L - 40:] for t in got[:3]] + [None, got[4]], u[:, L - 43:L - 40], bias=False)
