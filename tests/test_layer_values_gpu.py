"""The operators around the SSD core at the values and widths that
test_layer_gpu.py does not reach: rows of tiny values in 8 bits, groups of three
vectors to a lane, and the precision of what is done in fp32 (the activations, the
three bf16 parts of an fp32 operand, the segments of a long sum), each against the
formula in 64 bits.

Tolerances count roundings as in test_layer_gpu.py: U = 2^-24 of the result for one in
fp32, 2^-149 absolute below its normal range.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from test_layer_gpu import (BF16, E4M3, E4M3_SUBNORMAL_HALF, F32, HALF, U, check, check_norm, gen, norm64,  # noqa: E402
                            norm_rel, quantize_rows, randn)

pytestmark = pytest.mark.gpu

DENORMAL = 2.0 ** -149


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import selective_state_space_17_b200 as _ssd
    return _ssd


# ---------------------------------------------------------------- rms_norm

@pytest.mark.parametrize("mode", ["plain", "residual", "gate"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,groups,eps", [(64, 1, 1e-5), (97, 1, 1e-5), (4096, 1, 1e-5), (4096, 4, 1e-5), (40000, 1, 1e-5),
                                          (512, 1, 1e-12), (512, 4, 1e-12)])
def test_norm_of_tiny_rows_in_8_bits(ssd, D, groups, eps, dtype, mode):
    """Rows from below the smallest scale's to above 448 / FLT_MAX, zeros among them,
    in registers and read twice: what is stored times the scale is the formula's."""
    g = gen(D + groups)
    tops = torch.tensor([1e-39, 1e-38, 2e-38, 1e-37, 5e-37, 1e-36, 1.3e-36, 1.5e-36, 3e-36, 1e-35, 1e-30],
                        device="cuda")
    v = randn(g, len(tops), D)
    v = v / v.abs().amax(-1, keepdim=True) * tops[:, None]
    v[:, 3::7] = 0
    kw = {}
    if mode == "residual":
        kw["residual"] = torch.zeros_like(v)
    if mode == "gate":
        kw["gate"] = torch.full((len(tops), D), 3.0, device="cuda", dtype=dtype)
    x, weight = v.to(dtype), torch.ones(D, device="cuda")
    q, s, _ = ssd.rms_norm(x, weight, eps=eps, groups=groups, quantize=True, **kw)
    _, want = norm64(x, weight, kw.get("residual"), kw.get("gate"), eps, groups)
    rel, rho = norm_rel(D, groups), eps ** -0.5
    # v and v w may lie below fp32's normal range, each within half a step of it, and rho
    # carries that to y; the scale is at least 2^-126, the end of that range
    absolute = rho * DENORMAL
    scale = (want.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    check("scale", s, scale, scale * (rel + 2 * U) + absolute / 448)
    check("y", q.double() * s.double()[:, None], want,
          want.abs() * (rel + 8 * U + HALF[E4M3]) * (1 + 2.0 ** -20) + absolute
          + s.double()[:, None] * E4M3_SUBNORMAL_HALF * 1.001)


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("mode", ["plain", "residual", "gate"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,D,groups", [(600, 10240, 16), (601, 8320, 16), (700, 12288, 16), (593, 12160, 16),
                                           (600, 5120, 16), (600, 9600, 15), (600, 15360, 32)])
def test_norm_many_rows_in_many_groups(ssd, rows, D, groups, dtype, mode, quantize):
    """More than four rows to an SM, groups of 65 to 96 vectors of 16 bytes: the forms of
    two and three vectors to a lane at their most warps."""
    g = gen(rows + D)
    kw = {}
    if mode == "residual":
        kw["residual"] = randn(g, rows, D, scale=2.0)
    if mode == "gate":
        kw["gate"] = randn(g, rows, D, dtype=dtype)
    check_norm(ssd, randn(g, rows, D, dtype=dtype), 1 + 0.1 * randn(g, D), groups=groups, quantize=quantize, **kw)


# -------------------------------------------------------------- activations

def activated(ssd, v, act, out, M, variant=0):
    """act(v) for v [N] by way of a product of zeros and the bias, on M equal rows."""
    x = torch.zeros(M, 64, device="cuda", dtype=BF16)
    w = torch.zeros(v.numel(), 64, device="cuda", dtype=BF16)
    ssd.layer.set_linear_variant(variant)
    try:
        return ssd.linear(x, w, bias=v, activation=act, out_dtype=out)
    finally:
        ssd.layer.set_linear_variant(0)


def gelu64(v):
    return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))


def silu64(v):
    return v / (1 + torch.exp(-v))


# SiLU in fp32: e^-|v| (two units of 2^-23) times v, one plus it and the reciprocal (1 + 2),
# the product: 10 U
SILU_F32 = 10 * U


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,variant", [(3, 1), (3, 2), (300, 2), (300, 3)])
def test_linear_gelu_keeps_its_relative_precision(ssd, M, variant, out):
    """The tail of v < 0, where the result is far below v: relative to the result. The
    polynomial 4 U, its argument 2 U at a slope of 2.7, the power of two 5 U, products and
    sums 6 U: 24 U in all. bf16 leaves out what fp32 makes up for: the exponent v^2 / 2 has
    its square's, its factor's and their product's roundings, 1.25 v^2 U. erfc(-v) may lie
    below fp32's normal range, each of two roundings within half a step."""
    v = torch.cat([torch.linspace(-13, 10, 4093, device="cuda"), torch.tensor([0.0, 30.0, 1e30], device="cuda")])
    got = activated(ssd, v, "gelu", out, M, variant)
    want = gelu64(v.double())
    rel = 24 * U + (1.25 * U * v.double().clamp(-20, 20) ** 2 + HALF[BF16] * 1.01 if out is BF16 else 0)
    tol = want.abs() * rel + v.double().abs() * DENORMAL * (v < 0) + DENORMAL
    check("gelu", got, want.expand(M, -1), tol.expand(M, -1))


@pytest.mark.parametrize("M,variant", [(3, 1), (3, 2), (300, 2), (300, 3)])
def test_linear_silu_keeps_its_relative_precision_in_fp32(ssd, M, variant):
    """Down to where e^v leaves fp32's normal range, in which its two units are absolute."""
    v = torch.cat([torch.linspace(-95, 30, 4093, device="cuda"), torch.tensor([0.0, 100.0, 1e30], device="cuda")])
    got = activated(ssd, v, "silu", F32, M, variant)
    want = silu64(v.double())
    check("silu", got, want.expand(M, -1), (want.abs() * SILU_F32 + v.double().abs() * 4 * DENORMAL * (v < 0)).expand(M, -1))


@pytest.mark.parametrize("width,H,P", [(4, 16, 64), (3, 15, 33), (2, 16, 64)])
def test_conv_silu_keeps_its_relative_precision_in_fp32(ssd, width, H, P):
    """Inputs of zero and the bias: act(v) of given values, in prompts and single tokens."""
    G, N = 1, 20
    C = H * P + 2 * G * N
    v = torch.linspace(-95, 30, C, device="cuda")
    u, w = torch.zeros(2, 11, C, device="cuda"), torch.ones(C, width, device="cuda")
    want = silu64(v.double())
    tol = want.abs() * SILU_F32 + v.double().abs() * 4 * DENORMAL * (v < 0)
    x, Bm, Cm, _, _ = ssd.conv(u, w, v, H, P, G, N)
    got = torch.cat([t.reshape(2, 11, -1) for t in (x, Bm, Cm)], -1)
    check("conv", got, want.expand(2, 11, -1), tol.expand(2, 11, -1))
    x, Bm, Cm, _ = ssd.conv_step(u[:, 0], w, v, torch.zeros(2, width - 1, C, device="cuda"), H, P, G, N)
    got = torch.cat([t.reshape(2, -1) for t in (x, Bm, Cm)], -1)
    check("conv_step", got, want.expand(2, -1), tol.expand(2, -1))


@pytest.mark.parametrize("D", [64, 97, 2560, 20001])
def test_norm_gate_keeps_its_relative_precision_in_fp32(ssd, D):
    """Gates far below zero, whose squares are nothing beside eps = 1: y = silu(z) but for
    the root's four units and three products'."""
    z = torch.linspace(-80, -20, 5 * D, device="cuda").reshape(5, D)
    one = torch.ones(5, D, device="cuda")
    y, _, _ = ssd.rms_norm(one, one[0].clone(), gate=z, eps=1.0)
    want = silu64(z.double())
    check("y", y, want, want.abs() * (SILU_F32 + 8 * U))


# ------------------------------------------------------- products in fp32

@pytest.mark.parametrize("variant", [0, 1, 2, 3])
@pytest.mark.parametrize("M,K", [(3, 1), (3, 96), (40, 8), (40, 96), (300, 1), (300, 130)])
def test_linear_fp32_products_keep_24_bits(ssd, M, K, variant):
    """One factor to a row: y is a single product of two full significands. As three bf16
    parts, x = x1 + x2 + x3, the products left out are at most 2^-24 of it together; its
    sum is truncated once at its full size (2 U), and at most seven joins round (7 U)."""
    g = gen(M + K)
    x = torch.zeros(M, K, device="cuda")
    m = torch.arange(M, device="cuda")
    x[m, m % K] = (1 + torch.rand(M, generator=g, device="cuda")) * (1 - 2.0 * (m % 2))
    w = 1 + torch.rand(72, K, generator=g, device="cuda")
    ssd.layer.set_linear_variant(variant)
    try:
        got = ssd.linear(x, w)
    finally:
        ssd.layer.set_linear_variant(0)
    want = x.double() @ w.double().t()
    check("y", got, want, want.abs() * 11 * U)


@pytest.mark.parametrize("M", [3, 70, 1100])
@pytest.mark.parametrize("sx,sw", [(2.0 ** -124, 2.0 ** 110), (2.0 ** -112, 1.0), (2.0 ** 110, 2.0 ** -124),
                                   (2.0 ** -140, 2.0 ** 120), (2.0 ** -105, 2.0 ** 90)])
def test_linear_fp32_of_tiny_operands(ssd, M, sx, sw):
    """Values whose third or second bf16 part would lie below bf16's range keep their 24
    bits all the same; one such value among ordinary ones likewise."""
    g = gen(M)
    K = 96
    x, w = randn(g, M, K) * sx, randn(g, 72, K) * sw
    size = x.double().abs() @ w.double().abs().t()
    check("y", ssd.linear(x, w), x.double() @ w.double().t(), size * (2 * K + 28) * U + K * DENORMAL)
    x, w = randn(g, M, K), randn(g, 72, K)
    x[M - 1] = 0
    x[M - 1, 5] = sx * 1.2345678
    w[:, 5] *= sw
    size = x.double().abs() @ w.double().abs().t()
    check("y", ssd.linear(x, w), x.double() @ w.double().t(), size * (2 * K + 28) * U + K * DENORMAL)


@pytest.mark.parametrize("variant,M,N", [(2, 64, 20480), (3, 512, 2560)])
def test_linear_long_sums_are_not_biased(ssd, variant, M, N):
    """The tensor cores truncate as they add: a sum of 5120 positive products in one
    accumulator comes out 1.8e-5 too small on average. Joined every 768 products, 48
    additions of 16, it loses half a step of at most 2^-23 an addition of a sum that grows
    evenly: 24 x 2^-24 = 1.43e-6."""
    g = gen(variant)
    K = 5120
    x = torch.rand(M, K, generator=g, device="cuda").to(BF16)
    w = torch.rand(N, K, generator=g, device="cuda").to(BF16)
    ssd.layer.set_linear_variant(variant)
    try:
        got = ssd.linear(x, w, out_dtype=F32)
    finally:
        ssd.layer.set_linear_variant(0)
    want = x.double() @ w.double().t()
    mean = ((got.double() - want) / want).mean().item()
    assert abs(mean) < 24 * U, mean


# ---------------------------------------------- kernels one after another

def test_row_scales_of_the_kernel_before(ssd):
    """A norm writes the scales that the product behind it reads, which starts while the
    norm still runs: replays on changing rows give the bits of calls made one at a time."""
    g = gen(4)
    for M, D, N in ((1, 2048, 1024), (64, 2560, 1040), (700, 512, 2560)):
        xs = [randn(g, M, D, dtype=BF16, scale=10.0 ** i) for i in range(-3, 4)]
        weight = 1 + 0.1 * randn(g, D)
        w, ws = quantize_rows(randn(g, N, D))
        x, q, s = xs[0].clone(), torch.empty(M, D, device="cuda", dtype=E4M3), torch.empty(M, device="cuda")
        y = torch.empty(M, N, device="cuda")
        want = []
        for v in xs:
            x.copy_(v)
            ssd.rms_norm(x, weight, eps=1.0, quantize=True, y=q, scale=s)
            torch.cuda.synchronize()
            want.append(ssd.linear(q, w, x_scale=s, w_scale=ws, out_dtype=F32))
            torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):  # the product before still reads what the norm writes again
                ssd.rms_norm(x, weight, eps=1.0, quantize=True, y=q, scale=s)
                ssd.linear(q, w, x_scale=s, w_scale=ws, y=y)
        for _ in range(5):
            for v, expect in zip(xs, want):
                x.copy_(v)
                graph.replay()
                assert torch.equal(y, expect), (M, D, N)
