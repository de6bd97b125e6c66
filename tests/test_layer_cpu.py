"""Refusals of the operators around the SSD core (rms_norm, linear, conv,
conv_step), in the C ABI and in the Python binding. No GPU: every call fails its
checks before the first CUDA call, or has nothing to do."""
import pytest

torch = pytest.importorskip("torch")

F32, BF16, E4M3 = 0, 1, 2
NONE, SILU, GELU = 0, 1, 2
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 6


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_17_b200 import build
    build.build()
    from selective_state_space_17_b200 import layer
    return layer.lib


def P(i):
    """Aligned addresses 256 MiB apart, never dereferenced."""
    return 0x10000000 * (i + 1)


def norm(lib, **kw):
    a = dict(x=P(0), residual=None, gate=None, gate_stride=0, weight=P(1), y=P(2), scale=None,
             residual_out=None, rows=4, D=64, groups=1, eps=1e-5, dtype=BF16, rdtype=BF16, ydtype=BF16)
    a.update(kw)
    return lib.ssd_rms_norm(a["x"], a["residual"], a["gate"], a["gate_stride"], a["weight"], a["y"],
                            a["scale"], a["residual_out"], a["rows"], a["D"], a["groups"], a["eps"],
                            a["dtype"], a["rdtype"], a["ydtype"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(dtype=E4M3), INVALID), (dict(dtype=9), INVALID), (dict(ydtype=F32), INVALID),
    (dict(residual=P(3), rdtype=E4M3), INVALID), (dict(dtype=F32, ydtype=F32, residual=P(3)), INVALID),
    (dict(D=66, groups=33), UNSUPPORTED), (dict(D=(1 << 20) + 1), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(residual=P(3), gate=P(4), gate_stride=64), INVALID), (dict(residual_out=P(3)), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
    (dict(ydtype=E4M3), INVALID), (dict(scale=P(3)), INVALID),
    (dict(gate=P(3), gate_stride=63), INVALID),
    (dict(x=P(0) + 8), MISALIGNED), (dict(weight=P(1) + 4), MISALIGNED), (dict(y=P(2) + 2), MISALIGNED),
    (dict(residual=P(3) + 2), MISALIGNED), (dict(ydtype=E4M3, scale=P(3) + 4), MISALIGNED),
    (dict(gate=P(3) + 1, gate_stride=64), MISALIGNED),
    # outputs over inputs: y over part of x, 8-bit y over x, residual_out over half of the residual
    (dict(y=P(0) + 16), INVALID), (dict(y=P(0), ydtype=E4M3, scale=P(3)), INVALID),
    (dict(residual=P(3), residual_out=P(3) + 64), INVALID), (dict(residual=P(3), residual_out=P(2)), INVALID),
    (dict(y=P(1)), INVALID), (dict(gate=P(2) + 2, gate_stride=64), INVALID),
    (dict(rows=0, x=None, weight=None, y=None), OK),
])
def test_norm_refusals(lib, kw, want):
    assert norm(lib, **kw) == want


def linear(lib, **kw):
    a = dict(x=P(0), x_stride=32, w=P(1), xs=None, ws=None, bias=None, residual=None, y=P(2), M=4, N=48,
             K=32, act=NONE, dtype=BF16, ydtype=BF16, ws_ptr=None, ws_bytes=0)
    a.update(kw)
    return lib.ssd_linear(a["x"], a["x_stride"], a["w"], a["xs"], a["ws"], a["bias"], a["residual"],
                          a["y"], a["M"], a["N"], a["K"], a["act"], a["dtype"], a["ydtype"], a["ws_ptr"],
                          a["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(act=3), INVALID),
    (dict(dtype=3), INVALID), (dict(ydtype=E4M3), INVALID), (dict(ydtype=7), INVALID),
    (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 1, x_stride=1 << 21), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(xs=P(3)), INVALID), (dict(dtype=E4M3, xs=P(3)), INVALID), (dict(dtype=E4M3, ws=P(3)), INVALID),
    (dict(x_stride=31), INVALID), (dict(x=P(0) + 1), MISALIGNED), (dict(w=P(1) + 8), MISALIGNED),
    (dict(y=P(2) + 8), MISALIGNED), (dict(bias=P(3) + 4), MISALIGNED), (dict(residual=P(3) + 8), MISALIGNED),
    (dict(y=P(0)), INVALID), (dict(y=P(1) + 32), INVALID), (dict(residual=P(2) + 16), INVALID),
    (dict(bias=P(2)), INVALID), (dict(ws_ptr=P(3) + 8), MISALIGNED),
    # fp32 with more than a few tokens, and rows off 16 bytes, are copied first
    (dict(M=64, dtype=F32, ydtype=F32), WORKSPACE), (dict(M=64, K=31, x_stride=32), WORKSPACE),
    (dict(M=64, K=31, x_stride=31, ws_ptr=P(3), ws_bytes=1000), WORKSPACE),
    (dict(M=64, dtype=F32, ydtype=F32, ws_ptr=P(2) + 256, ws_bytes=1 << 27), INVALID),  # over y
    (dict(M=64, dtype=F32, ydtype=F32, ws_ptr=P(1), ws_bytes=1 << 27), INVALID),  # over w
    (dict(M=0, x=None, w=None, y=None), OK), (dict(N=0, x=None, w=None, y=None), OK),
])
def test_linear_refusals(lib, kw, want):
    assert linear(lib, **kw) == want


def test_linear_workspace_size(lib):
    """256 bytes of flag, then copies of what TMA cannot address: rows of whole
    128-byte blocks, three of them for an fp32 row."""
    size = lib.ssd_linear_workspace_size
    assert size(P(0), 2560, 64, 10576, 2560, BF16) == 0
    assert size(P(0), 2576, 64, 48, 2560, E4M3) == 0
    assert size(P(0), 2561, 8, 48, 2561, BF16) == 0  # few tokens: read as they lie
    assert size(P(0), 2560, 8, 48, 2560, F32) == 0
    row = 41 * 128  # 2561 bf16 elements are 5122 bytes
    assert size(P(0), 2561, 64, 48, 2561, BF16) == 256 + (64 + 48) * row
    assert size(P(0), 2561, 64, 48, 2560, BF16) == 256 + 64 * 40 * 128  # x's rows alone
    assert size(P(0) + 2, 2560, 64, 48, 2560, BF16) == 256 + 64 * 40 * 128
    assert size(P(0), 65, 64, 48, 65, F32) == 256 + (64 + 48) * 3 * 2 * 128
    assert size(P(0), 64, 0, 48, 64, F32) == 0 and size(P(0), 64, 64, 48, 0, F32) == 0


def conv(lib, **kw):
    a = dict(u=P(0), ub=1280, ur=160, weight=P(1), bias=P(2), dt_raw=P(3), db=16, dr=2, dt_bias=P(4),
             init=P(5), x=P(6), Bm=P(7), Cm=P(8), dt=P(9), fs=P(10), B=2, L=8, H=2, P=64, G=1, N=16,
             width=4, act=SILU, dtype=BF16)
    a.update(kw)
    return lib.ssd_conv(a["u"], a["ub"], a["ur"], a["weight"], a["bias"], a["dt_raw"], a["db"], a["dr"],
                        a["dt_bias"], a["init"], a["x"], a["Bm"], a["Cm"], a["dt"], a["fs"], a["B"],
                        a["L"], a["H"], a["P"], a["G"], a["N"], a["width"], a["act"], a["dtype"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(H=3, G=2), INVALID), (dict(B=-1), INVALID), (dict(P=300), UNSUPPORTED), (dict(dtype=E4M3), INVALID),
    (dict(width=0), INVALID), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(B=1, L=(1 << 30) + 1), UNSUPPORTED), (dict(act=GELU), INVALID), (dict(ur=-1), INVALID), (dict(ub=-1), INVALID),
    (dict(dr=-1), INVALID), (dict(db=-1), INVALID),
    *[(dict([(k, None)]), INVALID) for k in ("u", "weight", "x", "Bm", "Cm", "dt", "dt_raw")],
    *[(dict([(k, P(11) + 4)]), MISALIGNED)
      for k in ("weight", "bias", "dt_bias", "init", "x", "Bm", "Cm", "dt", "fs")],
    (dict(u=P(0) + 1), MISALIGNED), (dict(dt_raw=P(3) + 1), MISALIGNED),
    (dict(fs=P(5)), INVALID), (dict(fs=P(5) + 16), INVALID), (dict(x=P(0) + 160), INVALID),
    (dict(Bm=P(7), Cm=P(7)), INVALID), (dict(dt=P(6)), INVALID),
])
def test_conv_refusals(lib, kw, want):
    assert conv(lib, **kw) == want


def test_conv_without_tokens_needs_no_operands(lib):
    none = dict(u=None, weight=None, bias=None, dt_raw=None, dt_bias=None, init=None, x=None, Bm=None,
                Cm=None, dt=None, fs=None)
    assert conv(lib, L=0, **none) == OK
    assert conv(lib, B=0, **none) == OK


def test_conv_step_refusals(lib):
    def call(u=P(0), weight=P(1), state=P(2), x=P(3), Bm=P(4), Cm=P(5), dt_raw=None, dt=None, B=2, width=4):
        return lib.ssd_conv_step(u, 160, weight, None, dt_raw, 2, None, state, x, Bm, Cm, dt, B, 2, 64, 1,
                                 16, width, SILU, BF16, None)
    for k in ("u", "weight", "state", "x", "Bm", "Cm"):
        assert call(**{k: None}) == INVALID, k
    assert call(dt=P(6)) == INVALID and call(dt_raw=P(6)) == INVALID
    assert call(state=P(2) + 8) == MISALIGNED
    assert call(state=P(0)) == INVALID  # the state over the inputs
    assert call(width=7) == UNSUPPORTED
    assert call(B=0, u=None, weight=None, state=None, x=None, Bm=None, Cm=None) == OK


def test_binding_rejects_host_tensors_and_bad_types():
    import selective_state_space_17_b200 as ssd
    x, w = torch.zeros(2, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.linear(x, torch.zeros(8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.conv(torch.zeros(1, 2, 160), torch.zeros(160, 4), None, 2, 64, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.conv_step(torch.zeros(1, 160), torch.zeros(160, 4), None, torch.zeros(1, 3, 160), 2, 64, 1, 16)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ssd.rms_norm([1.0], w)


def test_binding_refuses_sizes_beyond_int():
    """ctypes would cut them to 32 bits."""
    from selective_state_space_17_b200.layer import _sizes
    _sizes("x", 1, (1 << 31) - 1, 0)
    for bad in (1 << 31, (1 << 32) + 5, -1):
        with pytest.raises(ValueError, match="out of range"):
            _sizes("x", 3, bad)


def test_row_stride_of_views():
    from selective_state_space_17_b200.layer import _row_stride
    t = torch.zeros(3, 5, 40)
    assert _row_stride(t, "t") == 40
    assert _row_stride(t[..., 8:24], "t") == 40
    assert _row_stride(t[:1, :, :7], "t") == 40
    assert _row_stride(t[:, :1, :7], "t") == 200
    assert _row_stride(t.expand(2, 3, 5, 40)[0], "t") == 40
    for bad in (t[:, ::2, :7], t.transpose(0, 1)[..., :7]):
        with pytest.raises(ValueError, match="evenly spaced"):
            _row_stride(bad, "t")
