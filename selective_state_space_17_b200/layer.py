"""ctypes binding of the operators around the SSD core (see include/ssd.h).

A Mamba-2 layer is ``rms_norm`` -> ``linear`` (in-projection) -> ``conv`` ->
``ssd.forward`` -> ``rms_norm`` with the gate -> ``linear`` (out-projection with
the residual); one token at a time ``conv_step`` and ``ssd.step`` take the
places of ``conv`` and ``ssd.forward``. Argument marshalling only, like
``ssd.py``: the computation runs in the CUDA library, asynchronously on the
current stream of the tensors' device or on ``stream``. With ``stream`` given,
outputs are allocated on it; as with any tensor of another stream, inputs must
be ready on it and stay alive until it has read them.
"""
from __future__ import annotations

import ctypes

import torch

from .ssd import SSD_BF16, SSD_F32, _check, _need, lib

SSD_E4M3 = 2
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}

_vp, _i, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
lib.ssd_rms_norm.argtypes = [_vp] * 3 + [_i64] + [_vp] * 4 + [_i64, _i, _i, ctypes.c_float] + [_i] * 3 + [_vp]
lib.ssd_rms_norm.restype = _i
lib.ssd_linear.argtypes = [_vp, _i64] + [_vp] * 6 + [_i] * 6 + [_vp, ctypes.c_size_t, _vp]
lib.ssd_linear.restype = _i
lib.ssd_linear_workspace_size.argtypes = [_vp, _i64] + [_i] * 4
lib.ssd_linear_workspace_size.restype = ctypes.c_size_t
lib.ssd_conv.argtypes = ([_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64] + [_vp] * 7 + [_i] * 9 + [_vp])
lib.ssd_conv.restype = _i
lib.ssd_conv_step.argtypes = [_vp, _i64, _vp, _vp, _vp, _i64] + [_vp] * 6 + [_i] * 8 + [_vp]
lib.ssd_conv_step.restype = _i

lib.ssd_set_linear_variant.argtypes = [_i]
lib.ssd_set_linear_variant.restype = None

_Tensor = torch.Tensor
_F32, _BF16, _E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
_IO = {_F32: SSD_F32, _BF16: SSD_BF16}
_UNIT = {_BF16: 8, _E4M3: 16}  # elements of 16 bytes
_OPERAND = {_F32: SSD_F32, _BF16: SSD_BF16, _E4M3: SSD_E4M3}


# The current device and stream as plain numbers: these calls stand in front of
# every launch, and the ones that build Stream objects take 2 us. (Likewise
# new_empty takes its sizes as arguments below: a tuple costs it 0.4 us more.)
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _arg(t, name, dtype, device, shape):
    """The address of a contiguous tensor argument on CUDA device number `device`
    (None stays None). The checks stand in one expression; a tensor that fails it
    goes to _need for its message."""
    if t is None:
        return None
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device
            and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, torch.device("cuda", device), shape)
    return t.data_ptr()


def _sizes(where, *sizes):
    """Refuses sizes that are no C int: ctypes would cut them to their low bits."""
    if min(sizes) < 0 or max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"{where}: a size is out of range in {sizes}")


def _io_code(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _need(t, name)
    code = _IO.get(t.dtype)
    if code is None:
        raise TypeError(f"I/O dtype must be bfloat16 or float32, got {t.dtype}")
    return code


def _strided(t, name, dtype, device, shape):
    """The address of an operand that may be a view with a contiguous last dimension."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape):
        _need(t.contiguous() if isinstance(t, torch.Tensor) else t, name, dtype, torch.device("cuda", device), shape)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr()


def _row_stride(t, name):
    """Elements from one row of the last dimension to the next, when every
    leading dimension steps by the same."""
    if t.is_contiguous():
        return t.shape[-1]
    stride = 0
    span = 0  # rows of the dimensions behind the one at hand
    for size, step in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if span == 0:
            stride, span = step, size
        elif step == stride * span:
            span *= size
        else:
            raise ValueError(f"{name}'s rows must be evenly spaced, got strides {t.stride()}")
    return stride


class _on:
    """Makes a tensor's device and the stream given for the call the current ones."""

    def __init__(self, t, stream):
        if stream is not None and stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        self._contexts = [torch.cuda.device(t.device)]
        if stream is not None:
            self._contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self._contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._contexts):
            c.__exit__(*exc)


def rms_norm(x, weight, residual=None, gate=None, eps: float = 1e-5, groups: int = 1,
             quantize: bool = False, y=None, scale=None, residual_out=None, stream=None):
    """Root-mean-square norm over the last dimension of x [..., D].

    v = x + residual, x * silu(gate) or x; y = v * weight / sqrt(mean(v^2) + eps),
    the mean over each of `groups` equal parts of the row. residual [..., D] is
    fp32 or x's dtype; v is returned in its dtype (in `residual_out`, which may
    be the residual itself). gate [..., D] may be a view with evenly spaced rows.
    With quantize, y is float8_e4m3fn and scale [...] fp32 holds one factor per
    row: y ~ scale * stored. Returns (y, scale or None, residual_out or None)."""
    code = _io_code(x, "x")
    dev = x.get_device()
    if stream is not None or dev != _device():
        with _on(x, stream):
            return rms_norm(x, weight, residual, gate, eps, groups, quantize, y, scale, residual_out)
    dtype, shape = x.dtype, x.shape
    if not shape:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    rows = x.numel() // D if D else 0
    _sizes("rms_norm", D, groups)
    px = _arg(x, "x", dtype, dev, shape)
    if weight is None:
        raise ValueError("weight is required")
    pw = _arg(weight, "weight", _F32, dev, (D,))
    pr = po = pg = None
    gate_stride, res_code = 0, code
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (_F32, dtype):
            raise TypeError(f"residual must be a tensor of torch.float32 or {dtype}")
        res_code = _IO[residual.dtype]
        pr = _arg(residual, "residual", residual.dtype, dev, shape)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
            po = residual_out.data_ptr()
        else:
            po = _arg(residual_out, "residual_out", residual.dtype, dev, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if gate is not None:
        if residual is not None:
            raise ValueError("residual and gate cannot be combined")
        pg = _strided(gate, "gate", dtype, dev, shape)
        gate_stride = _row_stride(gate, "gate")
    if quantize:
        if y is None:
            y = torch.empty_like(x, dtype=_E4M3)
        if scale is None:
            scale = x.new_empty(*shape[:-1], dtype=_F32) if len(shape) > 1 else x.new_empty((), dtype=_F32)
        py = _arg(y, "y", _E4M3, dev, shape)
        ps = _arg(scale, "scale", _F32, dev, shape[:-1])
    else:
        if scale is not None:
            raise ValueError("scale needs quantize=True")
        if y is None:
            y = torch.empty_like(x)
        py = _arg(y, "y", dtype, dev, shape)
        ps = None
    rc = lib.ssd_rms_norm(px, pr, pg, gate_stride, pw, py, ps, po, rows, D, groups, eps, code,
                          res_code, SSD_E4M3 if quantize else code, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_rms_norm")
    return y, scale, residual_out


def linear(x, w, bias=None, activation: str = "none", residual=None, x_scale=None, w_scale=None,
           out_dtype=None, y=None, stream=None):
    """act(x w^T + bias) + residual for x [..., K] and w [N, K], both fp32, both
    bf16, or both float8_e4m3fn with x_scale [...] (one per row of x, as
    rms_norm(quantize=True) gives them) and w_scale [N] in fp32.

    x may be a view with evenly spaced rows. bias [N] is fp32; activation is
    "none", "silu" or "gelu" (the one with erf); residual has the output's dtype
    and shape and may be y. The output [..., N] is out_dtype, by default y's, the
    residual's or x's dtype, and bf16 for 8-bit operands. fp32 operands keep their 24
    bits; infinities, NaN and values at the ends of the range (include/ssd.h) make the
    call several times slower."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        _need(x, "x")
    code = _OPERAND.get(x.dtype)
    if code is None:
        raise TypeError(f"x must be float32, bfloat16 or float8_e4m3fn, got {x.dtype}")
    dev = x.get_device()
    if stream is not None or dev != _device():
        with _on(x, stream):
            return linear(x, w, bias, activation, residual, x_scale, w_scale, out_dtype, y)
    dtype, lead = x.dtype, x.shape[:-1]
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or x.dim() < 1:
        raise ValueError("x must be [..., K] and w [N, K]")
    N, K = w.shape
    if x.shape[-1] != K:
        raise ValueError(f"w must have {x.shape[-1]} columns, as x has, got {K}")
    px = _strided(x, "x", dtype, dev, x.shape)
    x_stride = _row_stride(x, "x")
    pw = _arg(w, "w", dtype, dev, w.shape)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    if (dtype is _E4M3) != (x_scale is not None) or (dtype is _E4M3) != (w_scale is not None):
        raise ValueError("x_scale and w_scale go with float8_e4m3fn operands, both and only then")
    if out_dtype is None:
        out_dtype = (y.dtype if y is not None else residual.dtype if residual is not None
                     else _BF16 if dtype is _E4M3 else dtype)
    out_code = _IO.get(out_dtype)
    if out_code is None:
        raise TypeError(f"output dtype must be bfloat16 or float32, got {out_dtype}")
    shape = (*lead, N)
    if y is None:
        y = x.new_empty(*shape, dtype=out_dtype)
        py = y.data_ptr()
    else:
        py = _arg(y, "y", out_dtype, dev, shape)
    M = 1
    for n in lead:
        M *= n
    _sizes("linear", M, N, K)
    # operands that the tensor cores cannot take as they lie may need a copy; a
    # workspace of this call alone lives as long as the stream needs it (also in
    # a captured graph, whose memory pool keeps it)
    pws, nbytes = None, 0
    unit = _UNIT.get(dtype)
    if unit is None or K % unit or x_stride % unit or px % 16:
        nbytes = lib.ssd_linear_workspace_size(px, x_stride, M, N, K, code)
        if nbytes:
            workspace = x.new_empty((nbytes,), dtype=torch.uint8)
            pws = workspace.data_ptr()
    rc = lib.ssd_linear(px, x_stride, pw, _arg(x_scale, "x_scale", _F32, dev, lead),
                        _arg(w_scale, "w_scale", _F32, dev, (N,)), _arg(bias, "bias", _F32, dev, (N,)),
                        _arg(residual, "residual", out_dtype, dev, shape), py, M, N, K, act, code,
                        out_code, pws, nbytes, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_linear")
    return y


def _conv_weights(weight, bias, dt, dt_bias, C, H, dev):
    if not isinstance(weight, _Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, width]")
    if dt is None and dt_bias is not None:
        raise ValueError("dt_bias needs dt")
    W = weight.shape[1]
    return (W, _arg(weight, "weight", _F32, dev, (C, W)),
            None if bias is None else _arg(bias, "bias", _F32, dev, (C,)),
            None if dt_bias is None else _arg(dt_bias, "dt_bias", _F32, dev, (H,)))


def _conv_activation(activation):
    if activation not in ("none", "silu"):
        raise ValueError(f"activation must be none or silu, got {activation!r}")
    return ACTIVATIONS[activation]


def conv(u, weight, bias, H: int, P: int, G: int, N: int, dt=None, dt_bias=None,
         activation: str = "silu", initial_state=None, final_state=None,
         return_final_state: bool = True, stream=None):
    """Short causal convolution of u [B, L, C], C = H*P + 2*G*N, with weight
    [C, width] fp32 (width 2, 3 or 4; the last column multiplies the token
    itself) and bias [C] fp32 or None, cut into ``ssd.forward``'s operands.

    u, and dt [B, L, H] in u's dtype, may be views of the in-projection's rows.
    initial_state [B, width - 1, C] holds the inputs before token 0 (None: zeros).
    Returns (x [B, L, H, P], Bm, Cm [B, L, G, N], dt' [B, L, H] fp32 =
    softplus(dt + dt_bias) or None, final_state or None); final_state, the last
    width - 1 inputs, must not overlap initial_state."""
    code = _io_code(u, "u")
    dev = u.get_device()
    if stream is not None or dev != _device():
        with _on(u, stream):
            return conv(u, weight, bias, H, P, G, N, dt, dt_bias, activation, initial_state,
                        final_state, return_final_state)
    dtype = u.dtype
    _sizes("conv", H, P, G, N, *u.shape)
    C = H * P + 2 * G * N
    if u.dim() != 3 or u.shape[2] != C:
        raise ValueError(f"u must be [B, L, {C}], got shape {tuple(u.shape)}")
    B, L, _ = u.shape
    pu = _strided(u, "u", dtype, dev, u.shape)
    W, pw, pb, pdb = _conv_weights(weight, bias, dt, dt_bias, C, H, dev)
    act = _conv_activation(activation)
    x = u.new_empty(B, L, H, P)
    Bm = u.new_empty(B, L, G, N)
    Cm = torch.empty_like(Bm)
    out = pdt = po = None
    db = dr = 0
    if dt is not None:
        pdt = _strided(dt, "dt", dtype, dev, (B, L, H))
        db, dr, _ = dt.stride()
        out = u.new_empty(B, L, H, dtype=_F32)
        po = out.data_ptr()
    state_shape = (B, W - 1, C)
    if final_state is None and return_final_state:
        final_state = u.new_empty(*state_shape)
    ub, ur, _ = u.stride()
    rc = lib.ssd_conv(pu, ub, ur, pw, pb, pdt, db, dr, pdb,
                      _arg(initial_state, "initial_state", dtype, dev, state_shape), x.data_ptr(),
                      Bm.data_ptr(), Cm.data_ptr(), po,
                      _arg(final_state, "final_state", dtype, dev, state_shape), B, L, H, P, G, N, W,
                      act, code, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_conv")
    return x, Bm, Cm, out, final_state


def conv_step(u, weight, bias, state, H: int, P: int, G: int, N: int, dt=None, dt_bias=None,
              activation: str = "silu", stream=None):
    """``conv`` for one token per sequence, before ``ssd.step``: u [B, C] and
    dt [B, H] may be views; ``state`` [B, width - 1, C] is shifted in place.
    Returns (x [B, H, P], Bm, Cm [B, G, N], dt' [B, H] fp32 or None)."""
    code = _io_code(u, "u")
    dev = u.get_device()
    if stream is not None or dev != _device():
        with _on(u, stream):
            return conv_step(u, weight, bias, state, H, P, G, N, dt, dt_bias, activation)
    dtype = u.dtype
    _sizes("conv_step", H, P, G, N, *u.shape)
    C = H * P + 2 * G * N
    if u.dim() != 2 or u.shape[1] != C:
        raise ValueError(f"u must be [B, {C}], got shape {tuple(u.shape)}")
    B = u.shape[0]
    pu = _strided(u, "u", dtype, dev, u.shape)
    W, pw, pb, pdb = _conv_weights(weight, bias, dt, dt_bias, C, H, dev)
    act = _conv_activation(activation)
    if state is None:
        raise ValueError("state is required")
    ps = _arg(state, "state", dtype, dev, (B, W - 1, C))
    x = u.new_empty(B, H, P)
    Bm = u.new_empty(B, G, N)
    Cm = torch.empty_like(Bm)
    out = pdt = po = None
    dr = 0
    if dt is not None:
        pdt = _strided(dt, "dt", dtype, dev, (B, H))
        dr = dt.stride(0)
        out = u.new_empty(B, H, dtype=_F32)
        po = out.data_ptr()
    rc = lib.ssd_conv_step(pu, u.stride(0), pw, pb, pdt, dr, pdb, ps, x.data_ptr(), Bm.data_ptr(),
                           Cm.data_ptr(), po, B, H, P, G, N, W, act, code, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_conv_step")
    return x, Bm, Cm, out


def set_linear_variant(variant: int) -> None:
    """Test hook (not for use beside other threads' calls): 0 automatic, 1 SIMT, 2 the tensor-core kernel for few tokens,
    3 the one for many (see include/ssd.h)."""
    lib.ssd_set_linear_variant(int(variant))
