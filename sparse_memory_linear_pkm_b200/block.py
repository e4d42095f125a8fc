"""The operators around the recurrent core: the norm into a layer, the short
causal convolution, the selective scan, and the clipping of gradients.

As in the rest of the package every step runs in libsdm_b200.so; this module
checks and marshals arguments. Work goes to the current stream of the tensors'
device, whichever device is current. Token inputs (x, dt, z, B, C) may be slices
of a wider projection: contiguous in the last axes, evenly spaced over tokens
and batch rows.
"""

from __future__ import annotations

import array
import ctypes
import math
import operator

import torch

from . import native

_dtype = operator.attrgetter("dtype")
_CODE = {torch.float32: native.F32, torch.bfloat16: native.BF16}
_OUT = {"f32": native.F32, "bf16": native.BF16, "fp8blk": native.FP8_B16, "fp8row": native.FP8_ROW}


def _code(t: torch.Tensor, what: str) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    return code


def _device(t: torch.Tensor) -> int:
    """Index of the CUDA device that a call's first tensor lives on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    return dev


def _at(t: torch.Tensor | None, what: str, dev: int, shape=None, dtype=None, contiguous=True):
    """Address of a tensor (None for None) after checking where it lives and, when given, what it is."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, not on cuda:{dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _call(dev: int, fn, *args) -> None:
    """Enqueues a library call on the current stream of dev, whichever device is current."""
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        native.check(status)


def _workspace(nbytes: int, like: torch.Tensor):
    """Scratch of one call, from the allocator of the current stream (None for no bytes)."""
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _needed(lib, nbytes: int, nonempty: bool) -> int:
    if nbytes == 0 and nonempty:
        msg = lib.sdm_last_error().decode(errors="replace")
        if msg:
            raise native.SdmError(1, msg)
    return int(nbytes)


def _token_stride(t: torch.Tensor, inner: int, what: str) -> int:
    """Elements from token to token of a [B, T, ...] tensor whose later axes hold `inner` elements in order."""
    if t.is_contiguous():
        return inner
    shape, stride = t.shape, t.stride()
    run = 1
    for i in range(len(shape) - 1, 1, -1):
        if shape[i] > 1 and stride[i] != run:
            raise ValueError(f"{what} must be contiguous behind its token axis")
        run *= shape[i]
    B, T = shape[0], shape[1]
    step = stride[1] if T > 1 else (stride[0] if B > 1 else inner)
    if step < inner or (B > 1 and stride[0] != T * step):
        raise ValueError(f"{what} must be evenly spaced over tokens and batch rows")
    return step


# -------------------------------------------------------------------- norm --


def rmsnorm_residual(x: torch.Tensor, w: torch.Tensor, residual: torch.Tensor | None = None, out: str = "same",
                     eps: float = 1e-6, h: torch.Tensor | None = None):
    """h = x + residual (rounded to the residual's type; None without one) and
    y = h / sqrt(mean(h^2) + eps) * w over the last axis. Returns (y, h).

    ``out``: "same" (x's type), "f32" or "bf16"; "fp8blk": y is the buffer of
    codes and block exponents that quantize_fp8blk makes; "fp8row": y is (codes
    float8_e4m3fn [..., d], scales fp32 [...]). ``h``: where to put h (may be
    the residual itself)."""
    dev = _device(x)
    d = x.shape[-1] if x.dim() else 0
    n = x.numel() // d if d else 0
    x_code = _code(x, "x")
    if out != "same" and out not in _OUT:
        raise ValueError(f"out must be 'same' or one of {sorted(_OUT)}, got {out!r}")
    y_code = x_code if out == "same" else _OUT[out]
    res_code = native.F32
    if residual is not None:
        res_code = _code(residual, "residual")
        if h is None:
            h = torch.empty_like(residual)
    elif h is not None:
        raise ValueError("h needs a residual: without one it is x")
    scales = None
    if y_code == native.FP8_B16:
        y = x.new_empty(n * d + n * d // 16, dtype=torch.uint8)
        at_y = y.data_ptr()
        at_scales = at_y + n * d
    elif y_code == native.FP8_ROW:
        y = x.new_empty(x.shape, dtype=torch.float8_e4m3fn)
        scales = x.new_empty(x.shape[:-1], dtype=torch.float32)
        at_y, at_scales = y.data_ptr(), scales.data_ptr()
    else:
        y = x.new_empty(x.shape, dtype=torch.bfloat16 if y_code == native.BF16 else torch.float32)
        at_y, at_scales = y.data_ptr(), None
    _call(dev, native.load().sdm_rmsnorm_residual, _at(x, "x", dev), x_code,
          _at(residual, "residual", dev, x.shape), res_code, _at(w, "w", dev, (d,)), _code(w, "w"), n, d, eps,
          _at(h, "h", dev, x.shape, residual.dtype if residual is not None else None), at_y, y_code, at_scales)
    return (y if scales is None else (y, scales)), h


def dequantize_fp8blk(buf: torch.Tensor, shape, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of a block-scaled fp8 buffer (quantize_fp8blk, rmsnorm_residual
    with out="fp8blk") as a tensor of the given shape and type."""
    dev = _device(buf)
    y = buf.new_empty(shape, dtype=dtype)
    n = y.numel()
    if n % 16 or buf.numel() != n + n // 16:
        raise ValueError(f"a buffer of {n} values holds {n + n // 16} bytes, n a multiple of 16; got {buf.numel()}")
    at = _at(buf, "buf", dev, dtype=torch.uint8)
    _call(dev, native.load().sdm_dequantize_fp8blk, at, at + n, n // 16, y.data_ptr(), _code(y, "dtype"))
    return y


def dequantize_fp8row(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """codes [..., d] (float8_e4m3fn) times scales [...] (fp32), as values of the given type."""
    dev = _device(codes)
    d = codes.shape[-1]
    y = codes.new_empty(codes.shape, dtype=dtype)
    _call(dev, native.load().sdm_dequantize_fp8row, _at(codes, "codes", dev, dtype=torch.float8_e4m3fn),
          _at(scales, "scales", dev, codes.shape[:-1], torch.float32), codes.numel() // d if d else 0, d, y.data_ptr(),
          _code(y, "dtype"))
    return y


def rmsnorm_residual_backward(h: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, dh: torch.Tensor | None = None,
                              eps: float = 1e-6):
    """(dx, dw) for dy = dL/dy and dh = dL/dh (None: nothing else reads h); dx, in
    h's type, is the derivative of both x and the residual, dw is fp32."""
    dev = _device(h)
    d = h.shape[-1] if h.dim() else 0
    n = h.numel() // d if d else 0
    lib = native.load()
    ws_bytes = _needed(lib, lib.sdm_rmsnorm_residual_backward_workspace_bytes(n, d), n > 0)
    ws = _workspace(ws_bytes, h)
    dx = torch.empty_like(h)
    dw = h.new_empty(d, dtype=torch.float32)
    _call(dev, lib.sdm_rmsnorm_residual_backward, _at(h, "h", dev), _code(h, "h"), _at(w, "w", dev, (d,)),
          _code(w, "w"), _at(dy, "dy", dev, h.shape), _code(dy, "dy"), _at(dh, "dh", dev, h.shape, h.dtype), n, d, eps,
          dx.data_ptr(), dw.data_ptr(), None if ws is None else ws.data_ptr(), ws_bytes)
    return dx, dw


# ------------------------------------------------------------- convolution --


def _conv_sizes(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None):
    if x.dim() != 3 or w.dim() != 2 or w.shape[0] != x.shape[2]:
        raise ValueError(f"x must be [B, T, D] and w [D, K], got {tuple(x.shape)} and {tuple(w.shape)}")
    if bias is not None and bias.dtype != w.dtype:
        raise TypeError(f"bias must have w's type {w.dtype}, got {bias.dtype}")
    B, T, D = x.shape
    return B, T, D, w.shape[1]


def short_conv(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None, silu: bool = True,
               state: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
               y: torch.Tensor | None = None) -> torch.Tensor:
    """Causal depthwise convolution of x [B,T,D] with w [D,K] over the tokens, plus
    bias [D], then SiLU. ``state`` [B,K-1,D] holds the inputs before the first
    token and is updated in place (decode: T = 1 per call); without it they are
    zeros. ``lengths`` [B] int32: tokens of each row, y behind them is left as it
    is. Returns y [B,T,D] in x's type (``y`` itself when given)."""
    dev = _device(x)
    B, T, D, K = _conv_sizes(x, w, bias)
    if y is None:
        y = x.new_empty(x.shape) if lengths is None else x.new_zeros(x.shape)
    _call(dev, native.load().sdm_short_conv, _at(x, "x", dev, contiguous=False), _token_stride(x, D, "x"),
          _code(x, "x"), _at(w, "w", dev), _at(bias, "bias", dev, (D,)), _code(w, "w"), B, T, D, K, int(silu),
          _at(state, "state", dev, (B, K - 1, D), x.dtype), _at(lengths, "lengths", dev, (B,), torch.int32),
          _at(y, "y", dev, x.shape, x.dtype))
    return y


def short_conv_backward(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, bias: torch.Tensor | None = None,
                        silu: bool = True, state0: torch.Tensor | None = None, dstate: torch.Tensor | None = None,
                        lengths: torch.Tensor | None = None) -> dict:
    """Derivatives of short_conv for dy = dL/dy and dstate = dL/d(final state): dx
    (x's type), dw and dbias (fp32; None without bias), and dstate0 (None unless
    state0 or dstate is given). state0 is the state before the call."""
    dev = _device(x)
    B, T, D, K = _conv_sizes(x, w, bias)
    lib = native.load()
    ws_bytes = _needed(lib, lib.sdm_short_conv_backward_workspace_bytes(B, T, D, K), B * T * D > 0)
    ws = _workspace(ws_bytes, x)
    dx = x.new_empty(x.shape)
    dw = x.new_empty((D, K), dtype=torch.float32)
    dbias = x.new_empty(D, dtype=torch.float32) if bias is not None else None
    dstate0 = None
    if state0 is not None or dstate is not None:
        dstate0 = x.new_empty((B, K - 1, D))
    _call(dev, lib.sdm_short_conv_backward, _at(x, "x", dev, contiguous=False), _token_stride(x, D, "x"),
          _code(x, "x"), _at(w, "w", dev), _at(bias, "bias", dev, (D,)), _code(w, "w"), B, T, D, K, int(silu),
          _at(state0, "state0", dev, (B, K - 1, D), x.dtype), _at(lengths, "lengths", dev, (B,), torch.int32),
          _at(dy, "dy", dev, x.shape, x.dtype), _at(dstate, "dstate", dev, (B, K - 1, D), x.dtype), dx.data_ptr(),
          dw.data_ptr(), None if dbias is None else dbias.data_ptr(), None if dstate0 is None else dstate0.data_ptr(),
          None if ws is None else ws.data_ptr(), ws_bytes)
    return {"dx": dx, "dw": dw, "dbias": dbias, "dstate0": dstate0}


# ---------------------------------------------------------- selective scan --


def _selscan_args(dev, x, dt, A, B, C, D, z, dt_bias, softplus, lengths):
    """The shape structure and the addresses that the scan and its gradient share."""
    if x.dim() != 3 or A.dim() != 2 or A.shape[0] != x.shape[2]:
        raise ValueError(f"x must be [B, T, D] and A [D, N], got {tuple(x.shape)} and {tuple(A.shape)}")
    nb, T, nd = x.shape
    N = A.shape[1]
    if B.dim() != 4 or B.shape[:2] != x.shape[:2] or B.shape[3] != N or C.shape != B.shape:
        raise ValueError(f"B and C must be [B, T, G, N], got {tuple(B.shape)} and {tuple(C.shape)}")
    G = B.shape[2]
    shape = native.SelscanShape(nb, T, nd, N, G, _code(x, "x"), int(softplus), 0, _token_stride(x, nd, "x"),
                                _token_stride(dt, nd, "dt"), 0 if z is None else _token_stride(z, nd, "z"),
                                _token_stride(B, G * N, "B"), _token_stride(C, G * N, "C"))
    f32, t = torch.float32, x.dtype
    return shape, (_at(x, "x", dev, contiguous=False), _at(dt, "dt", dev, x.shape, t, False),
                   _at(A, "A", dev, dtype=f32), _at(B, "B", dev, None, t, False), _at(C, "C", dev, None, t, False),
                   _at(D, "D", dev, (nd,), f32), _at(z, "z", dev, x.shape, t, False),
                   _at(dt_bias, "dt_bias", dev, (nd,), f32), _at(lengths, "lengths", dev, (nb,), torch.int32))


def selective_scan(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                   dt_bias: torch.Tensor | None = None, softplus: bool = True, state: torch.Tensor | None = None,
                   lengths: torch.Tensor | None = None, y: torch.Tensor | None = None) -> torch.Tensor:
    """Selective state space scan over x, dt [B,T,D] with A [D,N] (fp32) and B, C
    [B,T,G,N]: h <- exp(delta A) h + delta x B, y = (C.h + D x) silu(z) with delta =
    softplus(dt + dt_bias). ``state`` [B,D,N] fp32 is read as the state before the
    first token and updated in place (decode: T = 1 per call); None starts from
    zeros. ``lengths`` [B] int32: tokens of each row, y behind them is left as it
    is. Returns y [B,T,D] in x's type (``y`` itself when given)."""
    dev = _device(x)
    shape, args = _selscan_args(dev, x, dt, A, B, C, D, z, dt_bias, softplus, lengths)
    lib = native.load()
    ref = ctypes.byref(shape)
    ws_bytes = lib.sdm_selective_scan_workspace_bytes(ref)
    ws = _workspace(ws_bytes, x)
    if y is None:
        y = x.new_empty(x.shape) if lengths is None else x.new_zeros(x.shape)
    at_state = _at(state, "state", dev, (shape.B, shape.D, shape.N), torch.float32)
    _call(dev, lib.sdm_selective_scan, ref, *args, at_state, at_state, _at(y, "y", dev, x.shape, x.dtype),
          None if ws is None else ws.data_ptr(), ws_bytes)
    return y


def selective_scan_backward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                            dy: torch.Tensor, D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                            dt_bias: torch.Tensor | None = None, softplus: bool = True,
                            state0: torch.Tensor | None = None, dstate: torch.Tensor | None = None,
                            lengths: torch.Tensor | None = None) -> dict:
    """Derivatives of selective_scan for dy = dL/dy and dstate = dL/d(final state):
    dx, ddt, dz, dB, dC (x's type), dA, dD, ddt_bias (fp32) and dstate0 (fp32, None
    unless state0 or dstate is given); None for inputs that are not there."""
    dev = _device(x)
    shape, args = _selscan_args(dev, x, dt, A, B, C, D, z, dt_bias, softplus, lengths)
    lib = native.load()
    ref = ctypes.byref(shape)
    ws_bytes = _needed(lib, lib.sdm_selective_scan_backward_workspace_bytes(ref), x.numel() > 0)
    ws = _workspace(ws_bytes, x)
    like = lambda t: t.new_empty(t.shape)  # noqa: E731
    states = (shape.B, shape.D, shape.N)
    out = {"dx": like(x), "ddt": like(x), "dA": like(A), "dB": like(B), "dC": like(B),
           "dD": None if D is None else like(D), "dz": None if z is None else like(x),
           "ddt_bias": None if dt_bias is None else like(dt_bias), "dstate0": None}
    if state0 is not None or dstate is not None:
        out["dstate0"] = A.new_empty(states)
    at = {k: None if v is None else v.data_ptr() for k, v in out.items()}
    _call(dev, lib.sdm_selective_scan_backward, ref, *args, _at(state0, "state0", dev, states, torch.float32),
          _at(dy, "dy", dev, x.shape, x.dtype), _at(dstate, "dstate", dev, states, torch.float32), at["dx"], at["ddt"],
          at["dA"], at["dB"], at["dC"], at["dD"], at["dz"], at["ddt_bias"], at["dstate0"],
          None if ws is None else ws.data_ptr(), ws_bytes)
    return out


# ---------------------------------------------------------------- clipping --


def grad_norm_clip(grads, max_norm: float, eps: float = 1e-6, out=None) -> torch.Tensor:
    """The 2-norm of all the tensors' values together (a 0-dim fp32 tensor on their
    device; nothing waits for it), with every value scaled by min(1, max_norm /
    (norm + eps)): in place, or into ``out``, a list of tensors of the same sizes
    (fp32 or bf16 each). max_norm = inf only measures, or copies into ``out``."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
    if not grads:
        raise ValueError("no gradients")
    dev = _device(grads[0])
    # A list has hundreds of tensors: each is asked as little as possible, and which one is wrong only then.
    at, codes, sizes = _flat(grads, dev, "gradient")
    if out is None:
        out_at, out_codes = ([0] * len(at) if max_norm == math.inf else at), codes
    else:
        out_at, out_codes, out_sizes = _flat(outs, dev, "output")
        if out_sizes != sizes:
            i = next(i for i, (a, b) in enumerate(zip(out_sizes, sizes)) if a != b)
            raise ValueError(f"output {i} has {out_sizes[i]} values, its gradient {sizes[i]}")
    table = [0] * (4 * len(at))  # an array of sdm_grad_tensor_t
    table[::4], table[1::4], table[2::4] = at, out_at, sizes
    table[3::4] = [a | b << 32 for a, b in zip(codes, out_codes)]
    packed = array.array("q", table)
    lib = native.load()
    ws_bytes = lib.sdm_grad_norm_clip_workspace_bytes(len(at))
    ws = _workspace(ws_bytes, grads[0])
    norm = grads[0].new_empty((), dtype=torch.float32)
    _call(dev, lib.sdm_grad_norm_clip, packed.buffer_info()[0], len(at), max_norm, eps, norm.data_ptr(),
          ws.data_ptr(), ws_bytes)
    return norm


def _flat(tensors, dev: int, what: str):
    """Addresses, type codes and sizes of contiguous tensors on dev."""
    T = torch.Tensor
    if set(map(T.get_device, tensors)) != {dev} or not all(map(T.is_contiguous, tensors)):
        i = next(i for i, t in enumerate(tensors) if not (t.is_contiguous() and t.get_device() == dev))
        raise ValueError(f"{what} {i} must be contiguous and on cuda:{dev}")
    types = list(map(_dtype, tensors))
    kinds = set(types)
    if not kinds <= _CODE.keys():
        i = next(i for i, t in enumerate(types) if t not in _CODE)
        raise TypeError(f"{what} {i} must be float32 or bfloat16, got {types[i]}")
    codes = [_CODE[types[0]]] * len(types) if len(kinds) == 1 else [_CODE[t] for t in types]
    return list(map(T.data_ptr, tensors)), codes, list(map(T.numel, tensors))
