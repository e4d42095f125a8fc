"""64-bit definitions of the operators around the recurrent core, on the CPU
(test-side only, no code shared with the package), and what their tests share."""

from __future__ import annotations

import torch

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # rounding to a type: at most this, relative
U = 2.0 ** -24


def d(t):
    return None if t is None else t.detach().cpu().double()


def assert_within(got: torch.Tensor, want: torch.Tensor, bound, what: str):
    """|got - want| <= bound elementwise; the output's own rounding comes on top."""
    g, w = d(got), d(want)
    assert g.shape == w.shape, (what, tuple(g.shape), tuple(w.shape))
    tol = bound + EPS[got.dtype] * (w.abs() + bound)
    bad = ~((g - w).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float(((g - w).abs() / (w.abs().max() + 1e-300)).max()))


# -------------------------------------------------------------------- norm --


def norm(x, w, residual, eps):
    h = d(x)
    if residual is not None:
        h = d((x.cpu().float() + residual.cpu().float()).to(residual.dtype))
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * d(w), h


def e4m3_grid() -> torch.Tensor:
    """The non-negative E4M3 values by code 0 .. 126."""
    codes = torch.arange(127)
    e, m = codes // 8, codes % 8
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10)).double()


def e4m3_codes(v: torch.Tensor) -> torch.Tensor:
    """Codes of the nearest E4M3 values of a 64-bit tensor, ties to even codes, at most 448; 0x7F for not a number."""
    grid = e4m3_grid()
    mid = (grid[1:] + grid[:-1]) / 2
    a = v.abs()
    low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    code = torch.where(low % 2 == 0, low, high)
    code = code + 128 * torch.signbit(v)
    return torch.where(torch.isnan(v), torch.full_like(code, 0x7F), code).to(torch.uint8)


def fp8blk(y: torch.Tensor):
    """Codes and exponents of blocks of 16 values of y: the least e with max <= 464 * 2^e, in [-127, 127]."""
    b = y.reshape(-1, 16)
    m = torch.nan_to_num(b.abs(), nan=0.0).amax(-1)
    e = torch.full_like(m, -127.0)
    for k in range(-127, 127):
        e = torch.where(m > 464.0 * 2.0 ** k, float(k + 1), e)
    e = torch.where(m == 0, 0.0, e)
    return e4m3_codes(b / torch.exp2(e)[:, None]).reshape(y.shape), e.to(torch.int8)


def fp8row(y: torch.Tensor):
    m = torch.nan_to_num(y.abs(), nan=0.0).amax(-1)
    c = torch.where(m > 0, (m / 448.0).float().clamp(min=2.0 ** -126), torch.ones((), dtype=torch.float32))
    return e4m3_codes(y / c.double()[..., None]), c


# ------------------------------------------------------------- convolution --


def conv(x, w, bias, silu, state=None, lengths=None):
    """y, final state and sum |w x| + |b| (which bounds the rounding errors)."""
    x, w = d(x), d(w)
    B, T, D = x.shape
    K = w.shape[1]
    full = torch.cat([torch.zeros(B, K - 1, D, dtype=torch.float64) if state is None else d(state), x], 1)
    u = torch.zeros(B, T, D, dtype=torch.float64)
    size = torch.zeros_like(u)
    for k in range(K):
        u = u + full[:, k:k + T] * w[:, k]
        size = size + (full[:, k:k + T] * w[:, k]).abs()
    if bias is not None:
        u, size = u + d(bias), size + d(bias).abs()
    y = u * torch.sigmoid(u) if silu else u
    n = [T] * B if lengths is None else [int(v) for v in lengths]
    after = torch.stack([full[i, n[i]:n[i] + K - 1] for i in range(B)])
    return y, after, size, u


# ---------------------------------------------------------- selective scan --


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, h0=None, lengths=None, absolute=False):
    """y [B,T,D] and the final state in 64 bits (differentiable when the inputs
    are 64-bit leaves). absolute: every term's absolute value instead, with the
    true decays: what relative errors of the terms are multiplied by."""
    f = (lambda t: t.abs()) if absolute else (lambda t: t)
    B, T, nd = x.shape
    rep = nd // Bm.shape[2]
    u = dt if dt_bias is None else dt + dt_bias
    delta = torch.where(u > 30, u, torch.log1p(torch.exp(u.clamp(max=30)))) if softplus else u
    h = torch.zeros(B, nd, A.shape[1], dtype=torch.float64) if h0 is None else f(h0)
    ys = []
    for t in range(T):
        dd = delta[:, t, :, None]
        new = torch.exp(dd * A) * h + f(dd * x[:, t, :, None] * Bm[:, t].repeat_interleave(rep, 1))
        h = new if lengths is None else torch.where((t < lengths)[:, None, None], new, h)
        y = (f(Cm[:, t]).repeat_interleave(rep, 1) * h).sum(-1)
        if D is not None:
            y = y + f(D * x[:, t])
        if z is not None:
            y = y * f(z[:, t] * torch.sigmoid(z[:, t]))
        ys.append(y)
    y = torch.stack(ys, 1) if T else torch.zeros(B, 0, nd, dtype=torch.float64)
    return y, h


def scan_step_error(dt, A, dt_bias, softplus=True):
    """Relative error that one step of the recurrence may add in fp32: the
    exponential (2 units in the last place, its argument rounded twice), the
    step size (its polynomial, exponential and sum: 2^-21 and 2^-22 |u|), the
    products and the sum; a split's summed step sizes add up to T roundings."""
    u = d(dt) if dt_bias is None else d(dt) + d(dt_bias)
    delta = torch.log1p(torch.exp(u.clamp(max=30))) if softplus else u.abs()
    span = float((delta.max() * d(A).abs().max())) if u.numel() else 0.0
    rel = 2.0 ** -21 + 2.0 ** -22 * float(u.abs().max() if u.numel() else 0.0)
    T = dt.shape[1]
    return 2.0 ** -21 + 4 * U + rel * (1 + span) + span * (T + 8) * U


def scan_errors(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None):
    """Bounds of the errors of an fp32 selective scan (y before its own rounding, final state), elementwise, with every
    step's error weighted by the decay that still applies to it: err_t = a_t err_{t-1} + what the step adds.

    That is, relative to the terms' absolute values: the step size's error (its exponential and polynomial 2^-21, its
    argument 2^-22 |u|) and 4 roundings for the input; for the state's decay its exponential (2^-22, and 4 roundings)
    and |delta_t A| times the step size's error and T + 8 roundings, which covers a split's summed step sizes: each of
    the sum's T roundings is at most 2^-24 of it, and the sum's terms are the tokens' step sizes."""
    T, N = x.shape[1], A.shape[1]
    rep = x.shape[2] // Bm.shape[2]
    u = dt if dt_bias is None else dt + dt_bias
    delta = torch.where(u > 30, u, torch.log1p(torch.exp(u.clamp(max=30))))
    rel = 2.0 ** -21 + 2.0 ** -22 * u.abs()
    h = torch.zeros(x.shape[0], x.shape[2], N, dtype=torch.float64, device=x.device) if h0 is None else h0.abs()
    err = torch.zeros_like(h)
    out = []
    for t in range(T):
        dd = delta[:, t, :, None]
        a = torch.exp(dd * A)
        term, r = (dd * x[:, t, :, None] * Bm[:, t].repeat_interleave(rep, 1)).abs(), rel[:, t, :, None]
        new = a * h + term
        e = a * err + (2.0 ** -22 + 4 * U + (dd * A).abs() * (r + (T + 8) * U)) * a * h + (r + 4 * U) * term
        if lengths is not None:
            on = (t < lengths)[:, None, None]
            new, e = torch.where(on, new, h), torch.where(on, e, err)
        h, err = new, e
        C = Cm[:, t].repeat_interleave(rep, 1).abs()
        size, b = (C * h).sum(-1), (C * err).sum(-1)
        if D is not None:
            size = size + (D * x[:, t]).abs()
        b = b + (N + 4) * U * size
        if z is not None:  # the gate's exponential and division, and its product
            zt = z[:, t]
            g = (zt * torch.sigmoid(zt)).abs()
            b = b * g + (6 + 1.2 * zt.abs()) * 2 * U * size * g
        out.append(b)
    return torch.stack(out, 1), err
