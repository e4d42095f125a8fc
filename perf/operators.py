"""Workloads of the operators around the recurrent core, for measuring them.

Each case names one operator call with its sizes; ``prepare`` makes its inputs,
``run`` makes one pass: in plain torch operations (``own`` false), or through the
package's entry points (``own`` true). ``exact`` gives the same results from the
definitions in 64 bits.

Operators: the RMS norm with the residual's addition (bf16/fp32 output or 8 bits
with scales) and its gradient, the short causal convolution and its gradient, the
selective scan and its gradient, and the global gradient norm with clipping.
"""

import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases --


def listed():
    return [
        # the norm into a layer for 64 sequences that decode one token each: latency
        {"name": "norm_step_blk", "op": "norm", "rows": 64, "d": 2048, "x": "bf16", "res": "bf16", "out": "fp8blk"},
        # the same over a prompt batch, fp32 residual stream, one scale per row for an 8-bit projection
        {"name": "norm_prompt_row", "op": "norm", "rows": 16384, "d": 4096, "x": "bf16", "res": "f32",
         "out": "fp8row"},
        # its gradient over a training batch of 8 x 4096 tokens
        {"name": "norm_train_grad", "op": "norm_grad", "rows": 32768, "d": 2048, "x": "bf16", "dh": True},
        # the convolution for 128 sequences that decode one token each, state carried: latency
        {"name": "conv_step", "op": "conv", "B": 128, "T": 1, "D": 4096, "K": 4, "x": "bf16", "silu": True,
         "bias": True, "ragged": False, "state": True, "packed": True},
        # a padded batch of prompts of unequal, odd lengths, read out of a wider projection
        {"name": "conv_prompt", "op": "conv", "B": 6, "T": 4099, "D": 4096, "K": 4, "x": "bf16", "silu": True,
         "bias": True, "ragged": True, "state": True, "packed": True},
        # its gradient over a training batch
        {"name": "conv_train_grad", "op": "conv_grad", "B": 8, "T": 4096, "D": 2048, "K": 4, "x": "bf16",
         "silu": True, "bias": True},
        # the scan for 128 sequences that decode one token each, state carried in place
        {"name": "scan_step", "op": "scan", "B": 128, "T": 1, "D": 4096, "N": 16, "G": 1, "x": "bf16", "z": True,
         "ragged": False, "state": True, "packed": True},
        # a padded batch of prompts
        {"name": "scan_prompt", "op": "scan", "B": 6, "T": 2047, "D": 2048, "N": 16, "G": 1, "x": "bf16",
         "z": True, "ragged": True, "state": True, "packed": True},
        # one long document: few rows, the long axis has to be split
        {"name": "scan_long", "op": "scan", "B": 1, "T": 65536, "D": 2048, "N": 16, "G": 1, "x": "bf16", "z": True,
         "ragged": False, "state": True, "packed": False},
        # the gradient of a training batch
        {"name": "scan_train_grad", "op": "scan_grad", "B": 2, "T": 4096, "D": 2048, "N": 16, "G": 1, "x": "bf16",
         "z": True},
        # the gradients of a small model, many tensors of few values: launches and host work count
        {"name": "clip_many_small", "op": "clip", "tensors": 160, "most": 65536, "x": "f32", "out": "f32"},
        # bf16 gradients of a large model into its fp32 master buffer
        {"name": "clip_large", "op": "clip", "tensors": 290, "most": 16777216, "x": "bf16", "out": "f32"},
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "conv", "conv_grad", "scan", "scan", "scan_grad", "clip"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        out = rng.choice(["same", "fp8blk", "fp8row"]) if op == "norm" else "same"
        d = _log(rng, 64, 8192)
        if out != "same":
            d = (d + 15) // 16 * 16
        rows = _log(rng, 1, min(32768, (1 << 26) // d))
        if op == "norm_grad":
            return {"op": op, "rows": rows, "d": d, "x": x, "dh": rng.random() < 0.7}
        return {"op": op, "rows": rows, "d": d, "x": x, "res": rng.choice(["bf16", "f32", ""]), "out": out}
    if op in ("conv", "conv_grad"):
        D = _log(rng, 64, 4096)
        T = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(128, (1 << 26) // (D * T))))
        c = {"op": op, "B": B, "T": T, "D": D, "K": rng.randint(2, 4), "x": x, "silu": rng.random() < 0.8,
             "bias": rng.random() < 0.7}
        if op == "conv":
            c.update(ragged=rng.random() < 0.5, state=rng.random() < 0.7, packed=rng.random() < 0.5)
        return c
    if op in ("scan", "scan_grad"):
        G = rng.choice([1, 1, 1, 2, 4])
        N = rng.choice([8, 16, 16, 16, 16, 24, 32, 64])
        D = G * _log(rng, 64 // G, 4096 // G)
        most = (1 << 30) if op == "scan" else (1 << 28)
        T = _log(rng, 1, min(32768, most // (D * N)))
        B = _log(rng, 1, max(1, min(128, most // (D * N * T))))
        c = {"op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "x": x, "z": rng.random() < 0.7}
        if op == "scan":
            c.update(ragged=rng.random() < 0.5, state=rng.random() < 0.7, packed=rng.random() < 0.5)
        return c
    return {"op": "clip", "tensors": _log(rng, 1, 300), "most": _log(rng, 4096, 1 << 22), "x": x,
            "out": "f32" if x == "f32" else rng.choice(["f32", "bf16"])}


def _sizes(case):
    """Element counts of a clip case's tensors: mostly matrices of the largest
    size and fractions of it, with vectors and odd sizes between them."""
    n, most = case["tensors"], case["most"]
    return [max(1, (most, most // 4, most // 256 + 1, most // 3 - 1, most // 1024)[i % 5] - (i % 7 == 6))
            for i in range(n)]


# ------------------------------------------------------------------ inputs --


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    dtype = TYPES[case["x"]]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    def uniform(*shape, low=0.0, high=1.0):
        return torch.rand(shape, generator=gen, device="cuda") * (high - low) + low

    s = dict(case)
    if op == "norm":
        s["x"] = normal(case["rows"], case["d"])
        s["res"] = normal(case["rows"], case["d"], scale=3.0, to=TYPES[case["res"]]) if case["res"] else None
        s["w"] = uniform(case["d"], low=0.5, high=1.5)
    elif op == "norm_grad":
        s["h"] = normal(case["rows"], case["d"], scale=3.0)
        s["dy"] = normal(case["rows"], case["d"], scale=0.1)
        s["dh"] = normal(case["rows"], case["d"], scale=0.1) if case["dh"] else None
        s["w"] = uniform(case["d"], low=0.5, high=1.5)
    elif op in ("conv", "conv_grad"):
        B, T, D, K = case["B"], case["T"], case["D"], case["K"]
        if case.get("packed"):  # the first half of a projection [B, T, 2 D]
            s["x"] = normal(B, T, 2 * D)[..., :D]
        else:
            s["x"] = normal(B, T, D)
        s["w"] = uniform(D, K, low=-1.0, high=1.0) / math.sqrt(K)
        s["b"] = normal(D, scale=0.1, to=torch.float32) if case["bias"] else None
        if op == "conv":
            s["state"] = normal(B, K - 1, D) if case["state"] else None
            s["lengths"] = _lengths(B, T, gen) if case["ragged"] else None
            s["y"] = torch.zeros((B, T, D), dtype=dtype, device="cuda")
        else:
            s["dy"] = normal(B, T, D, scale=0.1)
    elif op in ("scan", "scan_grad"):
        B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
        s["x"] = normal(B, T, D)
        # step sizes of a trained model: softplus(dt + bias) between 0.001 and 0.1, log-uniform
        step = torch.exp(uniform(D, low=math.log(0.001), high=math.log(0.1)))
        s["bias"] = step + torch.log(-torch.expm1(-step))
        s["dt"] = normal(B, T, D, scale=0.5)
        s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=torch.float32).repeat(D, 1)
                   * uniform(D, N, low=0.8, high=1.2))
        s["D_"] = uniform(D, low=0.5, high=1.5)
        if case.get("packed"):  # B and C as slices of one projection, z as half of another
            both = normal(B, T, 2 * G * N)
            s["Bm"] = both[..., :G * N].unflatten(-1, (G, N))
            s["Cm"] = both[..., G * N:].unflatten(-1, (G, N))
            s["z"] = normal(B, T, 2 * D)[..., D:] if case["z"] else None
        else:
            s["Bm"], s["Cm"] = normal(B, T, G, N), normal(B, T, G, N)
            s["z"] = normal(B, T, D) if case["z"] else None
        if op == "scan":
            s["state"] = normal(B, D, N, scale=0.1, to=torch.float32) if case["state"] else None
            s["lengths"] = _lengths(B, T, gen) if case["ragged"] else None
            s["y"] = torch.zeros((B, T, D), dtype=dtype, device="cuda")
        else:
            s["dy"] = normal(B, T, D, scale=0.1)
    else:
        sizes = _sizes(case)
        s["grads"] = [normal(n, scale=0.02 if i % 3 else 0.002) for i, n in enumerate(sizes)]
        s["flat"] = torch.empty(sum(-(-n // 8) * 8 for n in sizes), dtype=TYPES[case["out"]], device="cuda").zero_()
        at = [0]
        for n in sizes:
            at.append(at[-1] + -(-n // 8) * 8)
        s["outs"] = [s["flat"][a:a + n] for a, n in zip(at, sizes)]
        s["max_norm"] = 1.0
    return s


def _lengths(B, T, gen):
    n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = T
    return n


# -------------------------------------------------------------------- pass --


def run(s):
    op = s["op"]
    if own:
        import sparse_memory_linear_pkm_b200 as sdm

        if op == "norm":
            y, h = sdm.rmsnorm_residual(s["x"], s["w"], s["res"], out=s["out"], eps=EPS)
            if s["out"] == "fp8blk":
                return [sdm.dequantize_fp8blk(y, s["x"].shape, torch.bfloat16), h]
            if s["out"] == "fp8row":
                codes, scales = y
                return [sdm.dequantize_fp8row(codes, scales, torch.bfloat16), scales, h]
            return [y, h]
        if op == "norm_grad":
            return sdm.rmsnorm_residual_backward(s["h"], s["w"], s["dy"], s["dh"], eps=EPS)
        if op == "conv":
            y = sdm.short_conv(s["x"], s["w"], s["b"], silu=s["silu"], state=s["state"], lengths=s["lengths"],
                               y=s["y"])
            return [y, s["state"]]
        if op == "conv_grad":
            return sdm.short_conv_backward(s["x"], s["w"], s["dy"], s["b"], silu=s["silu"])
        if op == "scan":
            y = sdm.selective_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D_"], z=s["z"],
                                   dt_bias=s["bias"], softplus=True, state=s["state"], lengths=s["lengths"],
                                   y=s["y"])
            return [y, s["state"]]
        if op == "scan_grad":
            return sdm.selective_scan_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], D=s["D_"],
                                               z=s["z"], dt_bias=s["bias"], softplus=True)
        norm = sdm.grad_norm_clip(s["grads"], s["max_norm"], eps=EPS, out=s["outs"])
        return [norm, s["flat"]]
    return {"norm": _norm, "norm_grad": _norm_grad, "conv": _conv, "conv_grad": _conv_grad, "scan": _scan,
            "scan_grad": _scan_grad, "clip": _clip}[op](s)


def _norm(s):
    x, w = s["x"], s["w"]
    if s["res"] is not None:
        h = (x.float() + s["res"].float()).to(s["res"].dtype)
    else:
        h = x
    back = h if s["res"] is not None else None
    if s["out"] == "same":
        f = h.float()
        y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
        return [y.to(x.dtype), back]
    # which grid point a value rounds to is decided next to borders: 64 bits
    f = h.double()
    y = f * (1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)) * w.double()
    if s["out"] == "fp8blk":
        b = y.unflatten(-1, (-1, 16))
        m = b.abs().amax(-1, keepdim=True)
        frac, k = torch.frexp(m)  # m = frac 2^k
        e = torch.where(m > 0, (k - 9 + (frac > 0.90625)).clamp(-127, 127), torch.zeros_like(k))
        return [(_e4m3(torch.ldexp(b, -e)) * torch.ldexp(torch.ones_like(m), e)).flatten(-2).to(torch.bfloat16), back]
    m = y.abs().amax(-1, keepdim=True)
    c = torch.where(m > 0, (m / 448.0).float(), torch.ones_like(m, dtype=torch.float32))
    return [(_e4m3(y / c.double()).float() * c).to(torch.bfloat16), c.squeeze(-1), back]


def _e4m3(v):
    """v (64 bits) rounded to the nearest E4M3 value, ties to even, at most 448."""
    _, k = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (k - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _norm_grad(s):
    h, dy, w = s["h"].float(), s["dy"].float(), s["w"]
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    g = dy * w
    dx = g * r - h * (r * r * r) * (g * h).mean(-1, keepdim=True)
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(s["h"].dtype), (dy * h * r).sum(0)]


def _live(s, T):
    """[B, T, 1] truth values: the token is one of its sequence, not padding."""
    t = torch.arange(T, device="cuda")[None, :, None]
    n = s["lengths"]
    return t < (n[:, None, None] if n is not None else T)


def _windows(x, state, K):
    """x with the K - 1 inputs before it: [B, T + K - 1, D] in 32 bits."""
    before = state.float() if state is not None else x.new_zeros((x.shape[0], K - 1, x.shape[2]), dtype=torch.float32)
    return torch.cat([before, x.float()], 1)


def _conv(s):
    x, w, K = s["x"], s["w"], s["K"]
    T = x.shape[1]
    full = _windows(x, s["state"], K)
    u = sum(full[:, k:k + T] * w[:, k] for k in range(K))
    if s["b"] is not None:
        u = u + s["b"]
    y = u * torch.sigmoid(u) if s["silu"] else u
    s["y"].copy_(torch.where(_live(s, T), y, s["y"].float()))
    if s["state"] is not None:
        at = torch.arange(K - 1, device="cuda")[None, :] + (s["lengths"][:, None] if s["lengths"] is not None else T)
        s["state"].copy_(full.gather(1, at.long()[:, :, None].expand(x.shape[0], K - 1, x.shape[2])))
    return [s["y"], s["state"]]


def _conv_grad(s):
    x, w, K = s["x"], s["w"], s["K"]
    T = x.shape[1]
    full = _windows(x, None, K)
    u = sum(full[:, k:k + T] * w[:, k] for k in range(K))
    if s["b"] is not None:
        u = u + s["b"]
    du = s["dy"].float()
    if s["silu"]:
        g = torch.sigmoid(u)
        du = du * (g * (1 + u * (1 - g)))
    late = torch.cat([du, du.new_zeros((x.shape[0], K - 1, x.shape[2]))], 1)
    dx = sum(late[:, K - 1 - k:K - 1 - k + T] * w[:, k] for k in range(K))
    dw = torch.stack([(du * full[:, k:k + T]).sum((0, 1)) for k in range(K)], -1)
    return {"dx": dx.to(x.dtype), "dw": dw, "dbias": du.sum((0, 1)) if s["b"] is not None else None, "dstate0": None}


def _steps(s):
    """Step sizes [B, T, D] (0 for padding) and what softplus was taken of."""
    u = s["dt"].float() + s["bias"]
    return torch.where(u > 20, u, torch.log1p(torch.exp(u.clamp(max=20)))), u


def _spread(m, D):
    """[B, T, G, N] -> [B, T, D, N] in 32 bits: each group's row for its channels."""
    B, T, G, N = m.shape
    return m.float()[:, :, :, None].expand(B, T, G, D // G, N).reshape(B, T, D, N)


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 by doubling: every step joins runs twice as long."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1) if 2 * k < b.shape[1] else a
        k *= 2
    return b


def _scan(s):
    x, D = s["x"].float(), s["D"]
    T = x.shape[1]
    live = _live(s, T)
    delta, _ = _steps(s)
    delta = delta * live
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * _spread(s["Bm"], D)
    if s["state"] is not None:
        b[:, 0] += a[:, 0] * s["state"]
    h = _recur(a, b)
    del a, b
    y = (h * _spread(s["Cm"], D)).sum(-1) + x * s["D_"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["y"].copy_(torch.where(live, y, s["y"].float()))
    if s["state"] is not None:
        s["state"].copy_(h[:, -1])
    return [s["y"], s["state"]]


def _scan_grad(s):
    x, D, A, G = s["x"].float(), s["D"], s["A"], s["G"]
    B, T, _ = x.shape
    delta, u = _steps(s)
    a = torch.exp(delta[..., None] * A)
    Bm, Cm = _spread(s["Bm"], D), _spread(s["Cm"], D)
    b = (delta * x)[..., None] * Bm
    h = _recur(a, b)
    kept = h - b  # a_t h_{t-1}
    kept[:, 0] = 0
    e = s["dy"].float()
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        q = torch.sigmoid(z)
        y = (h * Cm).sum(-1) + x * s["D_"]
        dz = (e * y * (q * (1 + z * (1 - q)))).to(s["x"].dtype)
        e = e * (z * q)
    dC = (e[..., None] * h).unflatten(2, (G, -1)).sum(3)
    del b, h
    after = torch.cat([a[:, 1:], a[:, :1]], 1).flip(1)
    g = _recur(after, (e[..., None] * Cm).flip(1)).flip(1)
    del after, a, Cm
    dB = (g * (delta * x)[..., None]).unflatten(2, (G, -1)).sum(3)
    p = (g * Bm).sum(-1)
    g = g * kept
    du = (x * p + (g * A).sum(-1)) * torch.sigmoid(u)
    t = s["x"].dtype
    return {"dx": (delta * p + e * s["D_"]).to(t), "ddt": du.to(t), "dA": (g * delta[..., None]).sum((0, 1)),
            "dB": dB.to(t), "dC": dC.to(t), "dD": (e * x).sum((0, 1)), "dz": dz, "ddt_bias": du.sum((0, 1)),
            "dstate0": None}


def _clip(s):
    flat = torch.cat([g.float() for g in s["grads"]])
    norm = torch.sqrt((flat * flat).sum())
    flat = flat * (s["max_norm"] / (norm + EPS)).clamp(max=1.0)
    [o.copy_(g) for o, g in zip(s["outs"], flat.split([g.numel() for g in s["grads"]]))]
    return [norm, s["flat"]]


# -------------------------------------------------------------------- work --


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op, n = case["op"], SIZE[case["x"]]
    if op == "norm":
        e = case["rows"] * case["d"]
        r = SIZE[case["res"]] if case["res"] else 0
        out = {"same": n, "fp8blk": 2 * (1 + 1 / 16) + 2, "fp8row": 2 + 2}[case["out"]]
        return {"bytes": e * (n + 2 * r + out) + 4 * case["d"], "flops": 6 * e}
    if op == "norm_grad":
        e = case["rows"] * case["d"]
        return {"bytes": e * n * (3 + case["dh"]) + 8 * case["d"], "flops": 12 * e}
    if op in ("conv", "conv_grad"):
        e = case["B"] * case["T"] * case["D"]
        state = 2 * n * case["B"] * (case["K"] - 1) * case["D"] * bool(case.get("state"))
        live = 0.6 if case.get("ragged") else 1.0  # padding is neither read nor written
        more = 1 if op == "conv" else 3
        return {"bytes": live * e * n * (2 if op == "conv" else 3) + state + 4 * case["D"] * (case["K"] + 1),
                "flops": live * e * more * (2 * case["K"] + 4)}
    if op in ("scan", "scan_grad"):
        e = case["B"] * case["T"] * case["D"]
        bc = 2 * n * case["B"] * case["T"] * case["G"] * case["N"]
        par = 4 * case["D"] * (case["N"] + 2)
        live = 0.6 if case.get("ragged") else 1.0
        if op == "scan":
            state = 8 * case["B"] * case["D"] * case["N"] * bool(case["state"])
            return {"bytes": live * (e * n * (3 + case["z"]) + bc) + state + par, "flops": live * e * 7 * case["N"]}
        return {"bytes": e * n * (5 + 2 * case["z"]) + 2 * bc + 2 * par, "flops": e * 24 * case["N"]}
    total = sum(_sizes(case))
    return {"bytes": total * (n + SIZE[case["out"]]), "flops": 3 * total}


# ----------------------------------------------------- definitions, 64 bits --


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f = lambda t: None if t is None else t.double()  # noqa: E731
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_grad":
        h, w = f(s["h"]).requires_grad_(), f(s["w"]).requires_grad_()
        y = h / h.square().mean(-1, keepdim=True).add(EPS).sqrt() * w
        loss = (y * f(s["dy"])).sum() + (0 if s["dh"] is None else (h * f(s["dh"])).sum())
        return list(torch.autograd.grad(loss, [h, w]))
    if op in ("conv", "conv_grad"):
        return _exact_conv(s, op == "conv_grad")
    if op in ("scan", "scan_grad"):
        if s["T"] > 70000:
            return None
        return _exact_scan(s, op == "scan_grad")
    total = torch.stack([f(g).square().sum() for g in s["grads"]]).sum().sqrt()
    c = min(1.0, s["max_norm"] / (float(total) + EPS))
    flat = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
    at = 0
    for g in s["grads"]:
        flat[at:at + g.numel()] = f(g) * c
        at += -(-g.numel() // 8) * 8
    return [total, flat]


def _exact_norm(s):
    x, w = s["x"].double(), s["w"].double()
    h = x if s["res"] is None else x + s["res"].double()
    kept = h if s["res"] is None else h.to(s["res"].dtype).double()
    y = kept / torch.sqrt(torch.linalg.vecdot(kept, kept)[:, None] / s["d"] + EPS) * w
    back = None if s["res"] is None else h
    if s["out"] == "same":
        return [y, back]
    # every positive E4M3 value, and the borders between neighbours
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)]
                        + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device="cuda")
    border = (grid[1:] + grid[:-1]) / 2

    def nearest(v):
        a = v.abs()
        low, high = torch.bucketize(a, border), torch.bucketize(a, border, right=True)
        i = torch.where(low % 2 == 0, low, high)  # on a border: the even code
        return torch.copysign(grid[i], v)

    if s["out"] == "fp8blk":
        m = y.reshape(-1, 16).abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(m.clamp(min=1e-300) / 464.0))
        e = torch.where(m <= 464.0 * torch.exp2(e - 1), e - 1, torch.where(m > 464.0 * torch.exp2(e), e + 1, e))
        e = torch.where(m > 0, e.clamp(-127, 127), torch.zeros_like(e))
        return [(nearest(y.reshape(-1, 16) / torch.exp2(e)) * torch.exp2(e)).reshape(y.shape), back]
    m = y.abs().amax(-1)
    c = (m / 448.0).float().double()
    c[m == 0] = 1.0
    return [nearest(y / c[:, None]) * c[:, None], c, back]


def _exact_conv(s, grad):
    B, T, D, K = s["B"], s["T"], s["D"], s["K"]
    x, w = s["x"].double(), s["w"].double()
    b = torch.zeros(D, dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double()
    state = s.get("state")
    if grad:
        x, w, b = x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    full = torch.nn.functional.pad(x, (0, 0, K - 1, 0))
    if state is not None:
        full[:, :K - 1] = state.double()
    u = torch.einsum("btdk,dk->btd", full.unfold(1, K, 1), w) + b
    y = u / (1 + torch.exp(-u)) if s["silu"] else u
    if grad:
        dx, dw, db = torch.autograd.grad((y * s["dy"].double()).sum(), [x, w, b])
        return {"dx": dx, "dw": dw, "dbias": db if s["b"] is not None else None, "dstate0": None}
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    for i in range(B):
        y[i, n[i]:] = 0
    after = None if state is None else torch.stack([full[i, n[i]:n[i] + K - 1] for i in range(B)])
    return [y, after]


def _exact_scan(s, grad):
    B, T, D, N, G = s["B"], s["T"], s["D"], s["N"], s["G"]
    names = ["x", "dt", "A", "Bm", "Cm", "D_", "z", "bias"]
    v = {k: None if s[k] is None else s[k].double().requires_grad_(grad) for k in names}
    h = torch.zeros(B, D, N, dtype=torch.float64, device="cuda") if s.get("state") is None else s["state"].double()
    n = None if s.get("lengths") is None else s["lengths"][:, None, None]
    delta = torch.logaddexp(v["dt"] + v["bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
    rep = D // G
    ys = []
    for t in range(T):
        d = delta[:, t, :, None]
        new = torch.exp(d * v["A"]) * h + d * v["x"][:, t, :, None] * v["Bm"][:, t].repeat_interleave(rep, 1)
        h = new if n is None else torch.where(t < n, new, h)
        ys.append(torch.linalg.vecdot(h, v["Cm"][:, t].repeat_interleave(rep, 1)))
    y = torch.stack(ys, 1) + v["x"] * v["D_"]
    if v["z"] is not None:
        y = y * v["z"] / (1 + torch.exp(-v["z"]))
    if grad:
        want = [k for k in names if v[k] is not None]
        g = dict(zip(want, torch.autograd.grad((y * s["dy"].double()).sum(), [v[k] for k in want])))
        return {"dx": g["x"], "ddt": g["dt"], "dA": g["A"], "dB": g["Bm"], "dC": g["Cm"], "dD": g["D_"],
                "dz": g.get("z"), "ddt_bias": g["bias"], "dstate0": None}
    if n is not None:
        y = y * (torch.arange(T, device="cuda")[None, :, None] < n)
    return [y, None if s.get("state") is None else h]
