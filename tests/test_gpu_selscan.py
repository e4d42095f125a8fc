"""Selective scan and its gradient against 64-bit definitions."""

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def make(B, T, D, N, G=1, dtype=F32, gate=True, skip=True, bias=True, state=True, lengths=None, packed=False, seed=0):
    g = torch.Generator().manual_seed(seed)

    def rows(*inner):
        n = 1
        for v in inner:
            n *= v
        if packed:  # a slice of a wider row that starts at an odd element
            return torch.randn(B, T, 2 * n + 3, generator=g).to(dtype).cuda()[..., 3:n + 3].unflatten(-1, inner)
        return torch.randn(B, T, *inner, generator=g).to(dtype).cuda()

    v = dict(x=rows(D), dt=rows(D), B=rows(G, N), C=rows(G, N))
    v["A"] = -(torch.rand(D, N, generator=g) * 4 + 0.05).cuda()
    v["z"] = rows(D) if gate else None
    v["D"] = torch.randn(D, generator=g).cuda() if skip else None
    v["dt_bias"] = (torch.randn(D, generator=g) - 2).cuda() if bias else None
    v["state"] = torch.randn(B, D, N, generator=g).cuda() if state else None
    v["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return v


def wide(v):
    return {k: ref.d(v[k]) for k in ("x", "dt", "A", "z", "D", "dt_bias")} | {
        "Bm": ref.d(v["B"]), "Cm": ref.d(v["C"]), "h0": ref.d(v["state"]),
        "lengths": None if v["lengths"] is None else v["lengths"].cpu().long()}


def call(sdm, v, **kw):
    return sdm.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                              state=v["state"], lengths=v["lengths"], **kw)


def check(sdm, v, **kw):
    """One call against the definition: T steps of a relative error each, on the terms' absolute values."""
    w = wide(v)
    T, N = v["x"].shape[1], v["A"].shape[1]
    want, h = ref.scan(**w)
    size, hsize = ref.scan(**w, absolute=True)
    rel = (T + 1) * ref.scan_step_error(v["dt"], v["A"], v["dt_bias"])
    zs = 0.0 if v["z"] is None else (6 + 1.2 * w["z"].abs()) * 2 * ref.U
    y = call(sdm, v, **kw)
    live = torch.ones(want.shape[:2], dtype=torch.bool)
    if v["lengths"] is not None:
        live = torch.arange(T)[None] < w["lengths"][:, None]
    bound = (rel + (N + 4) * ref.U + zs) * size
    if v["z"] is not None and float(v["z"].min()) < -87:
        # below -87 exp(z) leaves fp32's normal range; the gate, there below 88 * 2^-126, is 0
        bound = bound + 88 * 2.0 ** -126 * ref.scan(**dict(w, z=None), absolute=True)[0]
    ref.assert_within(y.cpu()[live], want[live], bound[live], "y")
    if v["state"] is not None:
        ref.assert_within(v["state"], h, rel * hsize, "state")
    return y


SIZES = [(1, 1, 1, 1, 1), (2, 1, 8, 16, 1), (3, 2, 5, 3, 1), (2, 4, 6, 7, 2), (1, 5, 130, 16, 1), (2, 15, 12, 8, 3),
         (2, 16, 9, 17, 1), (1, 17, 64, 32, 2), (2, 33, 40, 33, 1), (1, 70, 24, 64, 4), (2, 130, 257, 16, 1)]


@pytest.mark.parametrize("B,T,D,N,G", SIZES)
@pytest.mark.parametrize("dtype,packed", [(F32, False), (BF16, False), (F32, True), (BF16, True)])
def test_values(sdm, B, T, D, N, G, dtype, packed):
    check(sdm, make(B, T, D, N, G, dtype, packed=packed, seed=T))


@pytest.mark.parametrize("N", [4, 16, 24, 64])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_split_token_axis(sdm, N, dtype):
    """Few channels and many tokens: the splits' maps are joined."""
    check(sdm, make(1, 700, 20, N, 2, dtype, seed=N))
    check(sdm, make(3, 513, 10, N, 1, dtype, lengths=[513, 200, 0], seed=N))


@pytest.mark.parametrize("gate,skip,bias,state", [(False, True, True, True), (True, False, False, False),
                                                  (False, False, True, False)])
def test_optional_inputs(sdm, gate, skip, bias, state):
    check(sdm, make(2, 21, 36, 16, gate=gate, skip=skip, bias=bias, state=state))
    check(sdm, make(2, 2, 36, 16, gate=gate, skip=skip, bias=bias, state=state))


def test_without_softplus(sdm):
    v = make(2, 20, 12, 16, state=True)
    v["dt"] = v["dt"].abs() * 0.1
    v["dt_bias"] = None
    w = wide(v)
    want, h = ref.scan(**w, softplus=False)
    size, hsize = ref.scan(**w, softplus=False, absolute=True)
    rel = 21 * ref.scan_step_error(v["dt"], v["A"], None, softplus=False)
    y = call(sdm, v, softplus=False)
    ref.assert_within(y, want, (rel + 40 * ref.U) * size, "y")
    ref.assert_within(v["state"], h, rel * hsize, "state")


@pytest.mark.parametrize("T", [3, 40, 600])
def test_lengths(sdm, T):
    """Rows of no, one and all tokens: later rows of y stay, nothing there is read, a row without tokens keeps its state."""
    lengths = [0, 1, T, T - 1, min(17, T)]
    v = make(5, T, 12, 16, lengths=lengths, seed=T)
    clean = {k: None if t is None else t.clone() for k, t in v.items()}
    for i, n in enumerate(lengths):
        for k in ("x", "dt", "B", "C", "z"):
            v[k][i, n:] = float("nan")
    y = torch.full(v["x"].shape, 3.0, device="cuda")
    before = v["state"].clone()
    call(sdm, v, y=y)
    assert torch.equal(v["state"][0], before[0])
    got = check(sdm, clean)
    for i, n in enumerate(lengths):
        assert bool((y[i, n:] == 3.0).all()) and torch.equal(y[i, :n], got[i, :n])
    assert torch.equal(v["state"], clean["state"])
    sdm.stream_check()


def test_tokens_one_by_one(sdm):
    """Decoding continues a prompt: within the errors of the definition over all tokens."""
    v = make(2, 30, 24, 16, seed=11)
    w = wide(v)
    want, h = ref.scan(**w)
    size, hsize = ref.scan(**w, absolute=True)
    rel = 31 * ref.scan_step_error(v["dt"], v["A"], v["dt_bias"])
    parts, at = [], 0
    for n in (20, 1, 1, 3, 1, 4):
        part = dict(v, **{k: v[k][:, at:at + n] for k in ("x", "dt", "B", "C", "z")})
        parts.append(call(sdm, {k: (t.contiguous() if k in ("x", "dt", "B", "C", "z") else t) for k, t in part.items()}))
        at += n
    zs = (6 + 1.2 * w["z"].abs()) * 2 * ref.U
    ref.assert_within(torch.cat(parts, 1), want, (rel + 20 * ref.U + zs) * size, "y")
    ref.assert_within(v["state"], h, rel * hsize, "state")


def test_far_step_sizes(sdm):
    """Steps of nearly nothing and of everything: decays of 1 and of 0, no overflow on the way."""
    v = make(1, 12, 8, 16, dtype=F32)
    v["dt"][:, ::3] = 60.0
    v["dt"][:, 1::3] = -60.0
    v["z"][:, ::2] = -200.0
    y = check(sdm, v)
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(v["state"]).all())


@pytest.mark.parametrize("N", [4, 16, 24, 64])
@pytest.mark.parametrize("where", ["input", "state"])
def test_infinite_state_outlasts_its_decay(sdm, N, where):
    """An infinite state of one channel stays infinite with its sign over splits whose decay is 0 in fp32, as token by
    token (no token's own decay is 0 here); other channels keep their bits."""
    v = make(1, 700, 20, N, 2, seed=N)
    v["dt_bias"] = v["dt_bias"] + 3  # some 50 of delta a split: e^(-4 * 50) is 0 in fp32
    clean = dict(v, state=v["state"].clone())
    clean_y = call(sdm, clean)
    if where == "input":
        v["x"][0, 60, 5] = float("inf")
    else:
        v["state"][0, 5] = torch.where(torch.arange(N, device="cuda") % 2 == 0, float("inf"), float("-inf"))
    w = wide(v)
    delta = torch.log1p(torch.exp(w["dt"] + w["dt_bias"]))
    assert float((delta[..., None] * w["A"]).min()) > -80 and float((delta[:, 96:144, 5, None] * w["A"][5]).sum(1).min()) < -110
    want, h = ref.scan(**w)
    assert bool(torch.isinf(h[0, 5]).all())
    y = call(sdm, v)
    assert torch.equal(ref.d(v["state"])[0, 5], h[0, 5])
    # which of infinity and not a number y is there is not said: states that pad N make 0 * inf of it
    assert torch.equal(torch.isfinite(ref.d(y)), torch.isfinite(want))
    rest = [c for c in range(20) if c != 5]
    assert torch.equal(y[..., rest], clean_y[..., rest]) and torch.equal(v["state"][:, rest], clean["state"][:, rest])


GRAD_SIZES = [(1, 1, 1, 1, 1), (2, 3, 8, 16, 1), (1, 9, 5, 3, 1), (2, 20, 6, 7, 2), (1, 64, 33, 16, 1),
              (2, 65, 24, 32, 2), (1, 130, 20, 64, 4), (2, 70, 140, 16, 1), (3, 200, 9, 8, 3)]


def gradients(sdm, v, dy, dstate, **kw):
    return sdm.selective_scan_backward(v["x"], v["dt"], v["A"], v["B"], v["C"], dy, D=v["D"], z=v["z"],
                                       dt_bias=v["dt_bias"], state0=v["state"], dstate=dstate, lengths=v["lengths"],
                                       **kw)


def wanted(v, dy, dstate, absolute=False):
    """Gradients in 64 bits; absolute: of the chain of absolute values, which bounds the sums of the terms' sizes."""
    w = wide(v)
    names = [k for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0") if w[k] is not None]
    leaves = [w[k].requires_grad_() for k in names]
    y, h = ref.scan(**w)
    if w["lengths"] is not None:
        y = torch.where((torch.arange(y.shape[1])[None] < w["lengths"][:, None])[..., None], y, 0.0)
    loss = (y * ref.d(dy)).sum() + (0 if dstate is None else (h * ref.d(dstate)).sum())
    to = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
          "h0": "dstate0"}
    return {to[k]: g for k, g in zip(names, torch.autograd.grad(loss, leaves, allow_unused=True))}


def sizes(v, dy, dstate):
    """Sums of the absolute values of every gradient's terms."""
    w = wide(v)
    x, dt, A, Bm, Cm = w["x"], w["dt"], w["A"], w["Bm"], w["Cm"]
    nb, T, nd = x.shape
    G = Bm.shape[2]
    rep = nd // G
    live = torch.ones(nb, T, 1, dtype=torch.float64)
    if w["lengths"] is not None:
        live = (torch.arange(T)[None] < w["lengths"][:, None]).double()[..., None]
    u = dt if w["dt_bias"] is None else dt + w["dt_bias"]
    delta = torch.log1p(torch.exp(u.clamp(max=30))) * live
    e = ref.d(dy).abs() * live
    z = w["z"]
    if z is not None:
        e0, e = e, e * (z * torch.sigmoid(z)).abs()
    h = torch.zeros(nb, nd, A.shape[1]).double() if w["h0"] is None else w["h0"].abs()
    hs, kept = [], []
    Bs, Cs = Bm.abs().repeat_interleave(rep, 2), Cm.abs().repeat_interleave(rep, 2)
    a = torch.exp(delta[..., None] * A)
    for t in range(T):
        kept.append(a[:, t] * h)
        h = kept[-1] + (delta * x.abs())[:, t, :, None] * Bs[:, t]
        hs.append(h)
    q = torch.zeros_like(h) if dstate is None else ref.d(dstate).abs()
    out = {k: torch.zeros(s).double() for k, s in (("dA", A.shape), ("dx", x.shape), ("ddt", x.shape))}
    out["dB"], out["dC"] = torch.zeros(Bm.shape).double(), torch.zeros(Bm.shape).double()
    y = torch.zeros(x.shape).double()
    for t in reversed(range(T)):
        g = Cs[:, t] * e[:, t, :, None] + q
        out["dC"][:, t] = (e[:, t, :, None] * hs[t]).unflatten(1, (G, rep)).sum(2)
        out["dB"][:, t] = (g * (delta * x.abs())[:, t, :, None]).unflatten(1, (G, rep)).sum(2)
        p, r = (g * Bs[:, t]).sum(-1), (g * A.abs() * kept[t]).sum(-1)
        out["dx"][:, t] = delta[:, t] * p + (0 if w["D"] is None else w["D"].abs() * e[:, t])
        out["ddt"][:, t] = (x.abs()[:, t] * p + r) * torch.sigmoid(u[:, t]) * live[:, t]
        out["dA"] += (g * delta[:, t, :, None] * kept[t]).sum(0)
        y[:, t] = (Cs[:, t] * hs[t]).sum(-1) + (0 if w["D"] is None else w["D"].abs() * x.abs()[:, t])
        q = a[:, t] * g
    out["dD"] = (e * x.abs()).sum((0, 1))
    out["ddt_bias"] = out["ddt"].sum((0, 1))
    out["dstate0"] = q
    if z is not None:
        out["dz"] = e0 * y * 1.1
    return out


@pytest.mark.parametrize("B,T,D,N,G", GRAD_SIZES)
@pytest.mark.parametrize("dtype,packed", [(F32, False), (BF16, False), (F32, True)])
def test_gradient(sdm, B, T, D, N, G, dtype, packed):
    lengths = None if B == 1 else [T] + [(7 * i) % (T + 1) for i in range(1, B)]
    v = make(B, T, D, N, G, dtype, lengths=lengths, packed=packed, seed=T)
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(B, T, D, generator=g).to(dtype).cuda()
    ds = torch.randn(B, D, N, generator=g).cuda()
    got = gradients(sdm, v, dy, ds)
    want, size = wanted(v, dy, ds), sizes(v, dy, ds)
    # both recurrences err by a step's error T times each; sums over n, channels and tokens add their roundings, the
    # gates their exponentials'
    zmax = 0.0 if v["z"] is None else float(v["z"].float().abs().max())
    rel = 2 * (T + 2) * ref.scan_step_error(v["dt"], v["A"], v["dt_bias"])
    rel += (N + D + B * T + 40 + 4 * (6 + 1.2 * zmax) * (1 + zmax)) * ref.U
    for k, w in want.items():
        ref.assert_within(got[k], w, rel * size[k], k)
    again = gradients(sdm, v, dy, ds)
    assert all(torch.equal(again[k], got[k]) for k in got if got[k] is not None)
    if lengths is not None:
        for k in ("dx", "ddt", "dB", "dC", "dz"):
            for i, n in enumerate(lengths):
                assert not got[k][i, n:].any(), k


@pytest.mark.parametrize("gate,skip,bias,state", [(False, True, True, False), (True, False, False, False)])
def test_gradient_of_optional_inputs(sdm, gate, skip, bias, state):
    v = make(2, 70, 20, 16, gate=gate, skip=skip, bias=bias, state=state, seed=2)
    dy = torch.randn(2, 70, 20, generator=torch.Generator().manual_seed(3)).cuda()
    got = gradients(sdm, v, dy, None)
    want, size = wanted(v, dy, None), sizes(v, dy, None)
    zmax = 0.0 if not gate else float(v["z"].abs().max())
    rel = 144 * ref.scan_step_error(v["dt"], v["A"], v["dt_bias"]) + (400 + 4 * (6 + 1.2 * zmax) * (1 + zmax)) * ref.U
    for k, w in want.items():
        ref.assert_within(got[k], w, rel * size[k], k)
    assert (got["dz"] is None) == (not gate) and (got["dD"] is None) == (not skip)
    assert (got["ddt_bias"] is None) == (not bias) and got["dstate0"] is None


def test_state_gradient_in_place(sdm):
    """dL/dh0 may be written over dL/dhT."""
    from sparse_memory_linear_pkm_b200 import native

    v = make(2, 200, 20, 16, seed=6)
    g = torch.Generator().manual_seed(7)
    dy, ds = torch.randn(2, 200, 20, generator=g).cuda(), torch.randn(2, 20, 16, generator=g).cuda()
    want = gradients(sdm, v, dy, ds)
    out = {k: torch.empty_like(t) for k, t in want.items() if k != "dstate0"}
    shape = native.SelscanShape(2, 200, 20, 16, 1, native.F32, 1, 0, 0, 0, 0, 0, 0)
    lib = native.load()
    n = lib.sdm_selective_scan_backward_workspace_bytes(shape)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    native.check(lib.sdm_selective_scan_backward(
        shape, *(p(v[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "lengths", "state")), p(dy), p(ds),
        *(p(out[k]) for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")), p(ds), p(ws), n,
        torch.cuda.current_stream().cuda_stream))
    assert torch.equal(ds, want["dstate0"]) and all(torch.equal(out[k], want[k]) for k in out)


def test_gradient_against_differences(sdm):
    v = make(2, 37, 6, 5, 2, seed=4)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(2, 37, 6, generator=g).cuda()
    got = gradients(sdm, v, dy, None)
    w = wide(v)
    to = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
          "h0": "dstate0"}
    way = {k: torch.randn(w[k].shape, generator=g).double() for k in to}

    def loss(t):
        return float((ref.scan(**{k: (w[k] + t * way[k] if k in way else w[k]) for k in w})[0] * ref.d(dy)).sum())

    slope = (loss(1e-6) - loss(-1e-6)) / 2e-6
    parts = [ref.d(got[to[k]]) * way[k] for k in to]
    # 38 steps' errors, and the differences' own
    rel = 80 * ref.scan_step_error(v["dt"], v["A"], v["dt_bias"]) + 1e-6
    assert abs(float(sum(p.sum() for p in parts)) - slope) <= rel * float(sum(p.abs().sum() for p in parts)) * 4


def test_empty(sdm):
    v = make(2, 0, 8, 16)
    before = v["state"].clone()
    assert call(sdm, v).shape == (2, 0, 8) and torch.equal(v["state"], before)
    got = gradients(sdm, v, v["x"], before)
    assert torch.equal(got["dstate0"], before) and not got["dA"].any() and not got["dD"].any()
