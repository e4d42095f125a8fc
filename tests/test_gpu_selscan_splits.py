"""The selective scan where its token axis is split, and its gradient, against
bounds that weight every step's error with the decay that still applies to it
(the CPU tests of the bounds show that they find a broken chain), against the
same sequence in short calls, on streams and in graphs."""

import pytest
import torch

import block_reference as ref
from test_gpu_selscan import BF16, F32, call, gradients, make, sizes, wanted, wide

pytestmark = pytest.mark.gpu
TOKENS = ("x", "dt", "B", "C", "z")


def workspace(v):
    """Bytes that the call takes: none unless the token axis is split."""
    from sparse_memory_linear_pkm_b200 import native

    (B, T, D), G, N = v["x"].shape, v["B"].shape[2], v["A"].shape[1]
    shape = native.SelscanShape(B, T, D, N, G, native.BF16 if v["x"].dtype == BF16 else native.F32, 1, 0, 0, 0, 0, 0, 0)
    return native.load().sdm_selective_scan_workspace_bytes(shape)


def tokens(v, a, b):
    return dict(v, **{k: None if v[k] is None else v[k][:, a:b].contiguous() for k in TOKENS})


SPLIT = [(1, 700, 20, 2, None), (3, 513, 10, 1, [513, 200, 0]), (1, 2500, 136, 1, None), (2, 1301, 65, 1, [77, 1301])]


@pytest.mark.parametrize("N", [4, 16, 24, 64])
@pytest.mark.parametrize("B,T,D,G,lengths", SPLIT)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values(sdm, B, T, D, G, N, lengths, dtype):
    v = make(B, T, D, N, G, dtype, lengths=lengths, seed=N + T)
    assert workspace(v) > 0
    w = wide(v)
    want, h = ref.scan(**w)
    by, bh = ref.scan_errors(**w)
    y = call(sdm, v)
    live = torch.ones(B, T, dtype=torch.bool)
    if lengths is not None:
        live = torch.arange(T)[None] < w["lengths"][:, None]
    ref.assert_within(y.cpu()[live], want[live], by[live], "y")
    ref.assert_within(v["state"], h, bh, "state")


@pytest.mark.parametrize("N", [4, 16, 64])
def test_same_as_short_calls(sdm, N):
    """One split call and calls of 60 tokens, none of them split, that carry the state: both within the bounds of the
    definition, so within twice those of each other."""
    v = make(2, 780, 24, N, 1, seed=N)
    assert workspace(v) > 0
    w = wide(v)
    by, bh = ref.scan_errors(**w)
    short = dict(v, state=v["state"].clone())
    parts = []
    for t in range(0, 780, 60):
        part = tokens(short, t, t + 60)
        assert workspace(part) == 0
        parts.append(call(sdm, part))
    y = call(sdm, v)
    ref.assert_within(y, torch.cat(parts, 1), 2 * by, "y")
    ref.assert_within(v["state"], short["state"], 2 * bh, "state")


def gradient_errors(v, dy, ds):
    """Bounds of the gradients' errors in fp32 (before a bf16 output's rounding), both recurrences' errors weighted by
    the decays that still apply to them, as ref.scan_errors does for the states; `rounded` relative to the sums of the
    terms' absolute values for the sums over states, channels and tokens."""
    w = wide(v)
    x, dt, A, Bm, Cm, z = (w[k] for k in ("x", "dt", "A", "Bm", "Cm", "z"))
    nb, T, nd = x.shape
    G, N, U = Bm.shape[2], A.shape[1], ref.U
    rep = nd // G
    live = torch.ones(nb, T, 1).double()
    if w["lengths"] is not None:
        live = (torch.arange(T)[None] < w["lengths"][:, None]).double()[..., None]
    u = dt + w["dt_bias"]
    delta = torch.log1p(torch.exp(u)) * live
    r = 2.0 ** -21 + 2.0 ** -22 * u.abs()                        # of delta
    sr = 2.0 ** -21 + r * delta + 4 * U * (u.abs() + delta)      # of sigmoid(u) = exp(u - delta)
    er = ((6 + 1.2 * z.abs()) * 2 + 1) * U                       # of e = dy silu(z)
    zr = 4 * (6 + 1.2 * z.abs()) * (1 + z.abs()) * U             # of dy silu'(z), relative to 1.1 dy
    rounded = (N + nd + nb * T + 40) * U
    e0 = ref.d(dy).abs() * live
    e = e0 * (z * torch.sigmoid(z)).abs()
    Bs, Cs = Bm.abs().repeat_interleave(rep, 2), Cm.abs().repeat_interleave(rep, 2)
    dA = delta[..., None] * A.abs()
    a = torch.exp(-dA)
    ar = 2.0 ** -22 + 4 * U + dA * (r[..., None] + (T + 8) * U)  # of a decay, with the state's roundings
    h, err = w["h0"].abs(), torch.zeros_like(w["h0"])
    hs, es, ks, kes = [], [], [], []
    for t in range(T):
        ks.append(a[:, t] * h)
        kes.append(a[:, t] * err + ar[:, t] * ks[-1])
        term = (delta * x.abs())[:, t, :, None] * Bs[:, t]
        h, err = ks[-1] + term, kes[-1] + (r[:, t, :, None] + 4 * U) * term
        hs.append(h)
        es.append(err)
    q = torch.zeros_like(h) if ds is None else ref.d(ds).abs()
    qe = torch.zeros_like(q)
    zeros = lambda t: torch.zeros(t.shape).double()  # noqa: E731
    out = {"dx": zeros(x), "ddt": zeros(x), "dz": zeros(x), "dB": zeros(Bm), "dC": zeros(Bm), "dA": zeros(A)}
    over = lambda m: m.unflatten(1, (G, rep)).sum(2)  # noqa: E731
    D, bias_sum = w["D"].abs(), zeros(x)
    for t in reversed(range(T)):
        et, d1, x1 = e[:, t, :, None], delta[:, t], x.abs()[:, t]
        first = Cs[:, t] * et
        g, ge = first + q, qe + (er[:, t, :, None] + 3 * U) * first
        out["dC"][:, t] = over(et * es[t] + (er[:, t, :, None] + rounded) * et * hs[t])
        wt = (d1 * x1)[..., None]
        out["dB"][:, t] = over(ge * wt + (r[:, t, :, None] + 4 * U + rounded) * g * wt)
        p, pe = (g * Bs[:, t]).sum(-1), (ge * Bs[:, t]).sum(-1)
        rr, re = (g * A.abs() * ks[t]).sum(-1), ((ge * ks[t] + g * kes[t]) * A.abs()).sum(-1)
        skip = D * e[:, t]
        out["dx"][:, t] = d1 * pe + (r[:, t] + rounded) * d1 * p + (er[:, t] + rounded) * skip
        sig = torch.sigmoid(u[:, t]) * live[:, t]
        bias_sum[:, t] = sig * (x1 * p + rr)
        out["ddt"][:, t] = sig * (x1 * pe + re) + (sr[:, t] + rounded) * bias_sum[:, t]
        out["dA"] += (d1[..., None] * (ge * ks[t] + g * kes[t] + (r[:, t, :, None] + rounded) * g * ks[t])).sum(0)
        y = (Cs[:, t] * hs[t]).sum(-1) + D * x1
        out["dz"][:, t] = 1.1 * e0[:, t] * ((Cs[:, t] * es[t]).sum(-1) + (rounded + zr[:, t]) * y)
        q, qe = a[:, t] * g, a[:, t] * ge + ar[:, t] * a[:, t] * g
    out["dD"] = ((er + rounded) * e * x.abs()).sum((0, 1))
    out["ddt_bias"] = (out["ddt"] + rounded * bias_sum).sum((0, 1))
    out["dstate0"] = qe
    return out


@pytest.mark.parametrize("N", [8, 16, 24, 64])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,G,lengths", [(1, 700, 20, 2, None), (2, 400, 36, 1, [400, 130])])
def test_gradient(sdm, B, T, D, G, N, lengths, dtype):
    v = make(B, T, D, N, G, dtype, lengths=lengths, seed=N)
    g = torch.Generator().manual_seed(1)
    dy, ds = torch.randn(B, T, D, generator=g).to(dtype).cuda(), torch.randn(B, D, N, generator=g).cuda()
    got, want, bound, size = gradients(sdm, v, dy, ds), wanted(v, dy, ds), gradient_errors(v, dy, ds), sizes(v, dy, ds)
    for k, w in want.items():
        assert float((bound[k].sum() / size[k].sum())) < 1e-3, k  # far below what a broken chain makes
        ref.assert_within(got[k], w, bound[k], k)


def test_gradient_in_parts(sdm):
    """The gradient of a sequence in one call, and in calls of 30 tokens (one split each) that hand dL/dh on."""
    v = make(2, 600, 20, 16, 1, seed=3)
    g = torch.Generator().manual_seed(4)
    dy, ds = torch.randn(2, 600, 20, generator=g).cuda(), torch.randn(2, 20, 16, generator=g).cuda()
    whole = gradients(sdm, v, dy, ds)
    starts, state = [], v["state"].clone()
    for t in range(0, 600, 30):
        starts.append(state.clone())
        call(sdm, dict(tokens(v, t, t + 30), state=state))
    parts, d = [], ds
    for t in reversed(range(0, 600, 30)):
        parts.append(gradients(sdm, dict(tokens(v, t, t + 30), state=starts[t // 30]), dy[:, t:t + 30].contiguous(), d))
        d = parts[-1]["dstate0"]
    parts.reverse()
    bound = gradient_errors(v, dy, ds)  # of either side
    for k in ("dx", "ddt", "dB", "dC", "dz"):
        ref.assert_within(whole[k], torch.cat([p[k] for p in parts], 1), 2 * bound[k], k)
    for k in ("dA", "dD", "ddt_bias"):
        ref.assert_within(whole[k], torch.stack([p[k].double() for p in parts]).sum(0), 2 * bound[k], k)
    ref.assert_within(whole["dstate0"], d, 2 * bound["dstate0"], "dstate0")


def all_of(sdm, v, dy):
    state = v["state"].clone()
    y = call(sdm, dict(v, state=state))
    q = gradients(sdm, v, dy, None)
    return [y, state] + [q[k] for k in sorted(q)]


def test_split_calls_on_two_streams(sdm):
    vs = [make(1, 700, 24, 16, seed=i) for i in range(2)]
    dys = [torch.randn(1, 700, 24, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    assert workspace(vs[0]) > 0
    alone = [all_of(sdm, v, dy) for v, dy in zip(vs, dys)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = all_of(sdm, vs[k], dys[k])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_split_calls_in_two_graphs(sdm):
    """Two captured calls replayed on two streams at once, on new inputs: each has its own scratch."""
    vs = [make(1, 700, 24, 16, seed=i) for i in range(2)]
    dys = [torch.randn(1, 700, 24, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    for v, dy in zip(vs, dys):
        all_of(sdm, v, dy)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for v, dy in zip(vs, dys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(all_of(sdm, v, dy))
    for v in vs:
        for k in TOKENS:
            v[k].mul_(0.5).add_(0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for v, dy, got in zip(vs, dys, outs):
        assert all(torch.equal(x, y) for x, y in zip(got, all_of(sdm, v, dy)))
    sdm.stream_check()
