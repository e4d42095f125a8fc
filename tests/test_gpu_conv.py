"""Short causal convolution and its gradient against 64-bit definitions."""

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def make(B, T, D, K, dtype=BF16, wtype=F32, bias=True, state=True, lengths=None, packed=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, 3 * D + 1 if packed else D, generator=g).to(dtype).cuda()
    if packed:  # starts at an odd element: not on any unit's boundary
        x = x[..., 1:D + 1]
    w = (torch.randn(D, K, generator=g) / K ** 0.5).to(wtype).cuda()
    b = torch.randn(D, generator=g).to(wtype).cuda() if bias else None
    s = torch.randn(B, K - 1, D, generator=g).to(dtype).cuda() if state else None
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return x, w, b, s, n


def bound(y, u, size, K, silu):
    """u: K + 1 roundings of its terms; SiLU's slope is at most 1.1, its exponential is off by (2 + 1.2 |u|) units in
    the last place, its division by two."""
    b = (K + 1) * ref.U * size
    return 1.1 * b + (6 + 1.2 * u.abs()) * 2 * ref.U * y.abs() if silu else b


CASES = [(1, 1, 1, 2), (2, 1, 8, 4), (3, 2, 5, 3), (2, 3, 64, 4), (1, 8, 12, 8), (2, 9, 33, 5), (2, 17, 40, 4),
         (1, 65, 128, 4), (3, 130, 36, 2), (2, 300, 260, 4)]


@pytest.mark.parametrize("B,T,D,K", CASES)
@pytest.mark.parametrize("dtype,silu,packed", [(BF16, True, False), (F32, True, True), (F32, False, False),
                                               (BF16, False, True)])
def test_values(sdm, B, T, D, K, dtype, silu, packed):
    x, w, b, s, _ = make(B, T, D, K, dtype, packed=packed, seed=T, wtype=BF16 if D % 2 else F32)
    want, after, size, u = ref.conv(x, w, b, silu, s)
    y = sdm.short_conv(x, w, b, silu=silu, state=s)
    assert y.dtype == dtype and y.is_contiguous()
    ref.assert_within(y, want, bound(want, u, size, K, silu), "y")
    assert torch.equal(ref.d(s), after)
    want, _, size, u = ref.conv(x, w, None, silu)
    ref.assert_within(sdm.short_conv(x, w, silu=silu), want, bound(want, u, size, K, silu), "y without state")


@pytest.mark.parametrize("K", [2, 4, 8])
def test_lengths(sdm, K):
    """Rows of 0, 1 and all tokens: y behind a row's end stays, what is there is not read, the state is the row's own."""
    lengths = [0, 1, 37, 40, K - 1, 16]
    x, w, b, s, n = make(6, 40, 24, K, F32, lengths=lengths, seed=K)
    for i, v in enumerate(lengths):
        x[i, v:] = float("nan")
    y = torch.full((6, 40, 24), 7.0, device="cuda")
    clean = torch.nan_to_num(x, nan=0.0)
    want, after, size, u = ref.conv(clean, w, b, True, s, lengths)
    sdm.short_conv(x, w, b, state=s, lengths=n, y=y)
    for i, v in enumerate(lengths):
        assert bool((y[i, v:] == 7.0).all())
        ref.assert_within(y[i, :v], want[i, :v], bound(want, u, size, K, True)[i, :v], f"row {i}")
    assert torch.equal(ref.d(s), after)
    sdm.stream_check()


def test_consecutive_calls_continue_one_sequence(sdm):
    """Any cut into calls, single tokens among them, gives the whole call's bits."""
    x, w, b, s, _ = make(2, 50, 20, 4, BF16, seed=3)
    whole_s = s.clone()
    whole = sdm.short_conv(x, w, b, state=whole_s)
    at, parts = 0, []
    for n in (1, 1, 2, 17, 1, 9, 19):
        parts.append(sdm.short_conv(x[:, at:at + n].contiguous(), w, b, state=s))
        at += n
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s, whole_s)


def test_lengths_out_of_range_are_reported(sdm):
    x, w, b, s, _ = make(2, 5, 8, 4, F32)
    n = torch.tensor([9, -3], dtype=torch.int32, device="cuda")
    y = sdm.short_conv(x, w, b, state=s, lengths=n)
    with pytest.raises(sdm.SdmError, match="SDM_ERR_DEVICE_FAULT"):
        sdm.stream_check()
    assert bool(torch.isfinite(y).all())
    sdm.stream_check()


@pytest.mark.parametrize("B,T,D,K", CASES + [(9, 70, 8, 4)])
@pytest.mark.parametrize("dtype,silu,packed", [(BF16, True, False), (F32, True, True), (F32, False, False)])
def test_gradient(sdm, B, T, D, K, dtype, silu, packed):
    lengths = None if B < 2 else [T] + [(3 * i) % (T + 1) for i in range(1, B)]
    x, w, b, s, n = make(B, T, D, K, dtype, lengths=lengths, packed=packed, seed=T + 1)
    g = torch.Generator().manual_seed(2)
    dy = torch.randn(B, T, D, generator=g).to(dtype).cuda()
    ds = torch.randn(B, K - 1, D, generator=g).to(dtype).cuda()
    got = sdm.short_conv_backward(x, w, dy, b, silu=silu, state0=s, dstate=ds, lengths=n)

    leaves = [ref.d(t).requires_grad_() for t in (x, w, b, s)]
    xx, ww, bb, ss = leaves
    full = torch.cat([ss, xx], 1)
    u = sum(full[:, k:k + T] * ww[:, k] for k in range(K)) + bb
    y = u * torch.sigmoid(u) if silu else u
    ends = [T] * B if lengths is None else lengths
    live = torch.stack([torch.arange(T) < v for v in ends])[..., None]
    after = torch.stack([full[i, v:v + K - 1] for i, v in enumerate(ends)])
    loss = torch.where(live, y * ref.d(dy), 0.0).sum() + (after * ref.d(ds)).sum()
    want = dict(zip(("dx", "dw", "dbias", "dstate0"), torch.autograd.grad(loss, leaves)))
    # du: SiLU's slope is off by its exponential's and division's units and u's roundings (its own slope <= 0.5)
    size = sum((full[:, k:k + T] * ww[:, k]).abs() for k in range(K)) + bb.abs()
    du = (ref.d(dy).abs() * live * 1.1).detach()
    ddu = du * ((14 + 2.4 * u.abs()) * 2 * ref.U * (1 + u.abs()) + (K + 1) * ref.U * size) if silu else du * 0
    ddu, size = ddu.detach(), None
    pad = lambda t: torch.cat([torch.zeros(B, K - 1, D).double(), t, torch.zeros(B, K - 1, D).double()], 1)  # noqa: E731
    # extended rows p = -(K-1) .. T-1: sum over k of w[k] du[p + K - 1 - k]
    spread = lambda t: sum((pad(t)[:, K - 1 - k:2 * K - 2 - k + T + K - 1 - (K - 1)] * ww.detach()[:, k].abs())  # noqa: E731
                           for k in range(K))
    ext = spread(ddu) + (K + 2) * ref.U * (spread(du) + 6.0)
    ref.assert_within(got["dstate0"], want["dstate0"], ext[:, :K - 1], "dstate0")
    ref.assert_within(got["dx"], want["dx"], ext[:, K - 1:], "dx")
    # sums of 64 tokens in a thread, 8 threads, then the blocks
    adds = (64 + 8 + B * T / 512 + 8 + 4) * ref.U
    ref.assert_within(got["dbias"], want["dbias"], (ddu + adds * du).sum((0, 1)), "dbias")
    dw = torch.stack([((ddu + adds * du) * full.detach()[:, k:k + T].abs()).sum((0, 1)) for k in range(K)], -1)
    ref.assert_within(got["dw"], want["dw"], dw, "dw")
    again = sdm.short_conv_backward(x, w, dy, b, silu=silu, state0=s, dstate=ds, lengths=n)
    assert all(torch.equal(again[k], got[k]) for k in got)
    for i, v in enumerate(ends):
        assert not got["dx"][i, max(v, 0):].any()


def test_gradient_against_differences(sdm):
    x, w, b, s, _ = make(2, 11, 6, 4, F32, seed=5)
    g = torch.Generator().manual_seed(6)
    dy = torch.randn(2, 11, 6, generator=g).cuda()
    got = sdm.short_conv_backward(x, w, dy, b, state0=s)
    v = {k: torch.randn(t.shape, generator=g).double() for k, t in (("dx", x), ("dw", w), ("dbias", b), ("dstate0", s))}

    def loss(t):
        y = ref.conv(ref.d(x) + t * v["dx"], ref.d(w) + t * v["dw"], ref.d(b) + t * v["dbias"], True,
                     ref.d(s) + t * v["dstate0"])[0]
        return float((y * ref.d(dy)).sum())

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    parts = [(ref.d(got[k]) * v[k]) for k in v]
    assert abs(float(sum(p.sum() for p in parts)) - slope) <= 2e-5 * float(sum(p.abs().sum() for p in parts))


def test_empty(sdm):
    x, w, b, s, _ = make(2, 0, 8, 4, F32)
    before = s.clone()
    assert sdm.short_conv(x, w, b, state=s).shape == (2, 0, 8) and torch.equal(s, before)
    got = sdm.short_conv_backward(x, w, x, b, state0=s, dstate=s)
    assert not got["dw"].any() and not got["dbias"].any() and torch.equal(got["dstate0"], s)


@pytest.mark.parametrize("K", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("dtype,D", [(BF16, 6), (F32, 5)])
def test_infinite_values_stay_in_their_window(sdm, K, dtype, D):
    """An infinite input reaches the K outputs that depend on it, an infinite dy the K inputs it depends on, and an
    infinite last input of a row no tap's gradient but the last one's: all others keep their bits."""
    x, w, b, _, n = make(2, 90, D, K, dtype, state=False, lengths=[90, 70], seed=K)
    dy = torch.randn(2, 90, D, generator=torch.Generator().manual_seed(K + 50)).to(dtype).cuda()
    at = 63  # its window crosses the runs of tokens
    bad = x.clone()
    bad[0, at] = float("inf")
    bad[1, 69] = float("inf")
    clean_y, y = sdm.short_conv(x, w, b, lengths=n), sdm.short_conv(bad, w, b, lengths=n)
    assert torch.equal(y[0, :at], clean_y[0, :at]) and torch.equal(y[0, at + K:], clean_y[0, at + K:])
    assert torch.equal(y[1, :69], clean_y[1, :69]) and torch.equal(y[1, 70:], clean_y[1, 70:])

    bad_dy = dy.clone()
    bad_dy[0, at] = float("inf")
    clean = sdm.short_conv_backward(x, w, dy, b, silu=False, lengths=n)
    dx = sdm.short_conv_backward(x, w, bad_dy, b, silu=False, lengths=n)["dx"]
    assert torch.equal(dx[0, :at - K + 1], clean["dx"][0, :at - K + 1])
    assert torch.equal(dx[0, at + 1:], clean["dx"][0, at + 1:]) and torch.equal(dx[1], clean["dx"][1])

    bad = x.clone()
    bad[1, 69] = float("inf")
    got = sdm.short_conv_backward(bad, w, dy, b, silu=False, lengths=n)
    assert torch.equal(got["dw"][:, :K - 1], clean["dw"][:, :K - 1]) and not got["dw"][:, K - 1].isfinite().any()
    assert torch.equal(got["dx"], clean["dx"]) and torch.equal(got["dbias"], clean["dbias"])
    sdm.stream_check()
