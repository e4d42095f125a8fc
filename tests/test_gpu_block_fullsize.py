"""The operators around the recurrent core at the ends of their ranges and in
the launch shapes that large calls take."""

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
F32, BF16 = torch.float32, torch.bfloat16


def small_integers(n: int) -> torch.Tensor:
    """n values 1 .. 8 in bf16, of a fixed seed, made on the device in parts."""
    g = torch.Generator(device="cuda").manual_seed(1)
    out = torch.empty(n, dtype=BF16, device="cuda")
    for part in out.split(1 << 28):
        part.copy_(torch.randint(1, 9, part.shape, generator=g, device="cuda", dtype=torch.int8))
    return out


def test_longest_sequence_of_the_scan(sdm):
    """The most tokens that a call takes, one channel: the last split's end, rounded up to whole tiles, lies above
    2^31. With steps of 1 and A = -60 nothing outlasts its token (e^-60 of it is left), so y is x, exactly."""
    T = 2 ** 31 - 1 - 4096
    x, one = small_integers(T).view(1, T, 1), torch.ones(T, dtype=BF16, device="cuda")
    state = torch.zeros(1, 1, 1, device="cuda")
    y = torch.zeros_like(x)
    sdm.selective_scan(x, one.view(1, T, 1), torch.full((1, 1), -60.0, device="cuda"), one.view(1, T, 1, 1),
                       one.view(1, T, 1, 1), softplus=False, state=state, y=y)
    assert torch.equal(y, x)
    assert float(state) == float(x[0, -1, 0])
    sdm.stream_check()


@pytest.mark.parametrize("K", [2, 8])
def test_longest_sequence_of_the_convolution(sdm, K):
    """The most tokens that a call takes: the last run's end lies above 2^31. The last tap alone gives y = x, the first
    alone the input K - 1 tokens before."""
    T = 2 ** 31 - 17
    x = small_integers(T).view(1, T, 1)
    state = torch.full((1, K - 1, 1), 9.0, dtype=BF16, device="cuda")
    y = torch.zeros_like(x)
    w = torch.zeros(1, K, device="cuda")
    w[0, K - 1] = 1.0
    sdm.short_conv(x, w, silu=False, state=state, y=y)
    assert torch.equal(y, x) and torch.equal(state, x[:, T - K + 1:])
    state.fill_(9.0)
    sdm.short_conv(x, w.flip(1).contiguous(), silu=False, state=state, y=y)
    assert torch.equal(y[:, K - 1:], x[:, :T - K + 1]) and bool((y[:, :K - 1] == 9.0).all())
    sdm.stream_check()


def rows(n, d, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, d, generator=g, device="cuda") * scale).to(dtype)


# Rows enough that every block of the launch takes several, and calls of so few that each takes one: a row's result does
# not depend on its block, so that all bits agree (the small calls' are held to the definitions elsewhere).
NORM = [(700_000, 24), (130_000, 500), (40_000, 512), (20_000, 1000), (12_000, 2044), (16_500, 2048), (4_000, 8192)]


@pytest.mark.parametrize("n,d", NORM)
@pytest.mark.parametrize("x,res", [(BF16, BF16), (BF16, F32), (F32, None)])
def test_norm_of_many_rows(sdm, n, d, x, res):
    xs, w = rows(n, d, x, 1), (rows(1, d, F32, 2)[0].abs() + 0.5)
    r = None if res is None else rows(n, d, res, 3, 3.0)
    xs[n // 3] = 0
    xs[n // 2] = float("nan")
    for out in ["same", "fp8blk", "fp8row"] if d % 16 == 0 else ["same"]:
        y, h = sdm.rmsnorm_residual(xs, w, r, out=out)
        few = max(1, 40_000 // d)
        for a in sorted({0, few, n // 3 - 1, n // 2 - 1, n - 2 * few, n - few} | set(range(0, n - few, n // 16))):
            part = slice(a, a + few)
            py, ph = sdm.rmsnorm_residual(xs[part].clone(), w, None if r is None else r[part].clone(), out=out)
            if out == "same":
                assert torch.equal(torch.nan_to_num(y[part]), torch.nan_to_num(py))
                assert torch.equal(torch.isnan(y[part]), torch.isnan(py))
            elif out == "fp8blk":
                m = py.numel() * 16 // 17
                assert torch.equal(y[a * d:a * d + m], py[:m])
                assert torch.equal(y[n * d + a * d // 16:n * d + (a * d + m) // 16], py[m:])
            else:
                assert torch.equal(y[0][part].view(torch.uint8), py[0].view(torch.uint8))
                assert torch.equal(y[1][part], py[1])
            if r is not None:
                assert torch.equal(torch.nan_to_num(h[part]), torch.nan_to_num(ph))


@pytest.mark.parametrize("n,d", [(200_000, 24), (20_000, 500), (9_001, 1000), (6_000, 2044), (9_000, 2048), (2_500, 8192)])
@pytest.mark.parametrize("h,dy,with_dh", [(BF16, BF16, True), (F32, F32, True), (BF16, F32, False), (F32, BF16, True)])
def test_norm_gradient_of_many_rows(sdm, n, d, h, dy, with_dh):
    hs, w, dys = rows(n, d, h, 1, 2.0), rows(1, d, F32, 2)[0].abs() + 0.5, rows(n, d, dy, 3)
    dh = rows(n, d, h, 4) if with_dh else None
    dx, dw = sdm.rmsnorm_residual_backward(hs, w, dys, dh)
    few = max(1, 40_000 // d)
    for a in sorted({0, few, n - 2 * few, n - few} | set(range(0, n - few, n // 16))):
        part = slice(a, a + few)
        pdx, _ = sdm.rmsnorm_residual_backward(hs[part].clone(), w, dys[part].clone(),
                                               None if dh is None else dh[part].clone())
        assert torch.equal(dx[part], pdx)
    want, size = torch.zeros(d, device="cuda").double(), torch.zeros(d, device="cuda").double()
    for a in range(0, n, 2000):
        f = hs[a:a + 2000].double()
        t = dys[a:a + 2000].double() * f / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6)
        want, size = want + t.sum(0), size + t.abs().sum(0)
    # a row's s (24 roundings), a thread's rows one after the other, its slots by 32, then a tree
    adds = n / 148 + 24 + 40 + 32
    assert bool(((dw.double() - want).abs() <= adds * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("B,T,D,K", [(10, 200, 1024, 4), (20, 333, 1024, 4), (40, 600, 1026, 4), (70, 130, 1001, 8),
                                     (33, 1000, 512, 2), (50, 500, 513, 5)])
@pytest.mark.parametrize("dtype,packed", [(BF16, False), (F32, True)])
def test_convolution_in_long_runs(sdm, B, T, D, K, dtype, packed):
    """Threads enough that each takes a run of 16, 32 or 64 tokens, against single sequences, which are walked in runs
    of 8: all bits agree, the states' too."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(B, T, 2 * D + 1 if packed else D, generator=g, device="cuda").to(dtype)
    x = x[..., 1:D + 1] if packed else x
    w, b = torch.randn(D, K, generator=g, device="cuda") / K, torch.randn(D, generator=g, device="cuda")
    state = torch.randn(B, K - 1, D, generator=g, device="cuda").to(dtype)
    lengths = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lengths[:4] = torch.tensor([T, 0, K - 2, T - 1], dtype=torch.int32)
    before = state.clone()
    y = torch.full((B, T, D), 3.0, dtype=dtype, device="cuda")
    sdm.short_conv(x, w, b, state=state, lengths=lengths, y=y)
    for i in range(B):
        s = before[i:i + 1].clone()
        one = torch.full((1, T, D), 3.0, dtype=dtype, device="cuda")
        sdm.short_conv(x[i:i + 1], w, b, state=s, lengths=lengths[i:i + 1], y=one)
        assert torch.equal(one, y[i:i + 1]) and torch.equal(s, state[i:i + 1])
    sdm.stream_check()


@pytest.mark.parametrize("dtype,out", [(F32, None), (BF16, None), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("shift", [0, 1])
def test_clipping_of_long_tensors(sdm, dtype, out, shift):
    """Chunks of many accesses a thread, whole and ragged ones, on and off 16-byte boundaries."""
    sizes = [30_000_001, 777, 0, 5_000_000, 2 ** 21, 65_537]
    bases = [rows(1, n + 1, dtype, n % 97)[0] for n in sizes]
    grads = [t[shift:n + shift] for t, n in zip(bases, sizes)]
    outs = None if out is None else [torch.empty(n + 1, dtype=out, device="cuda")[shift:n + shift] for n in sizes]
    before, beside = [g.clone() for g in grads], [t[0 if shift else n].clone() for t, n in zip(bases, sizes)]
    n = sum(float((g.double() ** 2).sum()) for g in before) ** 0.5
    norm = sdm.grad_norm_clip(grads, 3.0, out=outs)
    assert abs(float(norm) - n) <= 6 * 2.0 ** -24 * n  # as for short lists: sums beyond eight values have 64 bits
    c = 3.0 / (n + 1e-6)
    eps = 2.0 ** -24 if (out or dtype) == F32 else 2.0 ** -8
    for b, o in zip(before, grads if outs is None else outs):
        want = b.double() * c
        assert bool(((o.double() - want).abs() <= (9 * 2.0 ** -24 + eps) * want.abs()).all())
    for t, b, size in zip(bases, beside, sizes):  # what lies next to a tensor stays
        assert torch.equal(t[0 if shift else size], b)


@pytest.mark.parametrize("N,G", [(16, 1), (16, 4), (24, 1), (64, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_in_one_pass_over_a_full_device(sdm, N, G, dtype):
    """Channels enough that the token axis is not split, and more than one wave of blocks, against short calls of single
    sequences, which are not split either: the same arithmetic, so the same bits, whichever way the tokens are cut."""
    B, T, D = 20, 300, 4096
    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, dt, z, Bm, Cm = r(B, T, D), r(B, T, D), r(B, T, D), r(B, T, G, N), r(B, T, G, N)
    A = -(torch.rand(D, N, generator=g, device="cuda") * 4 + 0.05)
    bias, skip = torch.randn(D, generator=g, device="cuda") - 2, torch.randn(D, generator=g, device="cuda")
    state = torch.randn(B, D, N, generator=g, device="cuda")
    lengths = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lengths[:2] = torch.tensor([T, 0], dtype=torch.int32)
    before = state.clone()
    y = sdm.selective_scan(x, dt, A, Bm, Cm, D=skip, z=z, dt_bias=bias, state=state, lengths=lengths)
    for i in (0, 1, 2, 11, 19):
        s, n = before[i:i + 1].clone(), int(lengths[i])
        for a in range(0, n, 60):
            part = lambda t: t[i:i + 1, a:min(a + 60, n)].contiguous()  # noqa: E731
            got = sdm.selective_scan(part(x), part(dt), A, part(Bm), part(Cm), D=skip, z=part(z), dt_bias=bias, state=s)
            assert torch.equal(got[0], y[i, a:min(a + 60, n)])
        assert torch.equal(s, state[i:i + 1]) and not y[i, n:].any()
    sdm.stream_check()
