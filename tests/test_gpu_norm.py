"""RMS norm with the residual's addition, its 8-bit outputs and its gradient
against 64-bit definitions."""

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# The sum of squares is a thread's 16 squares, then a tree and at most 16 warps'
# sums: 16 + 5 + 16 roundings, halved by the square root; the root, the division
# and two products add five.
NORM_REL = (37 / 2 + 5) * ref.U


def make(rows, d, x=BF16, res=BF16, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    xs = (torch.randn(rows, d, generator=g) * scale).to(x).cuda()
    r = None if res is None else (torch.randn(rows, d, generator=g) * 3 * scale).to(res).cuda()
    w = (torch.rand(d, generator=g) + 0.5).cuda()
    return xs, w, r


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (5, 8), (2, 16), (33, 24), (7, 100), (9, 128), (4, 510), (5, 512),
                                    (3, 513), (2, 1024), (3, 1000), (2, 2047), (65, 2048), (2, 8191), (1, 8192)])
@pytest.mark.parametrize("x,res,out", [(BF16, BF16, "same"), (BF16, F32, "bf16"), (F32, F32, "same"),
                                       (F32, BF16, "f32"), (BF16, None, "f32"), (F32, None, "bf16")])
def test_values(sdm, rows, d, x, res, out):
    xs, w, r = make(rows, d, x, res, seed=d)
    y, h = sdm.rmsnorm_residual(xs, w, r, out=out, eps=1e-6)
    want, wh = ref.norm(xs, w, r, 1e-6)
    assert y.dtype == (x if out == "same" else {"f32": F32, "bf16": BF16}[out])
    ref.assert_within(y, want, NORM_REL * want.abs(), "y")
    if res is None:
        assert h is None
    else:
        assert h.dtype == res and torch.equal(ref.d(h), wh)


@pytest.mark.parametrize("rows,d", [(1, 16), (5, 32), (9, 256), (3, 528), (17, 2048), (2, 8192)])
@pytest.mark.parametrize("x,res", [(BF16, BF16), (F32, F32), (F32, None), (BF16, None)])
def test_codes_are_those_of_the_real_values(sdm, rows, d, x, res):
    """Codes, exponents and scales equal the 64-bit definition's bit for bit."""
    xs, w, r = make(rows, d, x, res, seed=rows)
    want, wh = ref.norm(xs, w, r, 1e-6)
    buf, h = sdm.rmsnorm_residual(xs, w, r, out="fp8blk", eps=1e-6)
    codes, exps = ref.fp8blk(want)
    n = rows * d
    assert torch.equal(buf[:n].cpu().reshape(rows, d), codes)
    assert torch.equal(buf[n:].cpu().view(torch.int8), exps)
    if res is not None:
        assert torch.equal(ref.d(h), wh)
    (got, scales), _ = sdm.rmsnorm_residual(xs, w, r, out="fp8row", eps=1e-6)
    codes, c = ref.fp8row(want)
    assert torch.equal(got.view(torch.uint8).cpu(), codes)
    assert torch.equal(scales.cpu(), c)


def test_codes_of_odd_rows(sdm):
    """Rows of zeros, of one value, of tiny and huge values, and blocks next to the exponent's border."""
    d = 64
    x = torch.randn(9, d, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1] = 0
    x[1, 5] = 3.0
    x[2] *= 1e-30
    x[3] *= 1e25
    x[4] = torch.linspace(-1, 1, d)
    x[5, :16] = 0
    x[6] = 1.0
    x[7, ::2] = 0.0
    x[8] *= 1e-4
    w = torch.ones(d)
    w[16:32] = 1e-6
    w[32:40] = 0.0
    x, w = x.cuda(), w.cuda()
    want, _ = ref.norm(x, w, None, 1e-6)
    buf, _ = sdm.rmsnorm_residual(x, w, None, out="fp8blk")
    codes, exps = ref.fp8blk(want)
    strip = lambda c: torch.where(c == 128, 0, c)  # noqa: E731  (the sign of a zero is not kept by every rounding)
    assert torch.equal(buf[9 * d:].cpu().view(torch.int8), exps)
    assert torch.equal(strip(buf[:9 * d].cpu().reshape(9, d)), strip(codes))
    (got, scales), _ = sdm.rmsnorm_residual(x, w, None, out="fp8row")
    codes, c = ref.fp8row(want)
    assert torch.equal(scales.cpu(), c)
    assert torch.equal(strip(got.view(torch.uint8).cpu()), strip(codes))


@pytest.mark.parametrize("d", [64, 2048])
@pytest.mark.parametrize("scale,w_scale,eps", [(1e-38, 0.01, 0.0), (1e-30, 1e-12, 0.0), (1e-25, 1e-16, 1e-55),
                                               (1e-42, 1.0, 0.0), (1e-20, 1e-22, 1e-44)])
def test_codes_of_products_below_the_normal_range(sdm, d, scale, w_scale, eps):
    """h w leaves fp32's normal range and a large s brings it back: the codes are still those of the real values."""
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(40, d, generator=g).double() * scale).float().cuda()
    w = ((torch.rand(d, generator=g).double() + 0.5) * w_scale).float().cuda()
    eps = float(torch.tensor(eps, dtype=torch.float32))  # as the call takes it
    want, _ = ref.norm(x, w, None, eps)
    strip = lambda c: torch.where(c == 128, 0, c)  # noqa: E731  (the sign of a zero is not kept by every rounding)
    buf, _ = sdm.rmsnorm_residual(x, w, None, out="fp8blk", eps=eps)
    codes, exps = ref.fp8blk(want)
    assert torch.equal(buf[40 * d:].cpu().view(torch.int8), exps)
    assert torch.equal(strip(buf[:40 * d].cpu().reshape(40, d)), strip(codes))
    (got, scales), _ = sdm.rmsnorm_residual(x, w, None, out="fp8row", eps=eps)
    codes, c = ref.fp8row(want)
    assert torch.equal(scales.cpu(), c)
    assert torch.equal(strip(got.view(torch.uint8).cpu()), strip(codes))


@pytest.mark.parametrize("out", ["f32", "fp8blk", "fp8row"])
def test_not_a_number_stays_in_its_row(sdm, out):
    xs, w, _ = make(3, 48, F32, None)
    clean = sdm.rmsnorm_residual(xs, w, None, out=out)[0]
    bad = xs.clone()
    bad[1, 20] = float("nan")
    got = sdm.rmsnorm_residual(bad, w, None, out=out)[0]
    rows = lambda r: (r if out == "f32" else r[:3 * 48].reshape(3, 48) if out == "fp8blk"  # noqa: E731
                      else r[0].view(torch.uint8))
    a, b = rows(clean), rows(got)
    assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert bool((torch.isnan(b[1]) if out == "f32" else b[1] == 0x7F).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decoding(sdm, dtype):
    """Both formats read back as E4M3 value times scale, rounded once."""
    xs, w, _ = make(7, 96, F32, None, seed=3, scale=30.0)
    buf, _ = sdm.rmsnorm_residual(xs, w, None, out="fp8blk")
    n = 7 * 96
    grid = ref.e4m3_grid()
    value = lambda c: torch.where(c >= 128, -grid[(c % 128).long()], grid[(c % 128).long()])  # noqa: E731
    want = value(buf[:n].cpu()).reshape(-1, 16) * torch.exp2(buf[n:].cpu().view(torch.int8).double())[:, None]
    got = sdm.dequantize_fp8blk(buf, (7, 96), dtype)
    assert torch.equal(got.cpu(), want.reshape(7, 96).to(dtype))
    (codes, scales), _ = sdm.rmsnorm_residual(xs, w, None, out="fp8row")
    want = (value(codes.view(torch.uint8).cpu()).float() * scales.cpu()[:, None]).to(dtype)
    assert torch.equal(sdm.dequantize_fp8row(codes, scales, dtype).cpu(), want)
    # a buffer made by the state's quantiser reads back too
    state = sdm.quantize_fp8blk(xs)
    assert sdm.dequantize_fp8blk(state, xs.shape).shape == xs.shape


@pytest.mark.parametrize("rows,d", [(9, 640), (70, 24), (5, 1001)])
def test_every_place_an_output_may_take(sdm, rows, d):
    """h and y over x or the residual, dx over h, dh or dy: the bits of separate outputs."""
    from sparse_memory_linear_pkm_b200 import native

    lib, st = native.load(), torch.cuda.current_stream().cuda_stream
    xs, w, r = make(rows, d, BF16, BF16, seed=4)
    want_y, want_h = sdm.rmsnorm_residual(xs, w, r)
    p = lambda t: t.data_ptr()  # noqa: E731
    for h_at, y_at in (("r", "x"), ("x", "r"), ("h", "x"), ("h", "r"), ("r", "y"), ("x", "y")):
        t = {"x": xs.clone(), "r": r.clone(), "h": torch.empty_like(r), "y": torch.empty_like(xs)}
        native.check(lib.sdm_rmsnorm_residual(p(t["x"]), native.BF16, p(t["r"]), native.BF16, p(w), native.F32, rows, d,
                                              1e-6, p(t[h_at]), p(t[y_at]), native.BF16, None, st))
        assert torch.equal(t[h_at], want_h) and torch.equal(t[y_at], want_y)
    dy, dh = (torch.randn(rows, d, generator=torch.Generator().manual_seed(i)).to(BF16).cuda() for i in range(2))
    want = sdm.rmsnorm_residual_backward(want_h, w, dy, dh)
    n = lib.sdm_rmsnorm_residual_backward_workspace_bytes(rows, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for at in ("h", "dy", "dh"):
        t = {"h": want_h.clone(), "dy": dy.clone(), "dh": dh.clone()}
        dw = torch.empty(d, device="cuda")
        native.check(lib.sdm_rmsnorm_residual_backward(p(t["h"]), native.BF16, p(w), native.F32, p(t["dy"]), native.BF16,
                                                       p(t["dh"]), rows, d, 1e-6, p(t[at]), p(dw), p(ws), n, st))
        assert torch.equal(t[at], want[0]) and torch.equal(dw, want[1])


def rows_of_scales(d, dtype, seed=0):
    """Rows whose squares leave fp32's range and rows that do not, side by side."""
    scales = [1e-44, 1e-42, 1e-38, 1.0, 1e-30, 1e-25, 3e-21, 1e-19, 1e-18, 1e-16, 3e15, 1e17, 1e20, 2.0, 1e30, 3e37]
    g = torch.Generator().manual_seed(seed + d)
    x = torch.randn(len(scales), d, generator=g).double().clamp(-4, 4) * torch.tensor(scales).double()[:, None]
    return x.to(dtype).cuda()


@pytest.mark.parametrize("d", [1, 7, 24, 128, 512, 600, 1000, 2048, 8191])
@pytest.mark.parametrize("dtype,eps", [(F32, 0.0), (F32, 1e-42), (F32, 1e-36), (F32, 1e30), (BF16, 0.0), (BF16, 1e-6)])
def test_rows_whose_squares_leave_the_range(sdm, d, dtype, eps):
    """Scaling by a power of two is exact, so the errors are those of other rows. (A row that rounded to zeros has no
    norm with eps = 0: not a number, as the definition.)"""
    x = rows_of_scales(d, dtype)
    w = (torch.rand(d, generator=torch.Generator().manual_seed(d)) + 0.5).cuda()
    eps = float(torch.tensor(eps, dtype=torch.float32))  # as the call takes it
    want, _ = ref.norm(x, w, None, eps)
    y, _ = sdm.rmsnorm_residual(x, w, None, out="f32", eps=eps)
    none = torch.isnan(want)
    assert torch.equal(torch.isnan(y.cpu()), none)
    want = torch.where(none, 0.0, want)
    # Below fp32's normal range (rows far below sqrt(eps)) roundings are absolute, half the least step of 2^-149 each:
    # that of h s, which w <= 1.5 multiplies, and that of its product with w: (1.5 + 1) 2^-150.
    ref.assert_within(torch.nan_to_num(y), want, NORM_REL * want.abs() + 2.5 * 2.0 ** -150, "y")


def test_infinite_values_of_a_row(sdm):
    """s is 0: 0 for finite values and not a number for infinite ones, and rows beside it keep their bits."""
    x = rows_of_scales(64, F32)
    w = torch.ones(64, device="cuda")
    clean = sdm.rmsnorm_residual(x, w, None, eps=0.0)[0]
    x[3, 5] = float("inf")
    x[13, 9] = float("-inf")
    y = sdm.rmsnorm_residual(x, w, None, eps=0.0)[0]
    for r in range(16):
        if r in (3, 13):
            assert bool((torch.isnan(y[r]) == torch.isinf(x[r])).all()) and not torch.nan_to_num(y[r]).any()
        else:
            assert torch.equal(y[r], clean[r])


def bf16_of(v: torch.Tensor) -> torch.Tensor:
    """64-bit values rounded to bf16 once: through fp32 cut off with its last bit set where something was."""
    f = v.float()
    odd = (f.view(torch.int32) - (f.double().abs() > v.abs()).int()) | (f.double() != v).int()
    return torch.where(torch.isfinite(f), odd.view(torch.float32), f).to(BF16)


def test_decoding_rounds_once(sdm):
    """Products of all codes with scales all over the range, also those whose fp32 rounding lies on a border of bf16,
    equal the real product rounded once; a scale that is not finite gives what its product is."""
    g = torch.Generator().manual_seed(0)
    scales = torch.exp2(torch.rand(8192, generator=g) * 270 - 149)
    scales[:4] = torch.tensor([float("inf"), float("nan"), 0.0, 2.0 ** -149])
    # 24-bit significands whose product with m = 9, 11, 13 or 15 is next to a border, an odd multiple of half a step
    near = torch.cat([(torch.arange(257, 512, 2) * 2.0 ** k / m).round() for m in (9, 11, 13, 15) for k in (18, 19, 20)])
    near = near[(near >= 2 ** 23) & (near < 2 ** 24)].float()
    scales[4:4 + near.numel()] = near * torch.exp2(torch.arange(near.numel()) % 200 - 140.0)
    codes = torch.arange(256, dtype=torch.uint8).repeat(8192, 1)
    grid = torch.cat([ref.e4m3_grid(), torch.full((1,), float("nan")).double()])
    values = torch.cat([grid, -grid])
    exact = values[codes.long()] * scales.double()[:, None]
    want = bf16_of(exact)
    nan = torch.isnan(exact)
    assert int((exact.float().to(BF16) != want)[~nan].sum()) > 100  # where rounding twice differs
    got = sdm.dequantize_fp8row(codes.cuda().view(torch.float8_e4m3fn), scales.cuda(), BF16).cpu()
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])
    wide = sdm.dequantize_fp8row(codes.cuda().view(torch.float8_e4m3fn), scales.cuda()).cpu()
    assert torch.equal(wide[~nan], exact.float()[~nan])


def test_in_place_residual_and_output(sdm):
    xs, w, r = make(9, 640, BF16, BF16, seed=4)
    y, h = sdm.rmsnorm_residual(xs, w, r)
    r2 = r.clone()
    y2, h2 = sdm.rmsnorm_residual(xs, w, r2, h=r2)
    assert h2 is r2 and torch.equal(h, r2) and torch.equal(y, y2)


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (200, 8), (33, 24), (7, 100), (300, 512), (5, 513), (1200, 1024),
                                    (9, 2047), (400, 2048), (3, 8192)])
@pytest.mark.parametrize("h,dy,with_dh", [(BF16, BF16, True), (F32, F32, True), (F32, BF16, False),
                                          (BF16, F32, False)])
def test_gradient(sdm, rows, d, h, dy, with_dh):
    hs, w, _ = make(rows, d, h, None, seed=d, scale=2.0)
    g = torch.Generator().manual_seed(5)
    dys = torch.randn(rows, d, generator=g).to(dy).cuda()
    dh = torch.randn(rows, d, generator=g).to(h).cuda() if with_dh else None
    dx, dw = sdm.rmsnorm_residual_backward(hs, w, dys, dh, eps=1e-6)
    assert dx.dtype == h and dw.dtype == F32
    hh, ww = ref.d(hs).requires_grad_(), ref.d(w).requires_grad_()
    y = hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + 1e-6) * ww
    loss = (y * ref.d(dys)).sum() + (0 if dh is None else (hh * ref.d(dh)).sum())
    wdx, wdw = torch.autograd.grad(loss, [hh, ww])
    H, G = ref.d(hs).abs(), (ref.d(dys) * ref.d(w)).abs()
    s = 1 / torch.sqrt((H * H).mean(-1, keepdim=True) + 1e-6)
    # every term carries the sums' 37 roundings (s^3: 3/2 of them) and a few products
    size = G * s + H * s ** 3 * (G * H).mean(-1, keepdim=True) + (0 if dh is None else ref.d(dh).abs())
    ref.assert_within(dx, wdx, 110 * ref.U * size, "dx")
    # dw adds rows in a thread one after the other, slots by 32, then a tree
    adds = -(-rows // 148) + 40 + 32
    ref.assert_within(dw, wdw, (adds + 24) * ref.U * (ref.d(dys).abs() * H * s).sum(0), "dw")
    again = sdm.rmsnorm_residual_backward(hs, w, dys, dh, eps=1e-6)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("d", [1, 7, 24, 512, 600, 2048])
@pytest.mark.parametrize("dtype,eps", [(F32, 0.0), (F32, 1e-40), (F32, 1e-6), (BF16, 0.0), (BF16, 1e25)])
def test_gradient_of_rows_whose_squares_leave_the_range(sdm, d, dtype, eps):
    scales = [1e-36, 1.0, 1e-30, 1e-25, 1e-21, 3e-19, 1e-15, 1e-10, 1e-9, 1e10, 1e12, 1e17, 1e20, 2.0, 1e30, 3e37]
    g = torch.Generator().manual_seed(d)
    h = (torch.randn(16, d, generator=g).double().clamp(-4, 4) * torch.tensor(scales).double()[:, None]).to(dtype).cuda()
    w = (torch.rand(d, generator=g) + 0.5).cuda()
    dy, dh = (torch.randn(16, d, generator=g).to(dtype).cuda() for _ in range(2))
    eps = float(torch.tensor(eps, dtype=torch.float32))  # as the call takes it
    hh, ww = ref.d(h).requires_grad_(), ref.d(w).requires_grad_()
    y = hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + eps) * ww
    wdx, wdw = torch.autograd.grad((y * ref.d(dy)).sum() + (hh * ref.d(dh)).sum(), [hh, ww])
    alone = torch.autograd.grad((hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + eps) * ww * ref.d(dy)).sum(), hh)[0]
    H, G = ref.d(h).abs(), (ref.d(dy) * ref.d(w)).abs()
    s = 1 / torch.sqrt((H * H).mean(-1, keepdim=True) + eps)
    size = G * s + H * s ** 3 * (G * H).mean(-1, keepdim=True)
    dx, dw = sdm.rmsnorm_residual_backward(h, w, dy, dh, eps=eps)
    ref.assert_within(dx, wdx, 110 * ref.U * (size + ref.d(dh).abs()), "dx")  # as for other rows
    adds = 1 + 40 + 32
    ref.assert_within(dw, wdw, (adds + 24) * ref.U * (ref.d(dy).abs() * H * s).sum(0), "dw")
    # without dh: below the type's normal range the fp32 value and its rounding are off by half a least step each
    least = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
    dx, _ = sdm.rmsnorm_residual_backward(h, w, dy, None, eps=eps)
    ref.assert_within(dx, alone, 110 * ref.U * size + 2.0 ** -150 + least / 2, "dx without dh")


def test_gradient_against_differences(sdm):
    """The loss' change along a direction, from 64-bit forward passes, is the gradient's product with it."""
    hs, w, _ = make(6, 40, F32, None, seed=8)
    g = torch.Generator().manual_seed(9)
    dy = torch.randn(6, 40, generator=g).cuda()
    dx, dw = sdm.rmsnorm_residual_backward(hs, w, dy)
    vx, vw = torch.randn(6, 40, generator=g).double(), torch.randn(40, generator=g).double()
    step = 1e-5
    loss = lambda t: float((ref.norm(ref.d(hs) + t * vx, ref.d(w) + t * vw, None, 1e-6)[0] * ref.d(dy)).sum())  # noqa: E731
    slope = (loss(step) - loss(-step)) / (2 * step)
    got = float((ref.d(dx) * vx).sum() + (ref.d(dw) * vw).sum())
    # the differences' own error is about step^2 = 1e-10 of the terms, the gradients' 110 * 2^-24
    size = float((ref.d(dx).abs() * vx.abs()).sum() + (ref.d(dw).abs() * vw.abs()).sum())
    assert abs(got - slope) <= 2e-5 * size


def test_empty(sdm):
    x, w = torch.empty(0, 32, device="cuda"), torch.ones(32, device="cuda")
    y, h = sdm.rmsnorm_residual(x, w, x.clone())
    assert y.shape == (0, 32) and h.shape == (0, 32)
    dx, dw = sdm.rmsnorm_residual_backward(x, w, x)
    assert dx.shape == (0, 32) and not dw.any()
