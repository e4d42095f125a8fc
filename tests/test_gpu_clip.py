"""Global gradient norm and clipping against 64-bit definitions."""

import math

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def total(grads):
    return math.sqrt(sum(float((ref.d(g) ** 2).sum()) for g in grads))


def check(sdm, grads, max_norm, outs=None, eps=1e-6):
    """The norm is exact but for eight squares' fp32 sum (8 roundings, halved) and its own rounding; c adds two, the
    product one."""
    n = total(grads)
    before = [ref.d(g).clone() for g in grads]
    got = sdm.grad_norm_clip(grads, max_norm, eps=eps, out=outs)
    assert got.dtype == F32 and got.shape == ()
    assert abs(float(got) - n) <= 6 * ref.U * n
    c = min(1.0, max_norm / (n + eps))
    for b, o in zip(before, grads if outs is None else outs):
        ref.assert_within(o.reshape(-1), (b * c).reshape(-1), 8 * ref.U * (b * c).abs().reshape(-1), "scaled")
    return got


SIZES = [[1], [3, 5], [2048], [2049, 7, 1, 4096], [100_003, 17, 0, 70_000, 8], [600_000, 1_000_001]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype,out", [(F32, None), (BF16, None), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_values(sdm, sizes, dtype, out, max_norm):
    g = torch.Generator().manual_seed(len(sizes))
    grads = [torch.randn(n, generator=g).to(dtype).cuda() for n in sizes]
    outs = None if out is None else [torch.empty(n, dtype=out, device="cuda") for n in sizes]
    check(sdm, grads, max_norm, outs)


def test_many_tensors(sdm):
    """More tensors than one launch takes, of mixed types and shapes, views that start anywhere."""
    g = torch.Generator().manual_seed(0)
    flat = torch.randn(200_000, generator=g).cuda()
    grads, at = [], 1
    for i in range(900):
        n = (i * 37) % 211
        grads.append(flat[at:at + n] if i % 3 else torch.randn(max(1, i % 5), 3, generator=g).to(BF16).cuda())
        at += n
    check(sdm, grads, 2.0, [torch.empty(t.shape, dtype=F32, device="cuda") for t in grads])
    check(sdm, grads, 2.0)


def test_untouched_where_nothing_is_clipped(sdm):
    g = torch.randn(5000, generator=torch.Generator().manual_seed(1)).cuda()
    before = g.clone()
    sdm.grad_norm_clip([g], 1e6)
    assert torch.equal(g, before)
    norm = sdm.grad_norm_clip([g], float("inf"))
    assert torch.equal(g, before) and abs(float(norm) - total([before])) <= 6 * ref.U * total([before])
    out = torch.empty_like(g)
    sdm.grad_norm_clip([g], float("inf"), out=[out])
    assert torch.equal(out, before)


@pytest.mark.parametrize("scale", [1e25, 1e-25, 1e-38])
def test_squares_beyond_fp32(sdm, scale):
    g = (torch.randn(3000, generator=torch.Generator().manual_seed(2)).double() * scale).float().cuda()
    n = total([g])
    got = sdm.grad_norm_clip([g], float("inf"))
    assert abs(float(got) - n) <= 6 * ref.U * n + 2.0 ** -149


def test_zero_and_empty(sdm):
    z = torch.zeros(70, device="cuda")
    assert float(sdm.grad_norm_clip([z, torch.empty(0, device="cuda")], 1.0)) == 0.0 and not z.any()
    assert float(sdm.grad_norm_clip([torch.empty(0, device="cuda")], 1.0)) == 0.0


def test_not_finite(sdm):
    """A norm that is not finite does what the formula says: 0 for infinity (0 * inf is not a number), NaN for NaN."""
    g = torch.ones(100, device="cuda")
    g[3] = float("inf")
    out = torch.empty_like(g)
    assert math.isinf(float(sdm.grad_norm_clip([g], 1.0, out=[out])))
    assert math.isnan(float(out[3])) and float(out[0]) == 0.0
    g[3] = float("nan")
    assert math.isnan(float(sdm.grad_norm_clip([g], 1.0, out=[out]))) and bool(torch.isnan(out).all())


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, F32)])
def test_infinite_max_norm_copies_whatever_the_norm_is(sdm, value, dtype, out_dtype):
    """max_norm = inf scales nothing: a gradient that is not finite leaves all other values as they are."""
    g = torch.randn(5000, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    g[77] = value
    rest = torch.randn(301, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    outs = [torch.empty(t.shape, dtype=out_dtype, device="cuda") for t in (g, rest)]
    norm = sdm.grad_norm_clip([g, rest], float("inf"), out=outs)
    assert not math.isfinite(float(norm))
    for got, want in zip(outs, (g, rest)):
        assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want.to(out_dtype), nan=7.0))
    before = g.clone()
    sdm.grad_norm_clip([g, rest], float("inf"))
    assert torch.equal(torch.nan_to_num(g, nan=7.0), torch.nan_to_num(before, nan=7.0))


def test_norm_beside_its_tensors(sdm):
    """The norm's place may touch a tensor, or be where one without values points."""
    from sparse_memory_linear_pkm_b200 import native

    lib = native.load()
    flat = torch.randn(2001, generator=torch.Generator().manual_seed(6)).cuda()
    want = flat.clone()
    n = total([want[:1000], want[1001:]])
    at = flat.data_ptr()
    table = (native.GradTensor * 3)(native.GradTensor(at, at, 1000, native.F32, native.F32),
                                    native.GradTensor(at + 4000, None, 0, native.F32, native.F32),
                                    native.GradTensor(at + 4004, at + 4004, 1000, native.F32, native.F32))
    ws = torch.empty(lib.sdm_grad_norm_clip_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    native.check(lib.sdm_grad_norm_clip(table, 3, 1.0, 1e-6, at + 4000, ws.data_ptr(), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream))
    assert abs(float(flat[1000]) - n) <= 6 * ref.U * n
    want[1000] = 0
    flat[1000] = 0
    ref.assert_within(flat, ref.d(want) / (n + 1e-6), 8 * ref.U * ref.d(want).abs(), "scaled")


def test_same_bits_every_time(sdm):
    g = [torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda() for n in (1_000_003, 77, 250_000)]
    first = sdm.grad_norm_clip(g, float("inf"))
    for _ in range(5):
        assert torch.equal(sdm.grad_norm_clip(g, float("inf")), first)
