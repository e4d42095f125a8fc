"""Host-side checks of the operators around the recurrent core: what they refuse,
and their sizes, without a GPU."""

import ctypes
import subprocess
import sys
from pathlib import Path

import pytest
import torch

from sparse_memory_linear_pkm_b200 import build as build_mod
from sparse_memory_linear_pkm_b200 import native

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
BYTE = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return native.load()


def refused(lib, status, text, code=1):
    assert status == code, (status, lib.sdm_last_error())
    assert text.encode() in lib.sdm_last_error(), lib.sdm_last_error()


def norm_args(**kw):
    d = dict(x=P, x_dtype=native.BF16, residual=P, res_dtype=native.F32, w=P, w_dtype=native.F32, n_rows=4, d=32,
             eps=1e-6, h=P, y=P, y_dtype=native.BF16, scales=None, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,text,code", [
    (dict(x=None), "x is NULL", 1), (dict(x=ODD), "x is not 16-byte", 1), (dict(w=None), "w is NULL", 1),
    (dict(h=None), "h is NULL", 1), (dict(y=None), "y is NULL", 1), (dict(residual=ODD), "residual", 1),
    (dict(x_dtype=native.FP8_B16), "x_dtype", 1), (dict(res_dtype=9), "res_dtype", 1), (dict(w_dtype=-1), "w_dtype", 1),
    (dict(y_dtype=4), "y_dtype", 1), (dict(d=0), "d must", 1), (dict(d=8193), "d above", 2),
    (dict(n_rows=-1), "n_rows", 1), (dict(eps=-1.0), "eps", 1), (dict(eps=float("nan")), "eps", 1),
    (dict(eps=float("inf")), "eps", 1), (dict(y_dtype=native.FP8_B16, d=40, scales=P), "multiple of 16", 1),
    (dict(y_dtype=native.FP8_B16), "scales is NULL", 1), (dict(y_dtype=native.FP8_ROW, scales=ODD), "scales", 1)])
def test_norm_refuses(lib, kw, text, code):
    refused(lib, lib.sdm_rmsnorm_residual(*norm_args(**kw)), text, code)


def test_norm_empty_and_sizes(lib):
    assert lib.sdm_rmsnorm_residual(*norm_args(x=None, w=None, h=None, y=None, residual=None, n_rows=0)) == 0
    size = lib.sdm_rmsnorm_residual_backward_workspace_bytes
    assert size(0, 32) == 0 and size(4, 0) == 0 and size(4, 8193) == 0
    # 2 lanes a row of 32: 64 rows a block, a slot of d sums each
    assert size(4, 32) == 64 * 32 * 4
    assert size(1, 2048) == 2048 * 4 and size(3, 2048) == 3 * 2048 * 4
    # at most 512 threads' worth of blocks on each of 148 SMs
    assert size(1 << 20, 2048) == 148 * 4 * 2048 * 4
    args = [P, native.F32, P, native.F32, P, native.F32, None, 3, 2048, 1e-6, P, P, P, size(3, 2048) - 1, None]
    refused(lib, lib.sdm_rmsnorm_residual_backward(*args), "workspace")
    args[12] = None
    refused(lib, lib.sdm_rmsnorm_residual_backward(*args), "workspace is NULL")
    args[5] = 7
    refused(lib, lib.sdm_rmsnorm_residual_backward(*args), "dy_dtype")


def test_norm_refuses_overlaps(lib):
    """An output may take a whole input's place where the types agree, not part of it or in another type."""
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(8)]
    next_row = lambda p, size=2: ctypes.c_void_p(p.value + 32 * size)  # noqa: E731
    base = dict(x=far[0], residual=far[1], res_dtype=native.BF16, w=far[2], h=far[3], y=far[4])
    for kw, text in ((dict(h=next_row(far[1])), "h overlaps residual"), (dict(h=next_row(far[0])), "h overlaps x"),
                     (dict(y=next_row(far[0])), "y overlaps x"), (dict(y=next_row(far[1])), "y overlaps residual"),
                     (dict(y=far[3]), "y overlaps h"), (dict(h=far[2]), "h overlaps w"), (dict(y=far[2]), "y overlaps w"),
                     (dict(res_dtype=native.F32, h=far[0]), "h overlaps x"),
                     (dict(y_dtype=native.F32, y=far[0]), "y overlaps x"),
                     (dict(y_dtype=native.FP8_ROW, y=far[0], scales=far[5]), "y overlaps x"),
                     (dict(y_dtype=native.FP8_B16, y=far[1], scales=far[5]), "y overlaps residual"),
                     (dict(y_dtype=native.FP8_ROW, scales=far[4]), "scales overlaps y"),
                     (dict(y_dtype=native.FP8_B16, scales=far[3]), "scales overlaps h"),
                     (dict(y_dtype=native.FP8_B16, scales=far[1]), "scales overlaps residual")):
        refused(lib, lib.sdm_rmsnorm_residual(*norm_args(**(base | kw))), text)
    size = lib.sdm_rmsnorm_residual_backward_workspace_bytes(3, 2048)
    base = [far[0], native.BF16, far[1], native.F32, far[2], native.F32, far[3], 3, 2048, 1e-6, far[4], far[5], P, size, None]
    row = lambda p: ctypes.c_void_p(p.value + 2048 * 2)  # noqa: E731
    for at, value, text in ((10, row(far[0]), "dx overlaps h"), (10, row(far[3]), "dx overlaps dh"),
                            (10, far[2], "dx overlaps dy"), (10, far[1], "dx overlaps w"), (11, far[0], "dw overlaps h"),
                            (11, far[1], "dw overlaps w"), (11, far[2], "dw overlaps dy"), (11, far[3], "dw overlaps dh"),
                            (11, far[4], "dw overlaps dx")):
        args = list(base)
        args[at] = value
        refused(lib, lib.sdm_rmsnorm_residual_backward(*args), text)


def test_decoding_refuses(lib):
    refused(lib, lib.sdm_dequantize_fp8blk(None, P, 1, P, native.F32, None), "codes is NULL")
    refused(lib, lib.sdm_dequantize_fp8blk(P, None, 1, P, native.F32, None), "exps is NULL")
    refused(lib, lib.sdm_dequantize_fp8blk(P, P, -1, P, native.F32, None), "n_blocks")
    refused(lib, lib.sdm_dequantize_fp8blk(P, P, 1, P, native.FP8_B16, None), "out_dtype")
    refused(lib, lib.sdm_dequantize_fp8row(P, P, 1, 24, P, native.F32, None), "multiple of 16")
    refused(lib, lib.sdm_dequantize_fp8row(P, ODD, 1, 32, P, native.F32, None), "scales")
    assert lib.sdm_dequantize_fp8blk(None, None, 0, None, native.F32, None) == 0
    assert lib.sdm_dequantize_fp8row(None, None, 0, 32, None, native.F32, None) == 0


def test_decoding_refuses_overlaps(lib):
    """A value takes more room than its code: decoding in place would write codes that are still to be read."""
    a, b, o = (ctypes.c_void_p(i << 24) for i in (2, 3, 4))
    for out, text in ((a, "out overlaps codes"), (ctypes.c_void_p(a.value + 496), "out overlaps codes")):
        refused(lib, lib.sdm_dequantize_fp8blk(a, b, 32, out, native.BF16, None), text)
        refused(lib, lib.sdm_dequantize_fp8row(a, b, 16, 32, out, native.F32, None), text)
    refused(lib, lib.sdm_dequantize_fp8blk(a, b, 32, b, native.F32, None), "out overlaps exps")
    refused(lib, lib.sdm_dequantize_fp8row(a, b, 16, 32, b, native.BF16, None), "out overlaps scales")
    refused(lib, lib.sdm_dequantize_fp8blk(a, ctypes.c_void_p(o.value + 64), 32, o, native.F32, None), "out overlaps exps")


def conv_args(**kw):
    d = dict(x=P, x_stride=0, in_dtype=native.BF16, w=P, bias=P, w_dtype=native.F32, B=2, T=9, D=24, K=4, silu=1,
             state=P, lengths=P, y=ctypes.c_void_p(1 << 24), stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,text,code", [
    (dict(x=None), "x is NULL", 1), (dict(x=BYTE), "x is not aligned", 1), (dict(w=None), "w is NULL", 1),
    (dict(bias=ODD), "bias", 1), (dict(state=ODD), "state", 1), (dict(lengths=ODD), "lengths", 1),
    (dict(y=None), "y is NULL", 1), (dict(y=ctypes.c_void_p((1 << 24) + 2)), "y is not 16-byte", 1),
    (dict(K=1), "K must", 1), (dict(K=9), "K must", 1), (dict(B=-1), "B, T and D", 1), (dict(B=65536), "B above", 2),
    (dict(x_stride=23), "x_stride", 1), (dict(in_dtype=2), "in_dtype", 1), (dict(w_dtype=2), "w_dtype", 1),
    (dict(T=2 ** 31 - 1, D=24), "above 2^31", 2), (dict(y=P), "y overlaps x", 1),
    (dict(state=ctypes.c_void_p((1 << 24) + 16)), "state overlaps y", 1), (dict(state=P), "state overlaps x", 1)])
def test_conv_refuses(lib, kw, text, code):
    refused(lib, lib.sdm_short_conv(*conv_args(**kw)), text, code)


def test_conv_empty_and_gradient(lib):
    for kw in (dict(B=0), dict(T=0), dict(D=0)):
        assert lib.sdm_short_conv(*conv_args(x=None, w=None, bias=None, state=None, lengths=None, y=None, **kw)) == 0
    size = lib.sdm_short_conv_backward_workspace_bytes
    assert size(2, 0, 24, 4) == 0 and size(2, 9, 24, 1) == 0
    # blocks of 8 segments of 64 tokens; a sum per tap and one for the bias
    assert size(2, 9, 24, 4) == (24 * 5 * 4 + 255) // 256 * 256
    assert size(3, 1024, 64, 3) == 6 * 64 * 4 * 4
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(8)]
    base = [P, 0, native.BF16, P, P, native.F32, 2, 9, 24, 4, 1, None, None, far[0], None, far[1], far[2], far[3], None,
            far[4], size(2, 9, 24, 4), None]
    for at, value, text in ((13, None, "dy is NULL"), (15, None, "dx is NULL"), (16, None, "dw is NULL"),
                            (15, far[0], "dx overlaps"), (19, None, "workspace"), (20, 8, "workspace is smaller"),
                            (18, ODD, "dstate0"), (9, 12, "K must")):
        args = list(base)
        args[at] = value
        refused(lib, lib.sdm_short_conv_backward(*args), text)
    args = list(base)
    args[11] = args[18] = far[5]
    refused(lib, lib.sdm_short_conv_backward(*args), "dstate0 overlaps")


def test_conv_refuses_outputs_on_any_input(lib):
    """Taps, bias and lengths count as inputs too, and the parameters' gradients as outputs."""
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(12)]
    for name, on in (("y", ("w", "bias", "lengths")), ("state", ("w", "bias", "lengths"))):
        for i, n in enumerate(on):
            kw = dict(x=far[0], w=far[1], bias=far[2], lengths=far[3], state=far[4], y=far[5])
            kw[name] = far[1 + i]
            refused(lib, lib.sdm_short_conv(*conv_args(**kw)), f"{name} overlaps {n}")
    need = lib.sdm_short_conv_backward_workspace_bytes(2, 9, 24, 4)
    names = {0: "x", 3: "w", 4: "bias", 11: "state0", 12: "lengths", 13: "dy", 14: "dstate", 15: "dx", 16: "dw",
             17: "dbias", 18: "dstate0"}
    base = [far[0], 0, native.BF16, far[1], far[2], native.F32, 2, 9, 24, 4, 1, *far[3:11], P, need, None]
    for i in (15, 16, 17, 18):
        for j in names:
            if i != j:
                args = list(base)
                args[i] = args[j]
                status = lib.sdm_short_conv_backward(*args)
                assert status == 1 and b" overlaps " in lib.sdm_last_error(), (names[i], names[j], status)
                assert names[i].encode() in lib.sdm_last_error() and names[j].encode() in lib.sdm_last_error()


def shape(**kw):
    d = dict(B=2, T=40, D=32, N=16, G=1, in_dtype=native.BF16, softplus=1, reserved=0, x_stride=0, dt_stride=0,
             z_stride=0, b_stride=0, c_stride=0)
    d.update(kw)
    return native.SelscanShape(**d)


@pytest.mark.parametrize("kw,text,code", [
    (dict(B=-1), "B, T and D", 1), (dict(N=0), "N must", 1), (dict(N=65), "N must", 1), (dict(G=0), "G must", 1),
    (dict(G=5), "G must", 1), (dict(in_dtype=2), "in_dtype", 1), (dict(reserved=1), "reserved", 1),
    (dict(x_stride=31), "x_stride", 1), (dict(dt_stride=1), "dt_stride", 1), (dict(z_stride=-1), "z_stride", 1),
    (dict(b_stride=15), "b_stride", 1), (dict(c_stride=3), "c_stride", 1), (dict(B=65536), "B above", 2),
    (dict(T=2 ** 31 - 1), "T above", 2)])
def test_scan_refuses_shapes(lib, kw, text, code):
    s = ctypes.byref(shape(**kw))
    assert lib.sdm_selective_scan_workspace_bytes(s) == 0
    assert lib.sdm_selective_scan_backward_workspace_bytes(s) == 0
    refused(lib, lib.sdm_selective_scan(s, *([P] * 13), 0, None), text, code)
    refused(lib, lib.sdm_selective_scan_backward(s, *([P] * 22), 0, None), text, code)


def test_scan_refuses_pointers(lib):
    s = ctypes.byref(shape())
    names = ["x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "lengths", "h0", "hT", "y"]
    for i, n in enumerate(names):
        args = [P] * 12
        args[i] = BYTE
        refused(lib, lib.sdm_selective_scan(s, *args, None, 0, None), n + " is not")
        if n in ("x", "dt", "A", "Bm", "Cm", "y"):
            args[i] = None
            refused(lib, lib.sdm_selective_scan(s, *args, None, 0, None), n + " is NULL")
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(12)]
    for i, text in ((11, "y overlaps"), (10, "hT overlaps")):
        for j in (0, 1, 3, 4, 6):
            args = list(far)
            args[i] = ctypes.c_void_p(far[j].value + 16)
            refused(lib, lib.sdm_selective_scan(s, *args, None, 0, None), f"{text} {names[j]}")
    args = list(far)
    args[10] = ctypes.c_void_p(far[9].value + 64)
    refused(lib, lib.sdm_selective_scan(s, *args, None, 0, None), "hT overlaps h0")
    assert lib.sdm_selective_scan(None, *([P] * 13), 0, None) == 1
    for kw in (dict(B=0), dict(D=0)):
        assert lib.sdm_selective_scan(ctypes.byref(shape(**kw)), *([None] * 13), 0, None) == 0
    # few channels, many tokens: two arrays of states before the splits
    long = shape(B=1, T=8192, D=32)
    need = lib.sdm_selective_scan_workspace_bytes(ctypes.byref(long))
    assert need == 2 * 256 * 32 * 16 * 4  # 256 splits of 32 tokens
    refused(lib, lib.sdm_selective_scan(ctypes.byref(long), *([P] * 12), P, need - 1, None), "workspace is smaller")
    refused(lib, lib.sdm_selective_scan(ctypes.byref(long), *([P] * 12), None, need, None), "workspace is NULL")
    assert lib.sdm_selective_scan_workspace_bytes(s) == 0


def test_scan_gradient_refuses(lib):
    s = shape()
    need = lib.sdm_selective_scan_backward_workspace_bytes(ctypes.byref(s))
    assert need > 0
    names = ["x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "lengths", "h0", "dy", "dhT", "dx", "ddt", "dA", "dB",
             "dC", "dD", "dz", "ddt_bias", "dh0", "workspace"]
    for i, n in enumerate(names):
        args = [P] * 22
        args[i] = BYTE
        refused(lib, lib.sdm_selective_scan_backward(ctypes.byref(s), *args, need, None), n + " is not")
        if n not in ("Dskip", "z", "dt_bias", "lengths", "h0", "dhT", "dh0"):
            args[i] = None
            refused(lib, lib.sdm_selective_scan_backward(ctypes.byref(s), *args, need, None), n + " is NULL")
    refused(lib, lib.sdm_selective_scan_backward(ctypes.byref(s), *([P] * 22), need - 1, None), "workspace is smaller")
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(22)]
    for i, j in ((12, 0), (13, 10), (18, 6), (15, 3), (16, 15), (14, 1)):
        args = list(far)
        args[i] = far[j]
        refused(lib, lib.sdm_selective_scan_backward(ctypes.byref(s), *args, need, None), f"{names[i]} overlaps {names[j]}")


def test_scan_refuses_outputs_on_any_input(lib):
    """Parameters, lengths and states count as inputs too, and every output as one."""
    s = shape()
    names = ["x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "lengths", "h0", "hT", "y"]
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(22)]
    for i in (10, 11):
        for j in (2, 5, 7, 8):
            args = far[:12]
            args[i] = far[j]
            refused(lib, lib.sdm_selective_scan(ctypes.byref(s), *args, None, 0, None), f"{names[i]} overlaps {names[j]}")
    need = lib.sdm_selective_scan_backward_workspace_bytes(ctypes.byref(s))
    names = ["x", "dt", "A", "Bm", "Cm", "Dskip", "z", "dt_bias", "lengths", "h0", "dy", "dhT", "dx", "ddt", "dA", "dB",
             "dC", "dD", "dz", "ddt_bias", "dh0"]
    for i in range(12, 21):
        for j in range(12):
            args = list(far)
            args[i] = ctypes.c_void_p(far[j].value + (16 if (i, j) == (20, 11) else 0))
            refused(lib, lib.sdm_selective_scan_backward(ctypes.byref(s), *args, need, None),
                    f"{names[i]} overlaps {names[j]}")
        for j in range(12, 21):
            if i != j:
                args = list(far)
                args[i] = far[j]
                status = lib.sdm_selective_scan_backward(ctypes.byref(s), *args, need, None)
                assert status == 1 and b" overlaps " in lib.sdm_last_error()


def test_calls_without_tokens_refuse_overlapping_states(lib):
    """There the state is copied: onto itself it stays, onto a part of itself the copy has no order."""
    a = ctypes.c_void_p(1 << 24)
    part = ctypes.c_void_p(a.value + 64)
    s = ctypes.byref(shape(T=0))
    none = [None] * 9
    refused(lib, lib.sdm_selective_scan(s, *none, a, part, None, None, 0, None), "hT overlaps h0")
    assert lib.sdm_selective_scan(s, *none, a, a, None, None, 0, None) == 0
    far = [ctypes.c_void_p((i + 2) << 24) for i in range(4)]
    args = [*none, None, None, a, None, None, far[1], None, None, None, None, None, part, None, 0, None]
    refused(lib, lib.sdm_selective_scan_backward(s, *args), "dh0 overlaps dhT")
    args = [None, 0, native.BF16, None, None, native.F32, 2, 0, 24, 4, 1, None, None, None, a, None, far[1], None, part,
            None, 0, None]
    refused(lib, lib.sdm_short_conv_backward(*args), "dstate0 overlaps dstate")


def clip(lib, entries, max_norm=1.0, eps=1e-6, norm=P, ws=P, ws_bytes=None):
    table = (native.GradTensor * max(1, len(entries)))(*[native.GradTensor(*e) for e in entries])
    n = lib.sdm_grad_norm_clip_workspace_bytes(len(entries)) if ws_bytes is None else ws_bytes
    return lib.sdm_grad_norm_clip(ctypes.byref(table), len(entries), max_norm, eps, norm, ws, n, None)


def test_clip_refuses(lib):
    a, o = 1 << 20, 1 << 24
    good = (a, o, 100, native.F32, native.F32)
    for entry, text in (((a, o, -1, 0, 0), "tensors[1].n"), ((0, o, 5, 0, 0), "tensors[1].grad is NULL"),
                        ((a + 2, o, 5, 0, 0), "tensors[1].grad is not"), ((a, o + 2, 5, 0, 0), "tensors[1].out is not"),
                        ((a, o, 5, 2, 0), "tensors[1].dtype"), ((a, o, 5, 0, 3), "tensors[1].out_dtype"),
                        ((a, a, 5, native.BF16, native.F32), "its own output")):
        refused(lib, clip(lib, [good, entry]), text)
    refused(lib, clip(lib, [(a, o, 2 ** 41, 0, 0)]), "2^40", 2)
    # the same tensor twice, outputs that overlap, an output on another's gradient, or inside its own
    for first, second in (((a, a, 100, 0, 0), (a, a, 100, 0, 0)), (good, (a + 4096, o + 396, 5, 0, 0)),
                          (good, (o + 200, 1 << 26, 10, 0, 0)), ((o + 200, 1 << 26, 10, 0, 0), good),
                          ((a, a, 1000, 0, 0), (a + 16, o, 4, 0, 0))):
        refused(lib, clip(lib, [first, (1 << 27, 1 << 28, 7, 1, 0), second]), "overlap in an output")
    refused(lib, clip(lib, [(a, a + 4, 100, 0, 0)]), "out overlaps its own grad")
    refused(lib, clip(lib, [good], max_norm=-1.0), "max_norm")
    refused(lib, clip(lib, [good], max_norm=float("nan")), "max_norm")
    refused(lib, clip(lib, [good], eps=-1.0), "eps")
    refused(lib, clip(lib, [good], norm=None), "norm is NULL")
    refused(lib, clip(lib, [good], ws=None), "workspace is NULL")
    refused(lib, clip(lib, [good], ws_bytes=8), "workspace is smaller")
    assert lib.sdm_grad_norm_clip(None, 3, 1.0, 0.0, P, P, 1 << 20, None) == 1
    assert lib.sdm_grad_norm_clip_workspace_bytes(-1) == 0


def test_clip_refuses_a_norm_inside_a_tensor(lib):
    """The pass that writes the norm reads gradients and writes outputs at the same time."""
    a, o, far = 1 << 24, 1 << 25, 1 << 26
    good = (far, far + (1 << 20), 100, native.F32, native.F32)
    for entry in ((a, o, 100, native.F32, native.F32), (a, o, 100, native.BF16, native.F32),
                  (a, o, 200, native.F32, native.BF16), (a, a, 100, native.F32, native.F32)):
        for at, size in ((entry[0], 2 if entry[3] else 4), (entry[1], 2 if entry[4] else 4)):
            for norm in (at, at + entry[2] * size - 4):
                refused(lib, clip(lib, [good, entry], norm=ctypes.c_void_p(norm)), "norm overlaps tensors[1]")
    refused(lib, clip(lib, [good, (a, None, 10, 0, 0)], norm=ctypes.c_void_p(a)), "norm overlaps tensors[1]")


LITTLE_MEMORY = """
import ctypes, resource
import torch
from sparse_memory_linear_pkm_b200 import native
lib = native.load()
n = 2_000_000
rows = torch.zeros(n, 4, dtype=torch.int64)
rows[:, 0] = rows[:, 1] = (1 << 30) + 64 * torch.arange(n)
rows[:, 2] = 8
pages = int(open("/proc/self/statm").read().split()[0])
resource.setrlimit(resource.RLIMIT_AS, (pages * resource.getpagesize() + (16 << 20),) * 2)
status = lib.sdm_grad_norm_clip(rows.data_ptr(), n, 1.0, 1e-6, 1 << 20, 1 << 20, 1 << 40, None)
print(status, lib.sdm_last_error().decode())
"""


def test_clip_reports_a_lack_of_host_memory(lib):
    """No C++ exception leaves the library: a list whose check finds no memory returns an error."""
    got = subprocess.run([sys.executable, "-c", LITTLE_MEMORY], cwd=Path(__file__).resolve().parent.parent,
                         capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-500:]
    assert got.stdout.startswith("2 not enough host memory"), got.stdout


def test_front_end_has_no_cpu_path():
    import sparse_memory_linear_pkm_b200 as sdm

    x, v = torch.zeros(2, 3, 16), torch.zeros(16)
    with pytest.raises(ValueError, match="CUDA device"):
        sdm.rmsnorm_residual(x, v)
    with pytest.raises(ValueError, match="CUDA device"):
        sdm.short_conv(x, torch.zeros(16, 4))
    with pytest.raises(ValueError, match="CUDA device"):
        sdm.selective_scan(x, x, torch.zeros(16, 4), torch.zeros(2, 3, 1, 4), torch.zeros(2, 3, 1, 4))
    with pytest.raises(ValueError, match="CUDA device"):
        sdm.grad_norm_clip([v], 1.0)
