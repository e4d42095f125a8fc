"""The operators around the recurrent core together, as a block of a model uses
them: training with gradients and clipping, a prompt and its tokens one by one,
on other streams, inside captured graphs, and what the front end refuses."""

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
B, T, D, N, K = 2, 48, 64, 16, 4


def params(seed=0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k)  # noqa: E731
    p = dict(norm=r(D).abs() + 0.5, w_in=r(D, 2 * D, k=D ** -0.5), conv=r(D, K, k=0.5), conv_b=r(D, k=0.1),
             w_x=r(D, D + 2 * N, k=D ** -0.5), bias=r(D) - 2, A=-(r(D, N).abs() + 0.1), skip=r(D), w_out=r(D, D, k=D ** -0.5))
    return {k: v.cuda() for k, v in p.items()}


def forward(sdm, p, x, res, conv_state=None, state=None, keep=False):
    """x + res -> norm -> projections -> convolution -> scan -> projection; the next block's input and residual."""
    y, h = sdm.rmsnorm_residual(x, p["norm"], res)
    xz = y @ p["w_in"]
    u, z = xz[..., :D], xz[..., D:]
    c = sdm.short_conv(u, p["conv"], p["conv_b"], state=conv_state)
    dbc = c @ p["w_x"]
    dt, Bm, Cm = dbc[..., :D], dbc[..., D:D + N].unflatten(-1, (1, N)), dbc[..., D + N:].unflatten(-1, (1, N))
    s = sdm.selective_scan(c, dt, p["A"], Bm, Cm, D=p["skip"], z=z, dt_bias=p["bias"], state=state)
    out = s @ p["w_out"]
    return (out, h, dict(y=y, u=u, z=z, c=c, dt=dt, Bm=Bm, Cm=Cm, s=s)) if keep else (out, h)


def backward(sdm, p, x, res, saved, h, dout):
    f = lambda a, b: a.reshape(-1, a.shape[-1]).T @ b.reshape(-1, b.shape[-1])  # noqa: E731
    g = {"w_out": f(saved["s"], dout)}
    q = sdm.selective_scan_backward(saved["c"], saved["dt"], p["A"], saved["Bm"], saved["Cm"], (dout @ p["w_out"].T),
                                    D=p["skip"], z=saved["z"], dt_bias=p["bias"])
    g["A"], g["skip"], g["bias"] = q["dA"], q["dD"], q["ddt_bias"]
    ddbc = torch.cat([q["ddt"], q["dB"].flatten(2), q["dC"].flatten(2)], -1)
    g["w_x"] = f(saved["c"], ddbc)
    v = sdm.short_conv_backward(saved["u"], p["conv"], q["dx"] + ddbc @ p["w_x"].T, p["conv_b"])
    g["conv"], g["conv_b"] = v["dw"], v["dbias"]
    dxz = torch.cat([v["dx"], q["dz"]], -1)
    g["w_in"] = f(saved["y"], dxz)
    dx, g["norm"] = sdm.rmsnorm_residual_backward(h, p["norm"], dxz @ p["w_in"].T)
    return dx, g


def wide_loss(p, x, res, dout):
    h = x + res
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * p["norm"]
    xz = y @ p["w_in"]
    full = torch.nn.functional.pad(xz[..., :D], (0, 0, K - 1, 0))
    u = sum(full[:, k:k + x.shape[1]] * p["conv"][:, k] for k in range(K)) + p["conv_b"]
    c = u * torch.sigmoid(u)
    dbc = c @ p["w_x"]
    s, _ = ref.scan(c, dbc[..., :D], p["A"], dbc[..., D:D + N].unflatten(-1, (1, N)),
                    dbc[..., D + N:].unflatten(-1, (1, N)), p["skip"], xz[..., D:], p["bias"])
    return ((s @ p["w_out"]) * dout).sum()


def test_training_step(sdm):
    """A block's loss gradients against 64-bit autograd, then their clipping."""
    p = params()
    g = torch.Generator().manual_seed(1)
    x, res, dout = (torch.randn(B, T, D, generator=g).cuda() for _ in range(3))
    torch.backends.cuda.matmul.allow_tf32 = False
    out, h, saved = forward(sdm, p, x, res, keep=True)
    dx, grads = backward(sdm, p, x, res, saved, h, dout)
    wide = {k: ref.d(v).requires_grad_() for k, v in p.items()}
    wx, wres = ref.d(x).requires_grad_(), ref.d(res)
    loss = wide_loss(wide, wx, wres, ref.d(dout))
    want = dict(zip(list(wide) + ["x"], torch.autograd.grad(loss, list(wide.values()) + [wx])))
    # Five products of 64 to 128 terms and the operators in a row, each within some 1e-5 of its terms: 1e-4 of the
    # largest value leaves a factor of about two for their passing through each other.
    for k, w in want.items():
        got = ref.d(dx if k == "x" else grads[k])
        assert float((got - w).abs().max()) <= 1e-4 * float(w.abs().max()), k
    tensors = [grads[k] for k in sorted(grads)]
    before = [t.clone() for t in tensors]
    norm = sdm.grad_norm_clip(tensors, 1.0)
    n = sum(float((ref.d(t) ** 2).sum()) for t in before) ** 0.5
    assert n > 1 and abs(float(norm) - n) <= 1e-6 * n
    for t, b in zip(tensors, before):
        ref.assert_within(t, ref.d(b) / (n + 1e-6), 8 * ref.U * ref.d(b).abs(), "clipped")
    sdm.stream_check()


def test_prompt_then_tokens(sdm):
    """A prompt in one call and its continuation token by token give the whole sequence's outputs."""
    p = params(2)
    g = torch.Generator().manual_seed(3)
    x, res = (torch.randn(B, T, D, generator=g).cuda() for _ in range(2))
    torch.backends.cuda.matmul.allow_tf32 = False
    whole, _ = forward(sdm, p, x, res)
    conv_state = torch.zeros(B, K - 1, D, device="cuda")
    state = torch.zeros(B, D, N, device="cuda")
    cut = 40
    parts = [forward(sdm, p, x[:, :cut].contiguous(), res[:, :cut].contiguous(), conv_state, state)[0]]
    for t in range(cut, T):
        parts.append(forward(sdm, p, x[:, t:t + 1].contiguous(), res[:, t:t + 1].contiguous(), conv_state, state)[0])
    got = torch.cat(parts, 1)
    # library products of other shapes and other orders of the scan's sums: as above
    assert float((got - whole).abs().max()) <= 1e-4 * float(whole.abs().max())


def everything(sdm, p, x, res, dout):
    out, h, saved = forward(sdm, p, x, res, keep=True)
    dx, grads = backward(sdm, p, x, res, saved, h, dout)
    q, _ = sdm.rmsnorm_residual(x, p["norm"], res, out="fp8blk")
    (codes, scales), _ = sdm.rmsnorm_residual(x, p["norm"], res, out="fp8row")
    norm = sdm.grad_norm_clip([grads[k] for k in sorted(grads)], 1.0)
    return [out, dx, norm, sdm.dequantize_fp8blk(q, x.shape), sdm.dequantize_fp8row(codes, scales)] + [
        grads[k] for k in sorted(grads)]


def test_two_streams_at_once(sdm):
    """Calls on two streams at the same time give what each gives alone."""
    ps = [params(i) for i in range(2)]
    ins = [[torch.randn(B, T, D, generator=torch.Generator().manual_seed(9 * i + j)).cuda() for j in range(3)]
           for i in range(2)]
    alone = [everything(sdm, p, *i) for p, i in zip(ps, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = everything(sdm, ps[k], *ins[k])
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_captured_and_replayed(sdm):
    """A graph of forward, gradients and clipping replays on new inputs; two graphs do not share scratch."""
    p = params(4)
    ins = [torch.randn(B, T, D, generator=torch.Generator().manual_seed(j)).cuda() for j in range(3)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        everything(sdm, p, *ins)
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(everything(sdm, p, *ins))
    for t in ins:
        t.mul_(0.5).add_(0.1)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = everything(sdm, p, *ins)
    for got in outs:
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_captured_decode_carries_its_state(sdm):
    """The one-token form inside a graph: every replay advances the states."""
    p = params(5)
    x, res = (torch.randn(B, 1, D, generator=torch.Generator().manual_seed(j)).cuda() for j in range(2))
    c0, h0 = torch.zeros(B, K - 1, D, device="cuda"), torch.zeros(B, D, N, device="cuda")
    want, cs, hs = [], c0.clone(), h0.clone()
    for i in range(4):
        want.append(forward(sdm, p, x * (i + 1), res, cs, hs)[0].clone())
    live, c, h = x.clone(), c0.clone(), h0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = forward(sdm, p, live, res, c, h)
    c.copy_(c0)
    h.copy_(h0)
    for i in range(4):
        live.copy_(x * (i + 1))
        graph.replay()
        assert torch.equal(out, want[i])
    assert torch.equal(c, cs) and torch.equal(h, hs)


def test_front_end_refuses(sdm):
    x = torch.zeros(2, 3, 16, device="cuda")
    w, A = torch.zeros(16, device="cuda"), torch.zeros(16, 4, device="cuda")
    Bm = torch.zeros(2, 3, 1, 4, device="cuda")
    bad = [
        (ValueError, "must have shape", lambda: sdm.rmsnorm_residual(x, w[:8].contiguous())),
        (ValueError, "out must be", lambda: sdm.rmsnorm_residual(x, w, out="int8")),
        (ValueError, "contiguous", lambda: sdm.rmsnorm_residual(x.transpose(0, 1), w)),
        (TypeError, "float32 or bfloat16", lambda: sdm.rmsnorm_residual(x.half(), w)),
        (ValueError, "h needs a residual", lambda: sdm.rmsnorm_residual(x, w, h=x)),
        (ValueError, "not on cuda", lambda: sdm.rmsnorm_residual(x, w.cpu())),
        (sdm.SdmError, "multiple of 16", lambda: sdm.rmsnorm_residual(x[..., :8].contiguous(), w[:8].contiguous(),
                                                                     out="fp8blk")),
        (ValueError, "bytes", lambda: sdm.dequantize_fp8blk(torch.zeros(17, dtype=torch.uint8, device="cuda"), (32,))),
        (TypeError, "must be", lambda: sdm.rmsnorm_residual_backward(x, w, x, x.bfloat16())),
        (ValueError, r"\[D, K\]", lambda: sdm.short_conv(x, A.T)),
        (sdm.SdmError, "K must", lambda: sdm.short_conv(x, A[:, :1].contiguous())),
        (TypeError, "w's type", lambda: sdm.short_conv(x, A, w.bfloat16())),
        (ValueError, "shape", lambda: sdm.short_conv(x, A, state=torch.zeros(2, 4, 16, device="cuda"))),
        (TypeError, "int32", lambda: sdm.short_conv(x, A, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))),
        (sdm.SdmError, "overlaps", lambda: sdm.short_conv(x, A, y=x)),
        (ValueError, "behind its token axis", lambda: sdm.short_conv(
            torch.zeros(2, 3, 32, device="cuda")[..., ::2], A)),
        (ValueError, "evenly spaced", lambda: sdm.short_conv(torch.zeros(2, 9, 16, device="cuda")[:, :3], A)),
        (ValueError, "evenly spaced", lambda: sdm.short_conv(torch.zeros(2, 1, 16, device="cuda").expand(2, 3, 16), A)),
        (ValueError, r"\[B, T, G, N\]", lambda: sdm.selective_scan(x, x, A, Bm[..., :3], Bm)),
        (ValueError, "shape", lambda: sdm.selective_scan(x, x[:, :2].contiguous(), A, Bm, Bm)),
        (TypeError, "must be", lambda: sdm.selective_scan(x, x.bfloat16(), A, Bm, Bm)),
        (TypeError, "must be", lambda: sdm.selective_scan(x, x, A.bfloat16(), Bm, Bm)),
        (sdm.SdmError, "G must", lambda: sdm.selective_scan(x, x, A, Bm.expand(2, 3, 5, 4).contiguous(),
                                                           Bm.expand(2, 3, 5, 4).contiguous())),
        (ValueError, "outputs for", lambda: sdm.grad_norm_clip([w], 1.0, out=[w, w])),
        (ValueError, "no gradients", lambda: sdm.grad_norm_clip([], 1.0)),
        (ValueError, "values, its gradient", lambda: sdm.grad_norm_clip([w], 1.0, out=[A])),
        (ValueError, "contiguous", lambda: sdm.grad_norm_clip([A.T], 1.0)),
        (sdm.SdmError, "max_norm", lambda: sdm.grad_norm_clip([w], -1.0)),
    ]
    for kind, text, f in bad:
        with pytest.raises(kind, match=text):
            f()
    sdm.stream_check()
