"""The selective scan's error bounds tell a scan whose splits are chained wrongly
from a right one (64-bit emulations on the CPU; the kernels are held to the same
bounds on the GPU)."""

import pytest
import torch

import block_reference as ref

B, T, D, G, SPLIT = 1, 700, 20, 2, 48


def inputs(N):
    g = torch.Generator().manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g).double()  # noqa: E731
    return dict(x=r(B, T, D), dt=r(B, T, D), Bm=r(B, T, G, N), Cm=r(B, T, G, N),
                A=-(torch.rand(D, N, generator=g).double() * 4 + 0.05), z=r(B, T, D), D=r(D), dt_bias=r(D) - 2,
                h0=r(B, D, N))


def in_splits(v, carry):
    """The scan in splits of SPLIT tokens; carry(state, start of the split, decay of the split) starts the next one."""
    h, ys = v["h0"], []
    for t in range(0, T, SPLIT):
        part = dict(v, **{k: v[k][:, t:t + SPLIT] for k in ("x", "dt", "Bm", "Cm", "z")}, h0=h)
        y, after = ref.scan(**part)
        alone = ref.scan(**dict(part, h0=None))[1]
        ys.append(y)
        h = carry(after, alone)
    return torch.cat(ys, 1), h


MISTAKES = {
    "each split starts from the one before alone": lambda after, alone: alone,
    "nothing is carried": lambda after, alone: torch.zeros_like(after),
    "a hundredth of what is carried is lost": lambda after, alone: alone + 0.99 * (after - alone),
}


@pytest.mark.parametrize("N", [4, 16, 24, 64])
def test_bounds_find_broken_chains(N):
    v = inputs(N)
    want, h = ref.scan(**v)
    by, bh = ref.scan_errors(**v)
    y, after = in_splits(v, lambda after, alone: after)
    assert bool(((y - want).abs() <= by).all()) and bool(((after - h).abs() <= bh).all())
    for name, carry in MISTAKES.items():
        y, _ = in_splits(v, carry)
        late = slice(SPLIT, None)
        assert bool(((y - want).abs() > 3 * by)[:, late].any()), name
    for k in (1.001, 0.999):
        assert bool(((k * want - want).abs() > by).any())
    # and they stay small against the terms themselves
    size = ref.scan(**v, absolute=True)[0]
    assert float((by / size).max()) < 2e-4
