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
