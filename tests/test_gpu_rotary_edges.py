"""rotary_embed far from the origin, against angles that lose nothing."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of
from gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,far", [(size, far) for far in (0, 12, 22) for size in (20, 28, 30, 34, 38, 40)] + [(48, 0), (48, 14)])
def test_cos_and_sin_of_any_position(size, far):
    """The pair (1, 0) turns to (cos, sin): |p f| up to 2^size, of positions up to 2^(size + far), which a double
    does not hold from 2^53 on.  Each is rounded once to binary32 (half a step below 1: 2^-25), after a series and
    a reduction that are off by less than 2^-32."""
    import torch
    say(f"rotary |p f| < 2^{size}, p < 2^{size + far}")
    g = np.random.default_rng([2026, 31, size, far])
    top = 1 << (size + far)
    positions = [top - 1, -top + 1, top - 12345, *(int(x) for x in g.integers(top // 2, top, 20)), *(-int(x) for x in g.integers(top // 2, top, 9))]
    freqs = [float(x) for x in 2.0 ** -far * g.uniform(0.1, 1.0, 14)] + [2.0 ** -far, 2.0 ** -far / 3]
    x = torch.zeros((len(positions), 1, 32), device="cuda")
    at, f = torch.tensor(positions, device="cuda"), torch.tensor(freqs, dtype=torch.float64, device="cuda")
    cos, sin = ref.turn_ref(positions, freqs)
    for interleaved in (False, True):
        x.zero_()
        (x[..., 0::2] if interleaved else x[..., :16]).fill_(1.0)
        y = f32_of(wsl.rotary_embed(x, at, f, interleaved=interleaved))[:, 0]
        c, s = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :16], y[:, 16:])
        assert np.abs(c - cos).max() <= 2.0 ** -25 + 2.0 ** -32
        assert np.abs(s - sin).max() <= 2.0 ** -25 + 2.0 ** -32


def test_turns_of_positions_that_differ_by_one():
    """Next to 2^60 neighbours are turned by their difference: rounded positions would be the same."""
    import torch
    positions, freqs = [(1 << 60) + i for i in range(-3, 4)], [2.0 ** -20, 2.0 ** -24 / 3]
    x = torch.zeros((7, 2, 16), device="cuda")
    x[..., :2] = 1.0
    y = f32_of(wsl.rotary_embed(x, torch.tensor(positions, device="cuda"), torch.tensor(freqs, dtype=torch.float64, device="cuda")))
    cos, sin = ref.turn_ref(positions, freqs)
    for h in range(2):
        assert np.abs(y[:, h, :2] - cos).max() <= 2.0 ** -25 + 2.0 ** -32 and np.abs(y[:, h, 2:4] - sin).max() <= 2.0 ** -25 + 2.0 ** -32


def test_positions_of_another_shape():
    """Flat positions of [n_seq][q_len] tokens are theirs in order; transposed ones are refused, not misread."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, freqs = torch.randn((3, 5, 4, 64), generator=gen, device="cuda"), wsl.rotary_freqs(64)
    at = torch.randint(0, 1000, (3, 5), generator=gen, device="cuda")
    want = wsl.rotary_embed(q, at, freqs)
    assert wsl.rotary_embed(q, at.view(-1), freqs).equal(want)
    assert wsl.rotary_embed(q.flatten(0, 1), at, freqs).equal(want.flatten(0, 1))
    assert wsl.rotary_embed(q, at[..., None], freqs).equal(want)
    for bad in (at.t().contiguous(), at[:2], at.view(-1)[:14], at.t(), at.int()):
        with pytest.raises(ValueError, match="positions"):
            wsl.rotary_embed(q, bad, freqs)
