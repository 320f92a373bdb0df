"""The cache, attention and verification calls together, as examples/speculative_decode.py uses them."""

import importlib.util
import os

import pytest

import weight_streaming_linear_amd as wsl

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", [wsl.WSL_KV_BF16, wsl.WSL_KV_E4M3])
@pytest.mark.parametrize("width", [0, 1, 4])
def test_a_drafter_that_is_the_target_is_always_believed(fmt, width):
    """The drafter computes its probabilities token by token, the target all of them in one sweep over
    the same weights: with u = 1/2 a draft falls only if the two differ by a factor of two."""
    import torch
    ex = _example()
    kw = dict(layers=2, hidden=512, heads=8, n_kv=2, ffn=1024, vocab=1000, capacity=256, page=16, fmt=fmt)
    target, drafter = (ex.Decoder(3, **kw) for _ in range(2))
    prompt = torch.randint(0, 1000, (3, 70), device="cuda", dtype=torch.int32,
                           generator=torch.Generator(device="cuda").manual_seed(3))
    added, stood = ex.decode(target, drafter, prompt, width, 5, lambda n, m: torch.full((n, m), 0.5, device="cuda"))
    assert (stood == width).all()
    assert added.shape == (5, 3, width + 1) and (added >= 0).all() and (added < 1000).all()


def test_a_drafter_that_is_not_the_target():
    """Tokens after the last that stands are -1, and the next round goes on from there."""
    import torch
    ex = _example()
    kw = dict(hidden=512, heads=8, n_kv=2, ffn=1024, vocab=1000, capacity=256, page=16)
    target, drafter = ex.Decoder(2, layers=2, **kw), ex.Decoder(2, layers=1, seed=5, **kw)
    gen = torch.Generator(device="cuda").manual_seed(4)
    prompt = torch.randint(0, 1000, (2, 40), device="cuda", dtype=torch.int32, generator=gen)
    added, stood = ex.decode(target, drafter, prompt, 3, 8, lambda n, m: torch.rand((n, m), generator=gen, device="cuda"))
    there = torch.arange(4, device="cuda") <= stood[..., None]
    assert torch.equal(added >= 0, there) and (stood < 3).any()
