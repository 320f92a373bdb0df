"""sample_logits where its definition is easily missed: thresholds above every weight."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", [40, 5000, 8192, 40001, 300000])
def test_min_p_above_one_keeps_the_first_alone(vocab, dtype):
    """No weight reaches it, and the first entry is kept always: of equal greatest logits the one of the least index,
    with probability 1.  At 1 all of them are kept."""
    import torch
    n = 8
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.randn((n, vocab), generator=gen, device="cuda").to(getattr(torch, dtype))
    for i in range(n):
        z[i, torch.randperm(vocab, generator=gen, device="cuda")[:9]] = 6.0
    u = torch.tensor([0.0, 0.3, 0.6, 0.9, 1 - 2.0 ** -24, 1.0, float("nan"), -1.0], device="cuda")
    above = [float(np.nextafter(np.float32(1), np.float32(2))), 1.5, 7.0, float("inf")]
    first = (z == 6.0).int().argmax(1)
    for min_p in above + [torch.tensor(above * 2, device="cuda")]:
        probs = torch.full(z.shape, -1.0, device="cuda")
        tokens = wsl.sample_logits(z, u, min_p=min_p, temperature=0.7, probs=probs)
        assert tokens.equal(first.int()), min_p
        assert probs.equal(torch.nn.functional.one_hot(first, vocab).float())
        assert wsl.sample_logits(z, min_p=min_p, top_k=5, top_p=0.9).equal(probs)
    mixed = torch.tensor([1.0, 1.5] * 4, device="cuda")
    probs = wsl.sample_logits(z, min_p=mixed)
    assert (probs > 0).sum(1).tolist() == [9, 1] * 4
    for i in range(n):
        assert (ref.sample_ref(f32_of(z[i]), min_p=float(mixed[i]))[1] > 0).tolist() == (probs[i] > 0).tolist()
