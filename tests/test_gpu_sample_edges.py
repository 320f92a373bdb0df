"""sample_logits where its definition is easily missed: thresholds above every weight, rows cut in other ways."""

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


@pytest.mark.parametrize("n,vocab", [(300, 3900), (300, 8000), (200, 32001), (520, 9000), (300, 131072), (70, 100003)])
def test_a_rows_token_does_not_depend_on_the_rows_beside_it(n, vocab):
    """Among many rows parts are longer, or waves fewer; sums agree to 2^-32, and so a u in the middle of an entry's share
    of 2^-20 or more (rounded to fp32: 2^-25) gives that entry, alone and among the others."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(vocab + n)
    z = 2.5 * torch.randn((n, vocab), generator=gen, device="cuda")
    how = dict(top_k=400, top_p=0.93, temperature=0.8)
    rows = [0, 1, n // 3, n // 2, n - 1]
    u = torch.rand(n, generator=gen, device="cuda")
    want = {}
    for r in rows:
        probs = ref.sample_ref(f32_of(z[r]), **{x: float(np.float32(v)) if x != "top_k" else v for x, v in how.items()})[1]
        up = np.cumsum(probs)
        at = int(np.searchsorted(up, u[r].item(), side="right"))
        if at >= vocab or probs[at] < 2.0 ** -20:
            at = int(probs.argmax())
        u[r], want[r] = float(up[at] - probs[at] / 2), at
    tokens = wsl.sample_logits(z, u, **how)
    for r in rows:
        alone = wsl.sample_logits(z[r:r + 1], u[r:r + 1], **how)
        assert alone.item() == tokens[r].item() == want[r]
    assert wsl.sample_logits(z, u, **how).equal(tokens)
