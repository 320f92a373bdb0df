"""Calls at the edges of what the cache, attention and verification calls take, on the GPU."""

import numpy as np
import pytest

import oracle.decode as od
import weight_streaming_linear_amd as wsl
from decode_cases import CacheCase, f32_of, probabilities
from gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,width", [(2, 3), (1, 3), (4, 1), (1, 1)])
@pytest.mark.parametrize("vocab", [501, 40009])
def test_a_drafter_with_one_distribution_for_every_position(n, width, vocab):
    """A broadcast q is refused, never taken for no q at all; copied out it gives what the definition does."""
    import torch
    say(f"verify, one q for all: n={n} width={width} vocab={vocab}")
    g = np.random.default_rng([2026, 12, n, width])
    p = torch.from_numpy(probabilities(g, n, width + 1, vocab)).cuda()
    one = torch.from_numpy(probabilities(g, 1, 1, vocab)).cuda()
    q = one.expand(n, width, vocab)
    drafts = torch.from_numpy(g.integers(0, vocab, (n, width)).astype(np.int32)).cuda()
    u = torch.from_numpy(g.random((n, width + 1)).astype(np.float32)).cuda()
    if n * width > 1:
        for a, b in ((p, q), (p[:1, :1].expand(n, width + 1, vocab), q.contiguous())):
            with pytest.raises(ValueError):
                wsl.verify_drafts(a, b, drafts, u)
    acc, tok = wsl.verify_drafts(p, q.contiguous(), drafts, u)
    for b in range(n):
        r, t = od.verify_ref(f32_of(p)[b], f32_of(q)[b], drafts[b].cpu().numpy(), u[b].cpu().numpy(), width, vocab)
        assert acc[b].item() == r and np.array_equal(tok[b].cpu().numpy(), t)
