"""lora_add where numbers come near the end of their type's range."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [3, 1100])
@pytest.mark.parametrize("rank", [8, 16, 40, 64, 128])
def test_sums_next_to_the_largest_number(m, rank):
    """A x is finite, and above what rounds to bf16's largest: the result is what the formula gives, over tokens one by one
    and over tiles of them."""
    import torch
    bf, n_out, k = torch.bfloat16, 70, 64
    a, b = torch.zeros((2, rank, k), device="cuda"), torch.zeros((2, n_out, rank), device="cuda")
    a[:, :, 0], a[0, :, 1], a[1, :, 1] = float(torch.finfo(bf).max), 1e36, -1e36
    b[:, torch.arange(n_out), torch.arange(n_out) % rank] = 2.0 ** -120
    x = torch.zeros((m, k), device="cuda")
    x[:, :2] = 1.0
    x[1::2] *= -1.0
    x, a, b = x.to(bf), a.to(bf), b.to(bf)
    ids = torch.arange(m, device="cuda").to(torch.int32) % 3 - 1
    base = torch.randn((m, n_out), device="cuda", generator=torch.Generator(device="cuda").manual_seed(rank))
    out = wsl.lora_add(base, x, a, b, ids)
    want, bound = ref.lora_ref(f32_of(base), f32_of(x), f32_of(a), f32_of(b), ids.tolist())
    assert (np.abs(f32_of(out) - want) <= bound).all()
