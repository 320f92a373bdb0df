"""rotary_embed on the GPU against a complex multiplication in 64 bits and more."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of
from gpu_common import say

pytestmark = pytest.mark.gpu


def _check(out, x, positions, freqs, interleaved, amplitude):
    import torch
    x64, f, p = f32_of(x), freqs.cpu().numpy(), positions.cpu().numpy().reshape(-1)
    x64 = x64.reshape(-1, *x64.shape[-2:])
    want, parts = ref.rotary_ref(x64, p, f, interleaved, amplitude)
    bound = ref.rotary_bound(x64, want, parts, p, f, interleaved, amplitude, out.dtype is torch.bfloat16)
    off = np.abs(f32_of(out).reshape(want.shape) - want)
    assert (off <= bound).all(), (off - bound).max()
    if out.dtype is x.dtype:
        assert out[..., 2 * len(f):].equal(x[..., 2 * len(f):])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot", [
    (1, 40, 8, 128, 128), (3, 1, 1, 16, 2), (2, 3, 1, 48, 10), (65, 8, 2, 64, 64), (7, 12, 3, 80, 40), (5, 2, 2, 96, 48),
    (9, 6, 1, 256, 256), (4, 5, 5, 192, 64), (33, 16, 4, 112, 112), (2, 300, 1, 32, 16), (513, 2, 1, 128, 32)])
@pytest.mark.parametrize("src,dst", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "bfloat16"),
                                     ("bfloat16", "float32")])
def test_against_the_formula(tokens, heads, kv, dim, rot, interleaved, src, dst):
    """Views of a fused projection, far positions, parts of heads."""
    import torch
    say(f"rotary {tokens}x{heads}+{kv}x{dim}/{rot} interleaved={interleaved} {src}->{dst}")
    gen = torch.Generator(device="cuda").manual_seed(tokens * 1000 + dim + rot)
    x = torch.randn((tokens, (heads + 2 * kv) * dim), generator=gen, device="cuda").mul_(3).to(getattr(torch, src))
    q, k = x[:, :heads * dim].unflatten(-1, (heads, dim)), x[:, heads * dim:(heads + kv) * dim].unflatten(-1, (kv, dim))
    positions = torch.randint(0, 1 << 20, (tokens,), generator=gen, device="cuda")
    freqs = wsl.rotary_freqs(rot)
    ofmt = wsl.WSL_OUT_F32 if dst == "float32" else wsl.WSL_OUT_BF16
    a, b = wsl.rotary_embed(q, positions, freqs, k=k, interleaved=interleaved, amplitude=1.25, ofmt=ofmt)
    assert a.dtype is b.dtype is getattr(torch, dst) and a.is_contiguous() and b.is_contiguous()
    _check(a, q, positions, freqs, interleaved, 1.25)
    _check(b, k, positions, freqs, interleaved, 1.25)
    alone = wsl.rotary_embed(q, positions, freqs, interleaved=interleaved, amplitude=1.25, ofmt=ofmt)
    assert alone.equal(a)


def test_positions_near_and_far():
    """0, -1, and up to 2^40 where a frequency is one: the angle keeps its turn."""
    import torch
    positions = torch.tensor([0, 1, -1, -1000003, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 40 - 1], device="cuda")
    x = torch.randn((8, 2, 64), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    freqs = torch.cat((torch.tensor([1.0, 0.0, 0.5, 3.0], dtype=torch.float64, device="cuda"), wsl.rotary_freqs(56)))
    for interleaved in (False, True):
        _check(wsl.rotary_embed(x, positions, freqs, interleaved=interleaved), x, positions, freqs, interleaved, 1.0)
    # position 0 turns nothing
    assert wsl.rotary_embed(x, torch.zeros_like(positions), freqs).equal(x)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 24, 10])
def test_in_place_in_four_dimensions(dtype, interleaved, rot):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rot)
    wide = torch.randn((3, 5, 20 * 64), generator=gen, device="cuda").to(getattr(torch, dtype))
    kept = wide.clone()
    q, k = wide[..., :12 * 64].unflatten(-1, (12, 64)), wide[..., 12 * 64:16 * 64].unflatten(-1, (4, 64))
    positions = torch.randint(0, 5000, (3, 5), generator=gen, device="cuda")
    freqs = wsl.rotary_freqs(rot, base=500000.0)
    want = wsl.rotary_embed(q, positions, freqs, k=k, interleaved=interleaved)
    got = wsl.rotary_embed(q, positions, freqs, k=k, interleaved=interleaved, out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert q.equal(want[0]) and k.equal(want[1]) and wide[..., 16 * 64:].equal(kept[..., 16 * 64:])


def test_turning_back_and_by_differences():
    """Turned by p and by -p a head is itself, and <turned q, turned k> depends on the distance alone."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, y = (torch.randn((50, 3, 128), generator=gen, device="cuda") for _ in range(2))
    freqs = wsl.rotary_freqs(128, scaling="bands", factor=8.0, trained=4096)
    at = torch.randint(0, 100000, (50,), generator=gen, device="cuda")
    back = wsl.rotary_embed(wsl.rotary_embed(x, at, freqs), -at, freqs)
    # two turns, each off by at most 3 * 2^-24 (|a| + |b|) and a little; a turn keeps |a|, |b| <= |a| + |b|
    bound = 2 * 3.1 * 2 ** -24 * (x[..., :64].abs() + x[..., 64:].abs()) * 2
    assert ((back - x).abs() <= bound.repeat(1, 1, 2)).all()
    dot = lambda p, q: (wsl.rotary_embed(x, p, freqs).double() * wsl.rotary_embed(y, q, freqs).double()).sum(-1)
    near, far = dot(at, at + 7), dot(at + 1000, at + 1007)
    size = x.double().norm(dim=-1) * y.double().norm(dim=-1)
    assert ((near - far).abs() <= 4 * 4 * 2 ** -24 * 2 ** 0.5 * size).all()


def test_more_tokens_than_workgroups():
    """Past 2^20 tokens each workgroup goes on with further ones."""
    import torch
    n = (1 << 20) + 3
    x = torch.randn((n, 1, 16), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(torch.bfloat16)
    at, freqs = torch.arange(n, device="cuda"), wsl.rotary_freqs(16)
    out = wsl.rotary_embed(x, at, freqs)
    some = torch.cat((torch.arange(5), torch.arange(n - 5, n))).cuda()
    _check(out[some], x[some], at[some], freqs, False, 1.0)
    assert out[: 1 << 19].equal(wsl.rotary_embed(x[: 1 << 19], at[: 1 << 19], freqs))


def test_empty_and_infinite():
    import torch
    freqs = wsl.rotary_freqs(32)
    none = torch.empty((0, 2, 32), device="cuda")
    assert wsl.rotary_embed(none, torch.empty(0, dtype=torch.int64, device="cuda"), freqs).shape == (0, 2, 32)
    x = torch.ones((2, 1, 48), device="cuda")
    x[0, 0, 40], x[1, 0, 47] = float("nan"), float("inf")       # behind what is turned
    x[1, 0, 3] = float("inf")
    out = wsl.rotary_embed(x, torch.tensor([3, 3], device="cuda"), freqs)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[0, 0, 40], [1, 0, 3], [1, 0, 19], [1, 0, 47]]


def test_a_stream_of_its_own_and_a_graph():
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((6, 4, 64), generator=gen, device="cuda")
    at, freqs = torch.arange(6, device="cuda"), wsl.rotary_freqs(64)
    want = wsl.rotary_embed(q, at, freqs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = wsl.rotary_embed(q, at, freqs, stream=s)
    s.synchronize()
    assert other.equal(want)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wsl.rotary_embed(q, at, freqs, out=out)
        at.add_(1)
    for i in range(4):
        graph.replay()
        assert out.equal(wsl.rotary_embed(q, torch.arange(6, device="cuda") + i, freqs))
