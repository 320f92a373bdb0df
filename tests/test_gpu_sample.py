"""sample_logits on the GPU against rows sorted in 64 bits."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of
from gpu_common import say

pytestmark = pytest.mark.gpu

OFF = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def _row(how, i):
    import torch
    return {x: float(np.float32(v[i].item() if torch.is_tensor(v) else v)) if x != "top_k" else
            int(v[i] if torch.is_tensor(v) else v) for x, v in {**OFF, **how}.items()}


def _check(z, u, status=None, probs_too=True, **how):
    """Tokens equal; probabilities zero where the definition's are, and right to fp32's half step and what
    their sum is off: a weight between 2^-(1/16) and 2^(1/16) of its unit, rounded to whole 2^-32 of it, is
    off by 2^-33 * 2^(1/16) of itself at most, its series by 2^-36 (0.0434^6 / 720): 2^-32.7 together, and
    so is a sum of them; the quotient's weight and division by 2^-49."""
    import torch
    probs = torch.full(z.shape, -1.0, device="cuda") if probs_too else None
    tokens = wsl.sample_logits(z, u, probs=probs, status=status, **how)
    if probs_too:
        assert wsl.sample_logits(z, u, **how).equal(tokens)
        assert wsl.sample_logits(z, **how).equal(probs)
    z64, uu = f32_of(z), u.cpu().numpy()
    for i in range(len(z64)):
        token, want = ref.sample_ref(z64[i], float(uu[i]), **_row(how, i))
        assert tokens[i].item() == token, (i, _row(how, i))
        if probs_too:
            got = probs[i].cpu().numpy().astype(np.float64)
            assert ((got > 0) == (want > 2.0 ** -150)).all(), (i, _row(how, i))
            assert (np.abs(got - want) <= want * (2.0 ** -24 + 2.0 ** -32) + 2.0 ** -150).all()
    return tokens


def _logits(seed, n, vocab, dtype, spread=2.5, pad=0, peaks=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = spread * torch.randn((n, vocab + pad), generator=gen, device="cuda")
    if peaks:
        z.scatter_add_(1, torch.randint(0, vocab, (n, peaks), generator=gen, device="cuda"),
                       4 * spread * torch.rand((n, peaks), generator=gen, device="cuda"))
    return z.to(getattr(torch, dtype))[:, :vocab], torch.rand(n, generator=gen, device="cuda")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,vocab,pad", [(3, 1, 0), (5, 2, 3), (4, 63, 0), (7, 1000, 1), (3, 1024, 0), (3, 1025, 2), (2, 4097, 0),
                                         (2, 8192, 5), (4, 32000, 0), (2, 32768, 0), (2, 32769, 1), (3, 50257, 0),
                                         (2, 65536, 0), (2, 151937, 3)])
def test_settings_against_the_definition(n, vocab, pad, dtype):
    say(f"sample n={n} vocab={vocab} pad={pad} {dtype}")
    for seed, how in enumerate([
            {}, dict(temperature=0.0), dict(temperature=0.7, top_k=1), dict(top_k=2), dict(top_k=50, temperature=1.3),
            dict(top_k=300), dict(top_k=vocab - 1 or 1), dict(top_k=vocab // 2 + 1, temperature=0.4), dict(top_p=0.9),
            dict(top_p=0.1, temperature=2.0), dict(top_p=0.999), dict(min_p=0.05), dict(min_p=1.0), dict(min_p=1e-6),
            dict(top_k=40, top_p=0.95, min_p=0.02, temperature=0.8), dict(top_k=2000, top_p=0.5, temperature=3.0)]):
        z, u = _logits(100 * vocab + seed, n, vocab, dtype, pad=pad, peaks=seed % 3)
        _check(z, u, probs_too=seed % 2 == 0 or vocab < 5000, **how)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,vocab,pad", [(2, 4096, 1), (2, 8193, 0), (2, 16385, 0), (1, 131072, 0), (2, 131073, 3), (1, 262144, 0),
                                         (2, 262145, 1), (1, 400000, 0)])
def test_where_parts_begin_and_end(n, vocab, pad, dtype):
    """Rows at the ends of what one workgroup, a part, and a table of parts hold."""
    for seed, how in enumerate([dict(top_k=300, top_p=0.9, temperature=0.9), dict(top_p=0.97), dict(min_p=0.001, temperature=0.8), {}]):
        z, u = _logits(vocab + seed, n, vocab, dtype, pad=pad, peaks=seed % 2)
        z[0, vocab - 1] = z[0].max() + 1        # the last entry is the greatest
        _check(z, u, probs_too=seed < 2, **how)


def test_settings_where_few_are_kept_far_apart():
    """Borders in cells that are empty, or hold one entry, over parts whose greatest entries differ by far."""
    import torch
    vocab = 60000
    z = torch.full((3, vocab), -400.0, device="cuda")
    z[:, 5], z[:, 20000], z[:, 59999] = 10.0, 9.0, -30.0
    z[1, 30000:34000] = torch.linspace(-60, 5, 4000, device="cuda")
    z[2, 100::7] = float("-inf")
    u = torch.tensor([0.2, 0.9, 0.99999], device="cuda")
    for how in (dict(top_k=2), dict(top_k=3), dict(top_k=50), dict(top_p=0.99), dict(top_p=1 - 2.0 ** -24), dict(min_p=0.3), dict(min_p=0.4),
                dict(min_p=1e-30), dict(top_k=30000, top_p=0.9999999), dict(top_k=4, min_p=1e-38, temperature=3.0),
                dict(temperature=40.0, top_k=59000), dict(temperature=200.0, top_p=0.9)):
        _check(z, u, **how)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", [777, 40001])
def test_settings_of_each_row(vocab, dtype):
    import torch
    n = 24
    z, u = _logits(vocab, n, vocab, dtype, spread=3.0, peaks=3)
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    pick = lambda values, dt: torch.tensor(values, dtype=dt, device="cuda")[torch.randint(0, len(values), (n,), generator=gen, device="cuda")]
    nan = float("nan")
    how = dict(temperature=pick([0.0, -1.0, nan, 0.3, 1.0, 2.5], torch.float32), top_k=pick([-5, 0, 1, 7, 300, 1 << 30], torch.int32),
               top_p=pick([-1.0, 0.0, 0.3, 0.9, 1.0, 2.0, nan], torch.float32), min_p=pick([-1.0, 0.0, 0.01, 0.5, 1.0, 7.0, nan], torch.float32))
    _check(z, u, **how)
    for name in how:
        _check(z, u, **{name: how[name]})


@pytest.mark.parametrize("vocab", [1024, 5000, 32768, 70000])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_equal_logits_go_by_their_index(vocab, dtype):
    """All weights are one: what is kept is the first k, or as many as p asks for, and the token is
    the u-th of them.  Sums are whole numbers: exact."""
    import torch
    z = torch.full((1, vocab), -3.75, dtype=getattr(torch, dtype), device="cuda")
    for k in (1, 2, 255, 256, 257, 1000, vocab - 1, vocab, vocab + 7):
        kept = min(k, vocab)
        p = wsl.sample_logits(z, top_k=k)[0]
        assert (p[:kept] == np.float32(1.0 / kept)).all() and (p[kept:] == 0).all()
        for u in (0.0, 0.25, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, float("nan"), -1.0):
            t = wsl.sample_logits(z, torch.tensor([u], device="cuda"), top_k=k).item()
            assert t == (min(int(max(u, 0.0) * kept), kept - 1) if u == u else kept - 1)
    for top_p in (0.5, 0.25, 0.75, 2.0 ** -10):
        kept = int(np.ceil(top_p * vocab))
        p = wsl.sample_logits(z, top_p=top_p)[0]
        assert (p[:kept] > 0).all() and (p[kept:] == 0).all()
        p = wsl.sample_logits(z, top_p=top_p, top_k=vocab // 2)[0]
        kept = int(np.ceil(top_p * (vocab // 2)))
        assert (p[:kept] > 0).all() and (p[kept:] == 0).all()
    assert (wsl.sample_logits(z, min_p=1.0) > 0).all()


@pytest.mark.parametrize("vocab", [3000, 40000])
def test_a_few_values_with_many_ties(vocab):
    """Whole logits from a handful of values, zeros of both signs, the border inside each of them."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.randint(-3, 4, (2, vocab), generator=gen, device="cuda").float()
    z[z == 0] *= torch.where(torch.rand(int((z == 0).sum()), generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    z[:, 17] = 3.0
    u = torch.rand(2, generator=gen, device="cuda")
    for k in (1, 2, vocab // 8, vocab // 3, vocab // 2, vocab - 3):
        _check(z, u, top_k=k, temperature=1.7)
        _check(z, u, top_k=k, top_p=0.8, temperature=1.7)
    for p in (0.05, 0.3, 0.62, 0.97, 0.9999):
        _check(z, u, top_p=p)


@pytest.mark.parametrize("vocab", [1500, 33000])
def test_masked_and_far_entries(vocab):
    """-infinity is out of the row; the type's lowest value, and logits far from each other, are in it."""
    import torch
    z, u = _logits(vocab, 6, vocab, "float32")
    inf, low = float("inf"), torch.finfo(torch.float32).min
    z[0, ::2] = -inf
    z[1, 1:] = -inf                              # one is left
    z[2, :] = low                                # all equal
    z[3, 5:] = low
    z[4, :] = torch.linspace(-3e38, 3e38, vocab, device="cuda")
    z[5, :700] += 1000.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for how in ({}, dict(top_k=20), dict(top_k=vocab - 2), dict(top_p=0.9), dict(min_p=0.1), dict(top_k=1000, top_p=0.9),
                dict(temperature=1e-30), dict(temperature=1e-45, top_k=9), dict(temperature=1e30, top_p=0.5),
                dict(temperature=inf, top_k=700), dict(temperature=5e-3, top_p=0.99)):
        _check(z, u, status=st, **how)
    # (linspace over more than the largest number leaves fp32: row 4 is one that cannot be sampled)
    unfit = bool((torch.isnan(z) | (z == inf)).any())
    assert st.item() == (wsl.WSL_STATUS_NONFINITE if unfit else 0)


@pytest.mark.parametrize("vocab", [1500, 33000])
def test_entries_all_over_the_range(vocab):
    import torch
    z = torch.linspace(-1.5e38, 1.5e38, vocab, device="cuda")[None].contiguous()
    z[0, 7], z[0, 8], z[0, 9] = 3.4e38, 1e-40, -3.4e38
    assert bool(torch.isfinite(z).all())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = torch.tensor([0.7], device="cuda")
    for how in ({}, dict(top_k=20), dict(top_k=vocab - 2), dict(top_p=0.9), dict(temperature=1e38, top_p=0.5),
                dict(temperature=3e38, top_k=vocab // 2), dict(temperature=float("inf"), top_k=700)):
        _check(z, u, status=st, **how)
    assert st.item() == 0


def test_a_tail_that_is_far_below_but_heavy():
    """One entry, and 2^16 others of 2^-33 each: u picks the tail where it should, and top-p reaches into it."""
    import torch
    vocab = 1 << 16
    z = torch.full((1, vocab), -33.0, device="cuda")
    z[0, 4321] = 0.0
    t = float(np.float32(1 / np.log(2)))
    one = wsl.sample_logits(z, torch.tensor([0.999], device="cuda"), temperature=t)
    assert one.item() == 4321
    _check(z, torch.tensor([1 - 2.0 ** -24], device="cuda"), temperature=t)
    _check(z, torch.tensor([0.0], device="cuda"), temperature=t)
    for p in (1 - 2.0 ** -17, 1 - 2.0 ** -18, 0.5):
        _check(z, torch.tensor([0.5], device="cuda"), temperature=t, top_p=p)


@pytest.mark.parametrize("vocab", [100, 2049, 32768, 50000])
def test_rows_that_cannot_be_sampled(vocab):
    import torch
    z, u = _logits(vocab, 5, vocab, "float32")
    z[0, vocab - 1] = float("nan")
    z[2, 3] = float("inf")
    z[3, :] = float("-inf")
    for how in ({}, dict(temperature=0.0), dict(top_k=5), dict(top_p=0.5)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = _check(z, u, status=st, **how)
        assert (t < 0).tolist() == [True, False, True, True, False] and st.item() == wsl.WSL_STATUS_NONFINITE


def test_many_rows_and_strides():
    import torch
    z, u = _logits(3, 700, 300, "float32", pad=11)
    _check(z, u, top_p=0.8, top_k=30)
    wide = torch.full((700, 320), 7.0, device="cuda")
    probs = wide[:, :300]
    tokens = torch.full((700,), -3, dtype=torch.int32, device="cuda")
    got = wsl.sample_logits(z, u, top_p=0.8, probs=probs, tokens=tokens)
    assert got is tokens and (wide[:, 300:] == 7.0).all() and ((probs.sum(1) - 1).abs() < 1e-5).all()
    one = wsl.sample_logits(z[5:6], u[5:6], top_p=0.8)
    assert one.item() == tokens[5].item()


@pytest.mark.parametrize("n,vocab", [(300, 3900), (300, 8000), (200, 32001), (70, 100003)])
def test_many_rows_at_once_are_as_few(n, vocab):
    """So many rows that waves or parts are others: probabilities as of one row (both right to 2^-32, then rounded),
    and tokens inside of them."""
    import torch
    z, u = _logits(vocab, n, vocab, "float32", peaks=2)
    how = dict(top_k=400, top_p=0.93, temperature=0.8)
    probs = torch.empty((n, vocab), device="cuda")
    tokens = wsl.sample_logits(z, u, probs=probs, **how)
    assert (probs.gather(1, tokens.long()[:, None]) > 0).all()
    for r in (0, n // 2, n - 1):
        one = torch.empty((1, vocab), device="cuda")
        wsl.sample_logits(z[r:r + 1], u[r:r + 1], probs=one, **how)
        assert (one[0] > 0).equal(probs[r] > 0)
        assert ((one[0] - probs[r]).abs() <= 2.0 ** -23 * 1.001 * one[0]).all()
    _check(z[:3], u[:3], **how)
    for r in (0, n - 1):
        _check(z[r:r + 1], u[r:r + 1], **how)


def test_a_long_row():
    import torch
    z, u = _logits(8, 1, 1 << 22, "bfloat16")
    _check(z, u, probs_too=True, top_p=0.9, top_k=100000)
    _check(z, u, probs_too=False)


def test_verification_takes_the_distribution():
    """Drafts sampled from q's filtered distribution; verify_drafts over both sides' distributions.  Where they
    are the same every draft stands."""
    import torch
    n, width, vocab = 6, 3, 2000
    z, u = _logits(4, n * (width + 1), vocab, "float32")
    p = wsl.sample_logits(z, top_p=0.9, temperature=0.8).view(n, width + 1, vocab)
    q = p[:, :width].contiguous()
    drafts = wsl.sample_logits(z, u, top_p=0.9, temperature=0.8).view(n, width + 1)[:, :width].contiguous()
    accepted, tokens = wsl.verify_drafts(p, q, drafts, torch.full((n, width + 1), 0.5, device="cuda"))
    assert (accepted == width).all() and (p.gather(2, tokens.long()[..., None]) > 0).all()


def test_a_graph_and_a_stream():
    import torch
    z, u = _logits(6, 4, 40000, "float32")
    out = torch.empty(4, dtype=torch.int32, device="cuda")
    nb = wsl.sample_logits_workspace_bytes(4, 40000)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wsl.sample_logits(z, u, top_p=0.9, top_k=500, tokens=out, workspace=ws)
        z.mul_(0.9)
    for _ in range(4):
        want = wsl.sample_logits(z, u, top_p=0.9, top_k=500)
        ws.fill_(255)
        graph.replay()
        assert out.equal(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = wsl.sample_logits(z, u, top_p=0.9, top_k=500, stream=s)
    s.synchronize()
    assert other.equal(wsl.sample_logits(z, u, top_p=0.9, top_k=500))
