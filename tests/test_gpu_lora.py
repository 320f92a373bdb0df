"""lora_add on the GPU against two products a row in 64 bits."""

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of
from gpu_common import say

pytestmark = pytest.mark.gpu


def _case(seed, m, k, n_out, rank, count, dtype, pad=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = r(m, k + 8 * pad).to(torch.bfloat16)[:, :k]
    base = (2 * r(m, n_out + pad)).to(getattr(torch, dtype))[:, :n_out]
    a, b = (r(count, rank, k) * k ** -0.5).to(torch.bfloat16), (r(count, n_out, rank) * rank ** -0.5).to(torch.bfloat16)
    ids = torch.randint(-1, count, (m,), generator=gen, device="cuda", dtype=torch.int32)
    return base, x, a, b, ids, 0.5 + torch.rand(count, generator=gen, device="cuda")


def _check(base, x, a, b, ids, scales, out):
    import torch
    want, bound = ref.lora_ref(f32_of(base), f32_of(x), f32_of(a), f32_of(b), ids.tolist(),
                               None if scales is None else scales.tolist())
    if out.dtype is torch.bfloat16:
        bound = bound + ref.HALF_BF16 * (np.abs(want) + bound)
    off = np.abs(f32_of(out) - want)
    assert (off <= bound).all(), (off - bound).max()
    none = (ids < 0) | (ids >= len(a))
    assert out[none].equal(base[none])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,k,n_out,rank,count,pad", [
    (1, 8, 1, 8, 1, 0), (1, 512, 640, 16, 3, 0), (5, 520, 333, 24, 2, 1), (48, 1024, 257, 32, 40, 0), (3, 4096, 100, 64, 2, 3),
    (64, 136, 700, 128, 5, 0), (65, 136, 700, 128, 5, 0), (17, 2000, 515, 40, 3, 1), (66, 1000, 333, 8, 70, 1),
    (130, 512, 1040, 16, 3, 0), (200, 2056, 64, 56, 4, 0), (300, 768, 130, 32, 1, 2), (100, 1536, 515, 104, 9, 0),
    (1100, 264, 130, 8, 3, 0), (520, 512, 1040, 16, 3, 0), (530, 2056, 70, 16, 70, 1), (700, 1544, 129, 24, 4, 0),
    (130, 640, 200, 64, 3, 0), (70, 1160, 333, 128, 2, 4)])
def test_against_the_formula(m, k, n_out, rank, count, pad, dtype):
    say(f"lora m={m} k={k} n_out={n_out} rank={rank} count={count} pad={pad} {dtype}")
    base, x, a, b, ids, scales = _case(m + k, m, k, n_out, rank, count, dtype, pad)
    kept = base.clone()
    out = wsl.lora_add(base, x, a, b, ids, scales)
    _check(base, x, a, b, ids, scales, out)
    assert base.equal(kept)
    _check(base, x, a, b, ids, None, wsl.lora_add(base, x, a, b, ids))
    same = wsl.lora_add(base, x, a, b, ids, scales, out=base)
    assert same is base and base.equal(out)


@pytest.mark.parametrize("m", [4, 64, 65, 200, 1100])
@pytest.mark.parametrize("rank,n_out", [(8, 80), (16, 128), (40, 129), (128, 64)])
def test_whole_numbers_are_exact(m, rank, n_out):
    """Small whole numbers: every sum is one that fp32 holds, so the result is equal.  A x runs up to
    2^22 and odd: it keeps all its bits on its way through the second product."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(m + rank)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda")
    k, count = 640, 3
    x, a = r(-64, 65, m, k), r(-64, 65, count, rank, k)
    b = torch.zeros((count, n_out, rank), dtype=torch.int64, device="cuda")
    for i in range(count):      # each output takes two entries of A x
        b[i].scatter_(1, r(0, rank, n_out, 2), r(-1, 2, n_out, 2))
    ids, base = r(-1, count, m).to(torch.int32), r(-1000, 1000, m, n_out)
    scales = torch.tensor([1.0, 2.0, -1.0], device="cuda")
    bf = torch.bfloat16
    out = wsl.lora_add(base.float(), x.to(bf), a.to(bf), b.to(bf), ids, scales)
    want, _ = ref.lora_ref(base.cpu().numpy(), x.cpu().numpy(), a.cpu().numpy(), b.cpu().numpy(), ids.tolist(), scales.tolist())
    assert (f32_of(out) == want).all()


@pytest.mark.parametrize("m", [9, 70, 200, 600])
def test_an_adapter_has_no_part_in_other_rows(m):
    """Adapters full of NaN and infinities, rows of x too: rows of other adapters and of none are as
    if they were not there."""
    import torch
    base, x, a, b, ids, scales = _case(m, m, 640, 150, 16, 5, "float32")
    ids[0], ids[1], ids[2] = -1, 0, 1
    want = wsl.lora_add(base, x, a, b, ids, scales)
    a[3], b[4], scales[2] = float("nan"), float("inf"), float("nan")
    b[3, ::2] = float("-inf")
    fine = (ids < 2).cpu()
    assert wsl.lora_add(base, x, a, b, ids, scales)[fine].equal(want[fine])
    x[ids == 0] = float("inf")
    fine = (ids == 1).cpu()
    assert wsl.lora_add(base, x, a, b, ids, scales)[fine].equal(want[fine])
    base[ids == -1] = -0.0
    base[0, 3] = float("nan")
    out = wsl.lora_add(base, x, a, b, ids, scales)
    none = (ids == -1).cpu()
    assert out[none].view(torch.int32).equal(base[none].view(torch.int32))


@pytest.mark.parametrize("m", [(1 << 19) + 17, 1 << 20])
def test_the_most_tokens(m):
    """Whole numbers, and a workspace with a guard behind it."""
    import torch
    say(f"lora m={m}")
    gen = torch.Generator(device="cuda").manual_seed(m)
    r = lambda *s: torch.randint(-8, 9, s, generator=gen, device="cuda")
    x, a, b, base = r(m, 16), r(2, 8, 16), r(2, 24, 8), r(m, 24)
    ids = torch.randint(-1, 2, (m,), generator=gen, device="cuda", dtype=torch.int32)
    bf, need = torch.bfloat16, wsl.lora_add_workspace_bytes(m, 8, 16)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device="cuda")
    out = wsl.lora_add(base.float(), x.to(bf), a.to(bf), b.to(bf), ids, workspace=ws[:need])
    want = base.float()
    for i in range(2):
        y = (x.float() @ a[i].float().t().contiguous()) @ b[i].float().t().contiguous()
        want = torch.where((ids == i)[:, None], want + y, want)
    assert out.equal(want) and (ws[need:] == 77).all()


@pytest.mark.parametrize("rank", [40, 64, 128])
@pytest.mark.parametrize("n_out", [150, 1024])
def test_high_ranks_of_many_tokens_apart(rank, n_out):
    """Six adapters among every 16 tokens, two of them and some rows full of NaN: the others are as before."""
    import torch
    base, x, a, b, ids, scales = _case(rank, 260, 1160, n_out, rank, 6, "float32")
    want = wsl.lora_add(base, x, a, b, ids, scales)
    _check(base, x, a, b, ids, scales, want)
    a[4], b[5] = float("nan"), float("nan")
    x[ids == 3] = float("nan")
    fine = (ids < 3).cpu()
    got = wsl.lora_add(base, x, a, b, ids, scales)
    assert got[fine].equal(want[fine]) and got[(ids > 2).cpu()].isnan().all()


@pytest.mark.parametrize("m", [5, 90, 1100])
def test_bad_ids_are_reported_and_left_out(m):
    import torch
    base, x, a, b, ids, scales = _case(7, m, 256, 96, 8, 3, "bfloat16")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wsl.lora_add(base, x, a, b, ids, scales, status=st)
    assert st.item() == 0
    for bad in (-2, 3, 2 ** 31 - 1, -2 ** 31):
        ids[m - 1] = bad
        st.zero_()
        out = wsl.lora_add(base, x, a, b, ids, scales, status=st)
        assert st.item() == wsl.WSL_STATUS_INDEX
        _check(base, x, a, b, ids, scales, out)


@pytest.mark.parametrize("m", [12, 150, 600])
def test_beside_a_packed_projection(m):
    """linear_gemm's output and its adapters in place, as a layer runs them, replayed from a graph with a
    poisoned workspace."""
    import torch
    k, n_out = 1024, 768
    base, x, a, b, ids, scales = _case(m, m, k, n_out, 16, 4, "float32")
    packed = wsl.nf4_pack((torch.randn((n_out, k), device="cuda") * k ** -0.5).to(torch.bfloat16))
    y = wsl.linear_gemm(packed, x, wfmt=wsl.WSL_W_NF4, n_out=n_out, k=k)
    want = wsl.lora_add(y, x, a, b, ids, scales)
    ws = torch.empty(wsl.lora_add_workspace_bytes(m, 16, k), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.copy_(y)
        wsl.lora_add(out, x, a, b, ids, scales, out=out, workspace=ws)
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
        assert out.equal(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = wsl.lora_add(y, x, a, b, ids, scales, stream=s)
    s.synchronize()
    assert other.equal(want)
    assert wsl.lora_add(y[:0], x[:0], a, b, ids[:0]).shape == (0, n_out)
