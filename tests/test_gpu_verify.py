"""verify_drafts on the GPU against the fp64 reference: whole numbers, equal."""

import numpy as np
import pytest

import oracle.decode as od
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of, probabilities
from gpu_common import say

pytestmark = pytest.mark.gpu


def _case(seed, n, width, vocab, bf16, one_hot, pad=0):
    import torch
    g = np.random.default_rng([2026, 11, seed])
    dt = torch.bfloat16 if bf16 else torch.float32
    p = probabilities(g, n, width + 1, vocab)
    q = np.exp(np.log(np.maximum(p[:, :width], 1e-30)) + 0.5 * g.standard_normal((n, width, vocab)))
    q /= q.sum(-1, keepdims=True)
    drafts = (q / -np.log(np.maximum(g.random(q.shape), 1e-12))).argmax(-1).astype(np.int32) if width else \
        np.zeros((n, 0), np.int32)
    u = g.random((n, width + 1)).astype(np.float32)

    def rows(x):
        t = torch.zeros(*x.shape[:2], vocab + pad, dtype=dt, device="cuda")[..., :vocab]
        t.copy_(torch.from_numpy(x.astype(np.float32)))
        return t
    return rows(p), None if one_hot else rows(q), torch.from_numpy(drafts).cuda(), torch.from_numpy(u).cuda()


def _want(p, q, drafts, u, n_drafts=None):
    p64, q64 = f32_of(p), None if q is None else f32_of(q)
    d, uu = drafts.cpu().numpy(), u.cpu().numpy()
    nd = [d.shape[1]] * len(d) if n_drafts is None else n_drafts.cpu().numpy()
    got = [od.verify_ref(p64[b], None if q is None else q64[b], d[b], uu[b], nd[b], p.shape[2]) for b in range(len(d))]
    return np.array([r for r, _ in got], dtype=np.int32), np.array([t for _, t in got], dtype=np.int32)


def _check(p, q, drafts, u, n_drafts=None, **kw):
    acc, tok = wsl.verify_drafts(p, q, drafts, u, n_drafts, **kw)
    want = _want(p, q, drafts, u, n_drafts)
    assert np.array_equal(acc.cpu().numpy(), want[0]), (acc, want[0])
    assert np.array_equal(tok.cpu().numpy(), want[1])
    return want


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("one_hot", [False, True])
@pytest.mark.parametrize("n,width,vocab,pad", [
    (1, 4, 1000, 0), (7, 3, 1, 0), (5, 0, 4097, 0), (64, 2, 4096, 0), (3, 12, 8191, 3), (2, 64, 501, 1),
    (16, 1, 32000, 0), (4, 5, 151937, 7), (3, 2, 1024, 1), (3, 2, 1025, 1), (2, 3, 2049, 0), (2, 1, 32768, 0),
    (2, 1, 32769, 1), (33, 2, 65536, 3)])
def test_against_the_definition(n, width, vocab, pad, bf16, one_hot):
    say(f"verify n={n} width={width} vocab={vocab} pad={pad} bf16={bf16} one_hot={one_hot}")
    for seed in range(3):
        p, q, drafts, u = _case(100 * n + seed, n, width, vocab, bf16, one_hot, pad)
        _check(p, q, drafts, u)


def test_ragged_drafts_and_bad_ones():
    import torch
    p, q, drafts, u = _case(1, 9, 6, 3001, False, False)
    n = torch.tensor([0, 1, 2, 3, 4, 5, 6, -3, 99], dtype=torch.int32, device="cuda")
    u[:, :6] = 0.0                       # what has any chance stands
    acc, _ = _check(p, q, drafts, u, n)
    assert acc.tolist() == [0, 1, 2, 3, 4, 5, 6, 0, 6]
    for one_hot in (False, True):
        for bad in (-1, 3001, 2 ** 31 - 1, -2 ** 31):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            d = drafts.clone()
            d[4, 2] = bad
            acc, _ = _check(p, None if one_hot else q, d, u, status=st)
            assert acc[4] == 2 and st.item() == wsl.WSL_STATUS_INDEX


@pytest.mark.parametrize("step", [1024, 1000, 7, 8192])
def test_borders(step):
    """Dyadic probabilities, so that every sum is exact: ties and the borders of each token."""
    import torch
    vocab = 8 * step
    p = torch.zeros(1, 2, vocab, device="cuda")
    p[0, :, ::step] = 0.125              # 8 tokens of 1/8: 0, step, ..
    q = torch.zeros(1, 1, vocab, device="cuda")
    q[0, 0, 0], q[0, 0, 5] = 0.25, 0.75
    d0 = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for u0, stands in ((0.5, 0), (float(np.nextafter(np.float32(0.5), np.float32(0))), 1), (0.0, 1)):
        acc, _ = _check(p, q, d0, torch.tensor([[u0, 0.0]], device="cuda"))
        assert acc[0] == stands
    for i in range(8):                   # after acceptance: 8 equal parts; the border belongs to the next
        _, tok = _check(p, q, d0, torch.tensor([[0.0, i / 8]], device="cuda"))
        assert tok[0, 1] == step * i
    for u1 in (1.0, 2.0, -1.0, float("nan"), float(np.nextafter(np.float32(1), np.float32(0)))):
        _check(p, q, d0, torch.tensor([[0.0, u1]], device="cuda"))
        _check(p, q, d0, torch.tensor([[0.9, u1]], device="cuda"))
    # nothing left of p once q is off it: p itself
    _, tok = _check(p, p[:, :1].contiguous(), d0 + 1, torch.tensor([[0.5, 0.99]], device="cuda"))
    assert tok[0, 0] == 7 * step
    # a drafter that was certain of a token that p gives everything
    sure = torch.zeros(1, 2, vocab, device="cuda")
    sure[0, :, 37] = 1.0
    _check(sure, None, d0 + 37, torch.tensor([[1.0, 0.3]], device="cuda"))


def test_rows_that_give_nothing():
    import torch
    nan, inf = float("nan"), float("inf")
    p = torch.zeros(5, 1, 5000, device="cuda")
    p[1] = nan
    p[2, 0, 7], p[2, 0, 9] = inf, 1.0
    p[3] = -1.0
    p[4, 0, 4999], p[4, 0, 3] = 1e-40, nan
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d, u = torch.zeros(5, 0, dtype=torch.int32, device="cuda"), torch.full((5, 1), 0.5, device="cuda")
    _, tok = _check(p, None, d, u, status=st)
    assert tok[:, 0].tolist() == [-1, -1, -1, -1, 4999] and st.item() == wsl.WSL_STATUS_NONFINITE


def test_a_large_vocabulary():
    """More chunks than the second kernel has threads."""
    import torch
    vocab = 1500001
    g = np.random.default_rng(9)
    p = torch.from_numpy(g.random((2, 2, vocab)).astype(np.float32)).cuda()
    q = torch.from_numpy(g.random((2, 1, vocab)).astype(np.float32)).cuda()
    for u1 in (0.0, 0.3, 0.999999):
        u = torch.tensor([[0.0, u1], [1e9, u1]], device="cuda")
        _check(p, q, torch.tensor([[7], [9]], dtype=torch.int32, device="cuda"), u)


@pytest.mark.parametrize("vocab", [20011, 40009])
def test_streams_graphs_and_workspaces(vocab):
    import torch
    p, q, drafts, u = _case(3, 6, 4, vocab, False, False)
    want = _want(p, q, drafts, u)
    ws = torch.full((wsl.verify_drafts_workspace_bytes(6, vocab) // 8,), float("nan"), dtype=torch.float64, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    acc, tok = wsl.verify_drafts(p, q, drafts, u, workspace=ws, stream=s)
    s.synchronize()
    assert np.array_equal(tok.cpu().numpy(), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wsl.verify_drafts(p, q, drafts, u, accepted=acc, tokens=tok, workspace=ws)
    for i in range(4):
        u.copy_(torch.rand(6, 5, device="cuda"))
        tok.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        want = _want(p, q, drafts, u)
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(tok.cpu().numpy(), want[1])


def test_refusals():
    import torch
    p, q, drafts, u = _case(4, 3, 2, 100, False, False)
    ok = dict(p=p, q=q, drafts=drafts, u=u)
    for bad in (dict(p=p[0]), dict(p=p.half()), dict(q=q.bfloat16()), dict(q=q[:, :1]), dict(p=p[:, :2]), dict(drafts=drafts.long()),
                dict(u=u.double()), dict(u=u[:, :2]), dict(u=None), dict(drafts=drafts.cpu()),
                dict(n_drafts=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(p=p.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(p=p[:, :, ::2], q=q[:, :, ::2]), dict(tokens=torch.zeros(3, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            wsl.verify_drafts(**{**ok, **bad})
    with pytest.raises(wsl.WSLError) as e:
        wsl.verify_drafts(torch.zeros(1, 66, 8, device="cuda"), None, torch.zeros(1, 65, dtype=torch.int32, device="cuda"),
                          torch.zeros(1, 66, device="cuda"))
    assert e.value.code == 2
