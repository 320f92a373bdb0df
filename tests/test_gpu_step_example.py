"""Pages, rotary positions, adapters and sampling together with the cache, attention and verification, as
examples/speculative_decode.py uses them; and a step of them against the same in 64 bits."""

import importlib.util
import math
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
def test_adapters_and_settings(fmt):
    """A drafter that is the target, with adapters: drafts stand as before, and each sequence's distribution is
    the one it has alone."""
    import torch
    ex = _example()
    kw = dict(layers=2, hidden=512, heads=8, n_kv=2, ffn=1024, vocab=1000, capacity=256, page=16, fmt=fmt, adapters=3,
              rank=24)
    target, drafter = (ex.Decoder(5, **kw) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randint(0, 1000, (5, 70), device="cuda", dtype=torch.int32, generator=gen)
    added, stood = ex.decode(target, drafter, prompt, 3, 5, lambda n, m: torch.full((n, m), 0.5, device="cuda"))
    assert (stood == 3).all() and (added >= 0).all()
    cut = dict(temperature=0.7, top_k=20, top_p=0.9)
    target, drafter = ex.Decoder(5, **kw, sampling=cut), ex.Decoder(5, **dict(kw, layers=1), sampling=cut)
    added, stood = ex.decode(target, drafter, prompt, 3, 5, lambda n, m: torch.rand((n, m), generator=gen, device="cuda"))
    there = torch.arange(4, device="cuda") <= stood[..., None]
    assert torch.equal(added >= 0, there)
    p = target.step(prompt[:, :9], torch.zeros(5, dtype=torch.int64, device="cuda"))
    assert ((p > 0).sum(-1) <= 20).all() and ((p.sum(-1) - 1).abs() < 1e-5).all()


def test_pages_of_a_run_come_back():
    """After any number of rounds exactly the pages behind the lengths are held, none twice."""
    import torch
    ex = _example()
    kw = dict(layers=1, hidden=256, heads=4, n_kv=2, ffn=512, vocab=300, capacity=128, page=4)
    target, drafter = ex.Decoder(3, **kw), ex.Decoder(3, seed=7, **kw)
    gen = torch.Generator(device="cuda").manual_seed(8)
    prompt = torch.randint(0, 300, (3, 21), device="cuda", dtype=torch.int32, generator=gen)
    ex.decode(target, drafter, prompt, 4, 9, lambda n, m: torch.rand((n, m), generator=gen, device="cuda"))
    for model in (target, drafter):
        lens, free = model.pages.lens.tolist(), model.pages.free[:model.pages.n_free.item()].tolist()
        held = [x for row, n in zip(model.table.tolist(), lens) for x in row[:-(-n // 4)]]
        assert sorted(held + free) == list(range(3 * 32))
    wsl.kv_pages_trim(target.pages, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert target.pages.n_free.item() == 3 * 32


def test_a_captured_step_goes_on_by_itself():
    """Pages, rotary positions, cache, attention, an adapter and the next token in one graph: replays give
    what eager steps give, token by token."""
    import torch
    n, heads, n_kv, dim, page, vocab, hidden = 3, 4, 2, 64, 8, 400, 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    packed = wsl.nf4_pack((r((heads + 2 * n_kv) * dim, hidden) * hidden ** -0.5).to(torch.bfloat16))
    head = wsl.nf4_pack((r(vocab, hidden) * 0.2).to(torch.bfloat16))
    embed = wsl.nf4_pack(r(vocab, hidden).to(torch.bfloat16))
    a, b = (r(2, 8, hidden) * hidden ** -0.5).to(torch.bfloat16), r(2, (heads + 2 * n_kv) * dim, 8).to(torch.bfloat16)
    ids, freqs = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda"), wsl.rotary_freqs(dim)
    uniforms = torch.rand((12, n), generator=gen, device="cuda")

    def fresh():
        return dict(pages=wsl.KVPages.empty(n, 6, 18, page), cache=wsl.KVCache.empty(18, n_kv, page, dim),
                    token=torch.tensor([3, 5, 7], dtype=torch.int32, device="cuda"), u=torch.zeros(n, device="cuda"))

    def step(s):
        slots, at = wsl.kv_pages_grow(s["pages"], 1)
        x = wsl.nf4_embed_rows(embed, vocab, hidden, s["token"].long())
        y = wsl.linear_gemm(packed, x, wfmt=wsl.WSL_W_NF4, n_out=(heads + 2 * n_kv) * dim, k=hidden)
        wsl.lora_add(y, x, a, b, ids, out=y)
        q, k, v = (z.unflatten(-1, (-1, dim)) for z in y.split((heads * dim, n_kv * dim, n_kv * dim), 1))
        wsl.rotary_embed(q, at, freqs, k=k, out=q, k_out=k)
        wsl.kv_cache_write(s["cache"], k, v, slots)
        out = wsl.attn_decode(s["cache"], q.to(torch.bfloat16)[:, None], s["pages"].table, s["pages"].lens)
        z = wsl.linear_gemm(head, out.view(n, -1), wfmt=wsl.WSL_W_NF4, n_out=vocab, k=hidden)
        wsl.sample_logits(z, s["u"], temperature=0.9, top_k=60, top_p=0.95, tokens=s["token"])

    eager, want = fresh(), []
    for i in range(12):
        eager["u"].copy_(uniforms[i])
        step(eager)
        want.append(eager["token"].tolist())
    s = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s)
    torch.cuda.current_stream().wait_stream(side)
    wsl.kv_pages_trim(s["pages"], torch.zeros(n, dtype=torch.int32, device="cuda"))
    s["token"].copy_(torch.tensor([3, 5, 7], dtype=torch.int32, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    got = []
    for i in range(12):
        s["u"].copy_(uniforms[i])
        graph.replay()
        got.append(s["token"].tolist())
    assert got == want and s["pages"].lens.tolist() == [12] * n
    assert math.isclose(float(s["pages"].n_free), 18 - 2 * n)
