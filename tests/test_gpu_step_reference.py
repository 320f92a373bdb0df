"""A step of examples/speculative_decode.py against a plain forward pass in 64 bits: its pages, positions, cache,
attention, adapters and distributions together, of all sequences and of each alone.

The tolerance is the plain pass's own: where the step rounds to bf16 (half a step is 2^-8 of the value at most), the
plain pass is run again with each number off by a random part of that, and what the logarithms of the probabilities
move by at most in eight such passes, twice, is how far the step may be from it.  (Roundings to nearest are off by
less on average than these, and the fp32 sums by 2^-16 of them.)  So that this is worth something, the mistakes that a
step could make have to move them by more than twice as much."""

import importlib.util
import os

import numpy as np
import pytest

import oracle.step as ref
import weight_streaming_linear_amd as wsl

pytestmark = pytest.mark.gpu

KW = dict(layers=2, hidden=256, heads=4, n_kv=2, ffn=512, vocab=300, capacity=96, page=4, adapters=3, rank=24)


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Plain:
    """A Decoder's weights in 64 bits, on the CPU, and the whole of a sequence in one pass."""

    def __init__(self, model):
        import torch
        self.m = model
        full = lambda w: wsl.nf4_dequant_tile(w[0], w[1], w[2], 0, 0, w[1], w[2]).double().cpu()
        self.embed = wsl.nf4_embed_rows(model.embed, model.vocab, model.hidden, torch.arange(model.vocab, device="cuda"),
                                        ofmt=wsl.WSL_OUT_F32).double().cpu()
        self.layers = [{name: full(w) if len(w) == 3 else tuple(t.double().cpu() for t in w) for name, w in layer.items()}
                       for layer in model.layers]
        self.head = full(model.head)

    def log_probs(self, tokens, adapter, gen=None, turn_keys=True, at=None):
        """[len(tokens)][vocab] of one sequence; gen: of the random parts of half steps."""
        import torch
        m, n = self.m, len(tokens)

        def off(x):
            return x if gen is None else x * (1 + 2.0 ** -8 * (2 * torch.rand(x.shape, generator=gen, dtype=torch.float64) - 1))

        def linear(layer, name, x):
            y = x @ layer[name].T
            if adapter >= 0 and name + "_lora" in layer:
                a, b = layer[name + "_lora"]
                y = y + (x @ a[adapter].T) @ b[adapter].T
            return y

        def turned(x):
            angle = at[:, None] * 10000.0 ** (-torch.arange(m.dim // 2, dtype=torch.float64) * 2 / m.dim)
            c, s = angle.cos()[:, None], angle.sin()[:, None]
            a, b = x[..., :m.dim // 2], x[..., m.dim // 2:]
            return torch.cat((a * c - b * s, a * s + b * c), -1)

        norm = lambda x: off(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5))
        at = torch.arange(n, dtype=torch.float64) if at is None else at
        ahead = torch.ones(n, n).triu(1).bool()
        h = self.embed[tokens]
        for layer in self.layers:
            y = linear(layer, "qkv", norm(h))
            q, k, v = (t.unflatten(-1, (-1, m.dim)) for t in y.split((m.heads * m.dim, m.n_kv * m.dim, m.n_kv * m.dim), 1))
            q, k, v = off(turned(q)), off(turned(k) if turn_keys else k), off(v)
            out = torch.empty(n, m.heads, m.dim, dtype=torch.float64)
            for i in range(m.heads):
                g = i * m.n_kv // m.heads
                p = torch.softmax((q[:, i] @ k[:, g].T * m.dim ** -0.5).masked_fill(ahead, float("-inf")), -1)
                out[:, i] = off(off(p) @ v[:, g])
            h = h + linear(layer, "o", out.flatten(1))
            gate, up = (norm(h) @ layer["up"].T).chunk(2, -1)
            h = h + off(torch.nn.functional.silu(gate) * up) @ layer["down"].T
        return torch.log_softmax(norm(h) @ self.head.T, -1)

    def tolerance(self, tokens, adapter, seed):
        import torch
        want = self.log_probs(tokens, adapter)
        gen = torch.Generator().manual_seed(seed)
        moved = max((self.log_probs(tokens, adapter, gen) - want).abs().max().item() for _ in range(8))
        return want, 2 * moved


def _run(model, first, drafts, then):
    """The log probabilities of prompts, of drafts behind them, of other tokens in place of all but three of these,
    and of one token more."""
    import torch
    n, length = first.shape
    lens = torch.full((n,), length, dtype=torch.int64, device="cuda")
    p = [model.step(first, torch.zeros_like(lens)), model.step(drafts, lens), model.step(then[:, :-1].contiguous(), lens + 3),
         model.step(then[:, -1:].contiguous(), lens + 2 + then.shape[1])]
    assert model.pages.lens.tolist() == [length + 3 + then.shape[1]] * n
    return [x.double().log().cpu() for x in p]


def test_a_step_against_the_formulas():
    import torch
    ex = _example()
    n, length = 5, 70
    model = ex.Decoder(n, **KW)
    plain = Plain(model)
    gen = torch.Generator(device="cuda").manual_seed(11)
    first, drafts, then = (torch.randint(0, KW["vocab"], (n, w), generator=gen, device="cuda", dtype=torch.int32) for w in (length, 9, 6))
    got = _run(model, first, drafts, then)
    ids = model.ids.tolist()
    assert ids == [0, 1, 2, -1, 0]
    for b in range(n):
        a, d, t = (x[b].long().cpu() for x in (first, drafts, then))
        fallen, whole = torch.cat((a, d)), torch.cat((a, d[:3], t))
        want_fallen, tol = plain.tolerance(fallen, ids[b], 2 * b)
        want, tol_whole = plain.tolerance(whole, ids[b], 2 * b + 1)
        tol = max(tol, tol_whole)
        # what a mistake would make of it
        other = [plain.log_probs(whole, -1 if ids[b] >= 0 else 0), plain.log_probs(whole, ids[b], turn_keys=False),
                 plain.log_probs(whole, ids[b], at=torch.zeros(len(whole), dtype=torch.float64)),
                 plain.log_probs(whole, (ids[b] + 1) % 3), plain.log_probs(torch.cat((a, d[:2], d[3:4], t)), ids[b])]
        for wrong in other:
            assert (wrong - want)[-len(t):].abs().max() > 2 * tol
        alone = ex.Decoder(1, **KW)
        alone.ids.fill_(ids[b])
        for name, rows in (("with others", [x[b] for x in got]),
                           ("alone", [x[0] for x in _run(alone, first[b:b + 1], drafts[b:b + 1], then[b:b + 1])])):
            off = [(rows[0] - want_fallen[:length]).abs().max(), (rows[1] - want_fallen[length:]).abs().max(),
                   (torch.cat(rows[2:]) - want[length + 3:]).abs().max()]
            print(f"sequence {b}, {name}: {[f'{x:.4f}' for x in off]} of {tol:.4f}", flush=True)
            assert max(off) <= tol


def test_a_steps_distributions_are_cut_as_asked():
    """The same weights with settings: the plain probabilities cut by the definition.  log of a probability is the
    logit but for a constant, to 2^-23: weights of the 0.7th part of it to 2^-22."""
    import torch
    ex = _example()
    cut = dict(temperature=0.7, top_k=20, top_p=0.9)
    gen = torch.Generator(device="cuda").manual_seed(12)
    tokens = torch.randint(0, KW["vocab"], (3, 17), generator=gen, device="cuda", dtype=torch.int32)
    lens = torch.zeros(3, dtype=torch.int64, device="cuda")
    whole = ex.Decoder(3, **KW).step(tokens, lens).double().log().cpu().numpy()
    got = ex.Decoder(3, **KW, sampling=cut).step(tokens, lens).double().cpu().numpy()
    for b in range(3):
        for i in range(17):
            want = ref.sample_ref(whole[b, i], temperature=float(np.float32(0.7)), top_k=20, top_p=float(np.float32(0.9)))[1]
            assert ((got[b, i] > 0) == (want > 0)).all()
            assert (np.abs(got[b, i] - want) <= 2.0 ** -20 * want).all()
