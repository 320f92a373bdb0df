#!/usr/bin/env python3
"""Drafting and verifying with the library's decode-side calls, on random weights.

A small decoder (NF4 linear layers, grouped-query attention, rotary positions) continues a few
sequences.  A shallower one drafts ``width`` tokens for each, one at a time; the target scores all
of them and the token before them in one sweep over its weights and its cache, and
``verify_drafts`` keeps what agrees with the target and samples the next token.  Lengths, drafts
and tokens stay on the device: nothing is read back until the end.

    python examples/speculative_decode.py [--e4m3] [--seqs 4] [--width 4] [--tokens 64]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_streaming_linear_amd as wsl  # noqa: E402

NF4, F32 = wsl.WSL_W_NF4, wsl.WSL_OUT_F32


class Decoder:
    """`layers` layers of random NF4 weights, each with a paged key-value cache for n_seq sequences."""

    def __init__(self, n_seq, layers, hidden=1024, heads=16, n_kv=4, ffn=2816, vocab=8000, capacity=1024, page=16,
                 fmt=wsl.WSL_KV_BF16, seed=0):
        self.hidden, self.heads, self.n_kv, self.ffn, self.vocab, self.page = hidden, heads, n_kv, ffn, vocab, page
        self.dim = hidden // heads
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def packed(n, k):
            w = torch.randn((n, k), generator=gen, device="cuda").mul_(k ** -0.5).to(torch.bfloat16)
            return wsl.nf4_pack(w), n, k

        self.embed = wsl.nf4_pack(torch.randn((vocab, hidden), generator=gen, device="cuda").to(torch.bfloat16))
        self.layers = [dict(qkv=packed((heads + 2 * n_kv) * self.dim, hidden), o=packed(hidden, hidden),
                            up=packed(2 * ffn, hidden), down=packed(hidden, ffn)) for _ in range(layers)]
        self.head = packed(vocab, hidden)
        pages = -(-capacity // page)
        self.table = torch.randperm(n_seq * pages, generator=gen, device="cuda").view(n_seq, pages).to(torch.int32)
        self.caches = [wsl.KVCache.empty(n_seq * pages, n_kv, page, self.dim, fmt) for _ in range(layers)]

    def linear(self, w, x):
        packed, n, k = w
        return wsl.linear_gemm(packed, x, wfmt=NF4, n_out=n, k=k, ofmt=F32)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)).to(torch.bfloat16)

    def rotate(self, x, at):
        """Rotary positions of x [n_seq, q_len, heads, dim] at the positions `at` [n_seq, q_len]."""
        half = self.dim // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        angle = at.double()[..., None, None] * freq
        c, s = angle.cos().float(), angle.sin().float()
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def step(self, tokens, lens):
        """Takes in tokens [n_seq, q_len] behind the `lens` [n_seq] that the cache holds of each sequence
        (on the device: that lens + q_len is within the capacity is for the caller to see to); returns the
        probabilities [n_seq, q_len, vocab] of what follows each."""
        n_seq, q_len = tokens.shape
        at = lens[:, None] + torch.arange(q_len, device="cuda")
        slots = (self.table.gather(1, at // self.page).long() * self.page + at % self.page).view(-1)
        kv_lens = (lens + q_len).to(torch.int32)
        q_heads, kv = self.heads * self.dim, self.n_kv * self.dim
        h = wsl.nf4_embed_rows(self.embed, self.vocab, self.hidden, tokens.reshape(-1).long(), ofmt=F32)
        for layer, cache in zip(self.layers, self.caches):
            x = self.linear(layer["qkv"], self.norm(h)).view(n_seq, q_len, -1)
            q = self.rotate(x[..., :q_heads].unflatten(-1, (self.heads, self.dim)), at)
            k = self.rotate(x[..., q_heads:q_heads + kv].unflatten(-1, (self.n_kv, self.dim)), at)
            v = x.view(n_seq * q_len, -1)[:, q_heads + kv:].unflatten(-1, (self.n_kv, self.dim))
            wsl.kv_cache_write(cache, k.flatten(0, 1), v, slots)
            out = wsl.attn_decode(cache, q.to(torch.bfloat16), self.table, kv_lens)
            h = h + self.linear(layer["o"], out.view(-1, self.hidden))
            gate, up = self.linear(layer["up"], self.norm(h)).chunk(2, -1)
            h = h + self.linear(layer["down"], (torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        return torch.softmax(self.linear(self.head, self.norm(h)), -1).view(n_seq, q_len, -1)


def pick(p, u):
    """A token of each row of p [n_seq, vocab] for numbers u [n_seq] in [0, 1)."""
    return wsl.verify_drafts(p[:, None], None, torch.empty(len(p), 0, dtype=torch.int32, device="cuda"), u[:, None])[1]


def most_tokens(length, width, rounds):
    """The tokens that the caches of a sequence hold at most: its prompt, and all drafts standing in every round."""
    return length + rounds * (width + 1)


def decode(target, drafter, prompt, width, rounds, uniform):
    """Continues prompt [n_seq, length] by `rounds` rounds of `width` drafts; uniform(n, m) gives random
    numbers in [0, 1) on the device.  Returns the tokens that every round added, -1 where there is none,
    and how many drafts stood, [rounds, n_seq, width + 1] and [rounds, n_seq]."""
    n_seq, length = prompt.shape
    if width < 0 or rounds < 1:
        raise ValueError(f"{rounds} rounds of {width} drafts")
    for model in (target, drafter):     # lengths are on the device from here on: nothing checks them there
        room = model.table.shape[1] * model.page
        if most_tokens(length, width, rounds) > room:
            raise ValueError(f"{length} tokens and {rounds} rounds of {width} drafts do not fit into {room}")
    lens = torch.zeros(n_seq, dtype=torch.int64, device=prompt.device)
    for i in range(0, length, 64):
        chunk = prompt[:, i:i + 64]
        p = target.step(chunk, lens)
        drafter.step(chunk, lens)
        lens = lens + chunk.shape[1]
    last = pick(p[:, -1].contiguous(), uniform(n_seq, 1)[:, 0])         # sampled, not in the caches yet
    added, stood = [], []
    for _ in range(rounds):
        drafts, q = [], []
        x = last
        for i in range(width + 1):          # the last draft is taken in too: its keys may be needed
            p = drafter.step(x, lens + i)[:, 0]
            if i < width:
                x = pick(p, uniform(n_seq, 1)[:, 0])
                drafts.append(x)
                q.append(p)
        drafts = torch.cat(drafts, 1) if width else last[:, :0].contiguous()
        p = target.step(torch.cat((last, drafts), 1), lens)
        accepted, tokens = wsl.verify_drafts(p, torch.stack(q, 1) if width else None, drafts, uniform(n_seq, width + 1))
        last = tokens.gather(1, accepted[:, None].long())
        lens = lens + 1 + accepted          # what a fallen draft left in the caches is written over
        added.append(tokens)
        stood.append(accepted)
    return torch.stack(added), torch.stack(stood)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--width", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = ap.parse_args()
    fmt = wsl.WSL_KV_E4M3 if a.e4m3 else wsl.WSL_KV_BF16
    length, rounds = 100, -(-a.tokens // (a.width + 1))
    kw = dict(fmt=fmt, capacity=max(1024, most_tokens(length, a.width, rounds)))
    target = Decoder(a.seqs, a.layers, **kw)
    drafter = Decoder(a.seqs, max(1, a.layers // 2), **kw)      # its weights only in the first layers: some drafts stand
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randint(0, target.vocab, (a.seqs, length), generator=gen, device="cuda", dtype=torch.int32)
    for name, model in (("another model", drafter), ("the target itself", Decoder(a.seqs, a.layers, **kw))):
        added, stood = decode(target, model, prompt, a.width, rounds,
                              lambda n, m: torch.rand((n, m), generator=gen, device="cuda"))
        print(f"drafts of {name}: {stood.float().mean():.2f} of {a.width} stand; sequence 0 goes on "
              f"{[t for t in added[:, 0].flatten().tolist() if t >= 0][:12]} ..")


if __name__ == "__main__":
    main()
