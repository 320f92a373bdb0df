"""Inputs shared by the tests of the key-value cache, its attention and draft verification."""

import numpy as np

import oracle.decode as od


def f32_of(t):
    """float64 numpy values of a torch tensor of any float type."""
    return t.detach().float().cpu().numpy().astype(np.float64)


class CacheCase:
    """A cache of random pages holding seeded sequences, as torch tensors on `device`, and the values
    (float64) it stands for.  Slots that no sequence uses hold NaN."""

    def __init__(self, seed, lens, n_kv, dim, page, e4m3, device, spare=3, order="phtd", k_fill=None, v_fill=None,
                 total_pages=None):
        import torch
        import weight_streaming_linear_amd as wsl
        g = np.random.default_rng([2026, 7, seed])
        self.lens = list(lens)
        per = max(1, max((n + page - 1) // page for n in lens) if lens else 1)
        used = per * len(lens)
        n_pages = total_pages or used + spare
        names = g.permutation(n_pages)[:used] if n_pages < 1 << 20 else n_pages - 1 - g.permutation(used)
        self.table = torch.from_numpy(names.reshape(len(lens), per).astype(np.int32)).to(device)
        shape = {"phtd": (n_pages, n_kv, page, dim), "pthd": (n_pages, page, n_kv, dim)}[order]
        self.dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        pool = [torch.full(shape, 0x7f, dtype=torch.uint8, device=device) if e4m3 else
                torch.full(shape, float("nan"), dtype=torch.bfloat16, device=device) for _ in range(2)]
        if order == "pthd":
            pool = [t.transpose(1, 2) for t in pool]
        self.raw = pool
        self.exp = [torch.full((n_pages, n_kv, page), 255, dtype=torch.uint8, device=device) if e4m3 else None
                    for _ in range(2)]
        self.values = [[], []]              # [k or v][sequence]: float64 [tokens][n_kv][dim]
        for b, n in enumerate(lens):
            pages = torch.from_numpy(names.reshape(len(lens), per)[b].astype(np.int64)).to(device)
            for w, fill in ((0, k_fill), (1, v_fill)):
                x = g.standard_normal((per * page, n_kv, dim)) * np.exp(0.5 * g.standard_normal((1, n_kv, 1)))
                x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).float().numpy()
                if fill is not None:
                    fill(b, x)
                if e4m3:
                    codes, exps = od.kv_encode(x[:n])
                    vals = od.kv_decode(codes, exps)
                    data = np.full(x.shape, 0x7f, np.uint8)
                    data[:n] = codes
                    ex = np.full(x.shape[:2], 255, np.uint8)
                    ex[:n] = exps
                    ex = torch.from_numpy(ex).view(per, page, n_kv).transpose(1, 2)
                    self.exp[w][pages] = ex.to(device)
                    t = torch.from_numpy(data)
                else:
                    vals = x[:n].astype(np.float64)
                    x[n:] = np.nan
                    t = torch.from_numpy(x).to(torch.bfloat16)
                pool[w][pages] = t.view(per, page, n_kv, dim).transpose(1, 2).to(device)
                self.values[w].append(vals)
        views = [t.view(torch.float8_e4m3fn) if e4m3 else t for t in pool]
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        if device != "cpu":
            self.cache = wsl.KVCache(views[0], views[1], *self.exp)


def probabilities(g, n_seq, rows, vocab, sharp=2.0):
    z = sharp * g.standard_normal((n_seq, rows, vocab))
    z = np.exp(z - z.max(-1, keepdims=True))
    return (z / z.sum(-1, keepdims=True)).astype(np.float32)
