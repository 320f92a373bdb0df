"""What a decode step does between its linear layers, its cache and its sampled tokens, as cases to be timed
and compared.

Four operators: the pages and slots of a paged key-value cache kept on the device, rotary positions, the
sampling of tokens from logits (and the distribution that is sampled), and low-rank adapters beside a shared
projection.  ``run`` computes them in plain torch operations, or (``own``) through the library's entry points.

Pages: a sequence of ``len`` tokens holds the ceil(len / page) first entries of its row of the block table; free
page numbers lie on a stack, free[0 .. n_free).  Growing by ``new`` tokens takes the missing pages off its top, in
the order of sequences and places; a sequence whose pages would reach below the stack's end is left as it is.
Trimming gives back what lies behind the new length, in the opposite order, so that growing again takes the
same pages.

Sampling: entries of a row are ordered by their logits, equal ones by their index.  K is the first top_k (all
where it is 0), w_j = exp((z_j - max z) / T), P the entries of K before which less than top_p * sum over K of w
lies, Q those with w_j >= min_p; K, P and Q together are kept, and the token is the least j for which the kept
w_0 + .. + w_j exceed u * (sum of the kept).  T = 0 keeps the first alone.
"""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one conversation's next token
        dict(name="pages_1x1", kind="pages", seqs=1, new=1, ragged=False, longest=4224, page=16),
        # a serving batch's drafts, all of which fall
        dict(name="pages_256x5_drafts", kind="pages", seqs=256, new=5, ragged=False, longest=8192, page=24),
        # prompts of many lengths taken in at once
        dict(name="pages_64_prompts", kind="pages", seqs=64, new=8192, ragged=True, longest=1000, page=16),
        # one token's queries and keys as the GEMV gives them, for a bf16 attention
        dict(name="rotary_1_token", kind="rotary", tokens=1, heads=40, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, scaling="none", far=4224, src="f32", out="bf16"),
        # a batch's drafts, a part of each head turned, pairs side by side
        dict(name="rotary_64x5_part", kind="rotary", tokens=320, heads=32, kv_heads=4, head_dim=96, rot_dim=48,
             interleaved=True, scaling="linear", far=32768, src="f32", out="f32"),
        # a long prompt far behind the trained length, after the prefill GEMM
        dict(name="rotary_8192_prompt", kind="rotary", tokens=8192, heads=48, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, scaling="bands", far=1000000, src="bf16", out="bf16"),
        # one conversation's token
        dict(name="sample_1x32000", kind="sample", seqs=1, vocab=32000, src="f32", spread=3.0, probs=False,
             top_k="some", top_p="some", min_p="none"),
        # a serving batch over a large vocabulary, every request with its own settings
        dict(name="sample_64x151937", kind="sample", seqs=64, vocab=151937, src="f32", spread=2.5, probs=False,
             top_k="mixed", top_p="mixed", min_p="mixed"),
        # the distributions of eight sequences' drafts and the token behind them, for their verification
        dict(name="probs_40x32000", kind="sample", seqs=40, vocab=32000, src="bf16", spread=3.0, probs=True,
             top_k="none", top_p="some", min_p="none"),
        # one token with its adapter
        dict(name="lora_1x5120", kind="lora", tokens=1, each=1, k=5120, n_out=5120, rank=16, adapters=8, src="f32"),
        # a serving batch of many adapters beside a fused projection
        dict(name="lora_48x7168", kind="lora", tokens=48, each=1, k=5120, n_out=7168, rank=32, adapters=40, src="f32"),
        # prompts of several requests
        dict(name="lora_4224x6144", kind="lora", tokens=4224, each=600, k=6144, n_out=6144, rank=16, adapters=12,
             src="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["pages", "rotary", "sample", "sample", "lora", "lora"])
    src = rng.choice(["f32", "bf16"])
    if kind == "pages":
        seqs, ragged = _spread(rng, 1, 2000), rng.random() < 0.5
        page = rng.choice([16, 32, 64, 128, 48, 24, 20, 1, 7])
        new = _spread(rng, 1, max(1, min(8192, 64 * 8192 // seqs))) if ragged else rng.choice([1, 1, 2, 3, 5, 8])
        longest = _spread(rng, 1, max(1, min(16384, (1 << 19) * min(page, 16) // (16 * seqs))))
        return dict(kind=kind, seqs=seqs, new=new, ragged=ragged, longest=longest, page=page)
    if kind == "rotary":
        kv_heads, head_dim = rng.choice([1, 2, 4, 8, 8]), rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 6, 8])
        most = 8192 * 56 * 128 // ((heads + kv_heads) * head_dim)
        return dict(kind=kind, tokens=_spread(rng, 1, min(8192, most // 2)), heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, rot_dim=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4]),
                    interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "bands", "base"]),
                    far=_spread(rng, 100, 1000000), src=src, out=rng.choice(["f32", "bf16"]))
    if kind == "sample":
        some = ["none", "some", "mixed"]
        return dict(kind=kind, seqs=_spread(rng, 1, 64), vocab=_spread(rng, 500, 151937), src=src,
                    spread=rng.choice([1.5, 2.5, 3.0, 4.0]), probs=rng.random() < 0.3, top_k=rng.choice(some),
                    top_p=rng.choice(some), min_p=rng.choice(some))
    k, n_out = 64 * rng.randint(8, 96), rng.choice([64 * rng.randint(8, 112), rng.randint(500, 7000)])
    tokens = _spread(rng, 1, 4000)
    rank = rng.choice([8, 16, 16, 32, 64]) if tokens < 500 else rng.choice([8, 16])
    return dict(kind=kind, tokens=tokens, each=min(tokens, rng.choice([1, 1, 5]) if tokens < 300 else _spread(rng, 50, 1000)),
                k=k, n_out=n_out, rank=rank, adapters=rng.choice([1, 4, 12, 40]) if tokens < 500 else rng.choice([1, 4, 12]),
                src=src)


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _freqs64(case):
    """The turning of each pair from position to position, in radians, scaled for far positions; plain Python."""
    d, base, factor, trained = case["rot_dim"], 10000.0, 8.0, 8192
    if case["scaling"] == "base":
        base *= factor ** (d / (d - 2))
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] == "bands":      # slow pairs are stretched, fast ones kept: by their turns over the trained length
        g = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for x in f]
        f = [x * (y + (1 - y) / factor) for x, y in zip(f, g)]
    return f


def _settings(gen, how, n, values, off):
    """None, one value for all, or a tensor of a value for each row (some of them off)."""
    if how == "none":
        return None
    if how == "some":
        return values[0]
    pick = torch.randint(0, len(values) + 1, (n,), generator=gen, device=DEV)
    return torch.tensor([*values, off], device=DEV)[pick]


def _prompts(n, longest):
    """Lengths of n prompts, spread over a factor of sixteen, and of every tenth sequence none."""
    i = torch.arange(n, device=DEV)
    return torch.where(i % 10 == 9, 0, (longest * torch.exp2(-4 * i.double() / n)).long())


def _total(case):
    n, new = case["seqs"], case["new"]
    return n * new if not case["ragged"] else sum(int(new * 2.0 ** (-4 * i / n)) for i in range(n) if i % 10 != 9)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=dict(case))
    kind = case["kind"]
    if kind == "pages":
        n, page, new = case["seqs"], case["page"], case["new"]
        lens = torch.randint(0, case["longest"] + 1, (n,), generator=gen, device=DEV)
        if case["ragged"]:
            s["new"] = _prompts(n, new)[torch.randperm(n, generator=gen, device=DEV)]
        else:
            s["new"] = torch.full((n,), new, device=DEV)
        s["total"] = _total(case)
        per = (case["longest"] + new + page - 1) // page
        held = (lens + page - 1) // page
        numbers = torch.randperm(n * per, generator=gen, device=DEV).to(torch.int32)
        entries = torch.arange(per, device=DEV) < held[:, None]
        taken = int(held.sum())
        s["table"] = torch.full((n, per), -1, dtype=torch.int32, device=DEV)
        s["table"][entries] = numbers[:taken]
        s["free"] = numbers.new_full((n * per,), -1)
        s["free"][:n * per - taken] = numbers[taken:]
        s["n_free"] = torch.tensor([n * per - taken], dtype=torch.int32, device=DEV)
        s["lens"], s["new"] = lens.to(torch.int32), s["new"].to(torch.int32)
        s["before"] = s["lens"].clone()
        return s
    if kind == "rotary":
        n, h, kh, d = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        x = torch.randn((n, (h + 2 * kh) * d), generator=gen, device=DEV).mul_(1.5).to(_dtype(case["src"]))
        s["q"] = x[:, :h * d].unflatten(-1, (h, d))
        s["k"] = x[:, h * d:(h + kh) * d].unflatten(-1, (kh, d))
        at = torch.randint(0, case["far"], (1,), generator=gen, device=DEV) + torch.arange(n, device=DEV)
        s["positions"] = at if n > 500 else torch.randint(0, case["far"], (n,), generator=gen, device=DEV)
        s["freqs"] = torch.tensor(_freqs64(case), dtype=torch.float64, device=DEV)
        s["amplitude"] = 1.0 if case["scaling"] != "bands" else 0.1 * math.log(8.0) + 1.0
        return s
    if kind == "sample":
        n, v = case["seqs"], case["vocab"]
        z = torch.randn((n, v), generator=gen, device=DEV)
        z *= case["spread"] * (0.7 + 0.6 * torch.rand((n, 1), generator=gen, device=DEV))
        few = torch.randint(0, v, (n, 6), generator=gen, device=DEV)     # what the context suggests
        z.scatter_add_(1, few, 3 * case["spread"] * torch.rand((n, 6), generator=gen, device=DEV))
        s["z"] = z.to(_dtype(case["src"]))
        s["u"] = torch.rand(n, generator=gen, device=DEV)
        s["temperature"] = 0.8 if case["top_p"] != "mixed" else \
            torch.tensor([0.0, 0.6, 0.8, 1.0, 1.3], device=DEV)[torch.randint(0, 5, (n,), generator=gen, device=DEV)]
        s["top_k"] = _settings(gen, case["top_k"], n, [50, 20, 400, 1, 5000], 0)
        s["top_p"] = _settings(gen, case["top_p"], n, [0.9, 0.5, 0.95, 0.99], 1.0)
        s["min_p"] = _settings(gen, case["min_p"], n, [0.05, 0.01, 0.2], 0.0)
        if torch.is_tensor(s["top_k"]):
            s["top_k"] = s["top_k"].to(torch.int32)
        return s
    m, k, n_out, r, count = (case[x] for x in ("tokens", "k", "n_out", "rank", "adapters"))
    s["x"] = torch.randn((m, k), generator=gen, device=DEV).to(torch.bfloat16)
    s["base"] = torch.randn((m, n_out), generator=gen, device=DEV).to(_dtype(case["src"]))
    s["a"] = (torch.randn((count, r, k), generator=gen, device=DEV) * k ** -0.5).to(torch.bfloat16)
    s["b"] = (torch.randn((count, n_out, r), generator=gen, device=DEV) * 0.3 * r ** -0.5).to(torch.bfloat16)
    s["scales"] = 0.5 + torch.rand(count, generator=gen, device=DEV)
    requests = (m + case["each"] - 1) // case["each"]
    ids = torch.randint(0, count, (requests,), generator=gen, device=DEV)
    ids[torch.rand(requests, generator=gen, device=DEV) < 0.1] = -1      # requests of the shared model alone
    if requests == 1:
        ids.clamp_(min=0)
    s["ids"] = ids.repeat_interleave(case["each"])[:m].to(torch.int32)
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_grow(s):
    lens, new, page, total = s["lens"].long(), s["new"].long(), s["case"]["page"], s["total"]
    table, free, left = s["table"], s["free"], s["n_free"].long()
    held = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - held
    off = need.cumsum(0) - need
    served = (need == 0) | (off + need <= left)
    start = new.cumsum(0) - new
    i = torch.arange(total, device=DEV)
    b = torch.repeat_interleave(torch.arange(len(lens), device=DEV), new, output_size=total)
    at = lens[b] + i - start[b]
    place = at // page
    fresh = place >= held[b]
    taken = free[(left - 1 - off[b] - place + held[b]).clamp(min=0)]
    number = torch.where(fresh & served[b], taken, table[b, place])
    table[b, place] = number
    slots = torch.where(served[b], number.long() * page + at % page, -1)
    positions = torch.where(served[b], at, -1)
    s["lens"] += torch.where(served, new, 0).to(torch.int32)
    s["n_free"] -= torch.where(served, need, 0).sum().to(torch.int32)
    return slots, positions


def _plain_trim(s, to):
    lens, page, table, free = s["lens"].long(), s["case"]["page"], s["table"], s["free"]
    keep = torch.minimum(lens, to.long())
    held, kept = (lens + page - 1) // page, (keep + page - 1) // page
    back = held - kept
    off, total = back.cumsum(0) - back, back.sum()
    place = torch.arange(table.shape[1], device=DEV)
    gone = (place >= kept[:, None]) & (place < held[:, None])
    dest = s["n_free"].long() + total - 1 - off[:, None] - place + kept[:, None]
    wide = torch.cat((free, free.new_empty(1)))
    wide[torch.where(gone, dest, len(free))] = table
    free.copy_(wide[:-1])
    s["n_free"] += total.to(torch.int32)
    s["lens"].copy_(keep)


def _plain_rotary(s):
    c = s["case"]
    d, half = c["rot_dim"], c["rot_dim"] // 2
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    out = []
    for x in (s["q"], s["k"]):
        x = x.float()
        turned = x[..., :d]
        if c["interleaved"]:
            a, b = turned[..., 0::2], turned[..., 1::2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = turned[..., :half], turned[..., half:]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        out.append(torch.cat((y, x[..., d:]), -1).to(_dtype(c["out"])))
    return tuple(out)


def _column(x, n, dtype, off):
    """A setting as a column of n rows."""
    if torch.is_tensor(x):
        return x.to(dtype)[:, None]
    return torch.full((n, 1), off if x is None else x, dtype=dtype, device=DEV)


def _plain_sample(s):
    z = s["z"].double()
    n, v = z.shape
    # settings are 32-bit numbers: 0.9 is what fp32 makes of it
    t, top_p, min_p = (_column(s[x], n, torch.float32, off).double()
                       for x, off in (("temperature", 1.0), ("top_p", 1.0), ("min_p", 0.0)))
    top_k = _column(s["top_k"], n, torch.int64, 0)
    greedy = t <= 0
    top_k = torch.where(greedy, 1, torch.where(top_k <= 0, v, top_k))
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = torch.exp((zs - zs[:, :1]) / torch.where(greedy, 1.0, t))
    w = w * (torch.arange(v, device=DEV) < top_k)
    before = w.cumsum(1) - w
    before[:, 0] = 0
    keep = (w > 0) & (w >= min_p)
    keep &= (top_p >= 1) | (before < top_p * w.sum(1, keepdim=True))
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, w * keep)
    up = w.cumsum(1)
    token = (up > s["u"].double()[:, None] * up[:, -1:]).to(torch.uint8).argmax(1).to(torch.int32)
    return (token, (w / w.sum(1, keepdim=True)).float()) if s["case"]["probs"] else token


def _plain_lora(s):
    a, b, ids = s["a"].float(), s["b"].float(), s["ids"].long()
    count, r, k = a.shape
    h = torch.matmul(s["x"].float(), a.view(count * r, k).T).view(-1, count, r)
    mine = (ids[:, None] == torch.arange(count, device=DEV)).float() * s["scales"]
    h = (h * mine[..., None]).view(-1, count * r)
    y = torch.matmul(h, b.transpose(1, 2).reshape(count * r, -1))
    return (s["base"].float() + y).to(s["base"].dtype)


def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        import weight_streaming_linear_amd as wsl
        if kind == "pages":     # taken for the step, and given back: the drafts fell, the prompts are done with
            if "pages" not in s:
                s["pages"] = wsl.KVPages(s["table"], s["lens"], s["free"], s["n_free"], c["page"])
            new = dict(new=s["new"], n_tokens=s["total"]) if c["ragged"] else dict(new=c["new"])
            slots, positions = wsl.kv_pages_grow(s["pages"], **new)
            wsl.kv_pages_trim(s["pages"], s["before"])
            return slots, positions, s["table"], s["lens"], s["free"], s["n_free"]
        if kind == "rotary":
            ofmt = wsl.WSL_OUT_F32 if c["out"] == "f32" else wsl.WSL_OUT_BF16
            return wsl.rotary_embed(s["q"], s["positions"], s["freqs"], k=s["k"], interleaved=c["interleaved"],
                                    amplitude=s["amplitude"], ofmt=ofmt)
        if kind == "sample":
            how = {x: s[x] for x in ("temperature", "top_k", "top_p", "min_p") if s[x] is not None}
            if c["probs"]:
                probs = torch.empty((c["seqs"], c["vocab"]), dtype=torch.float32, device=DEV)
                return wsl.sample_logits(s["z"], s["u"], probs=probs, **how), probs
            return wsl.sample_logits(s["z"], s["u"], **how)
        return wsl.lora_add(s["base"], s["x"], s["a"], s["b"], s["ids"], s["scales"])
    if kind == "pages":
        slots, positions = _plain_grow(s)
        _plain_trim(s, s["before"])
        return slots, positions, s["table"], s["lens"], s["free"], s["n_free"]
    if kind == "rotary":
        return _plain_rotary(s)
    return _plain_sample(s) if kind == "sample" else _plain_lora(s)


def work(case):
    """One pass: every input read once and every output written once."""
    kind = case["kind"]
    if kind == "pages":
        tokens = _total(case)
        return dict(bytes=16 * tokens + 16 * tokens / case["page"] + 24 * case["seqs"], flops=4 * tokens)
    size = 4 if case["src"] == "f32" else 2
    if kind == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return dict(bytes=n * case["head_dim"] * (size + (4 if case["out"] == "f32" else 2)),
                    flops=3 * n * case["rot_dim"])
    if kind == "sample":
        n = case["seqs"] * case["vocab"]
        return dict(bytes=n * (size + (4 if case["probs"] else 0)), flops=4 * n)
    m, r, k, n = case["tokens"], case["rank"], case["k"], case["n_out"]
    requests = -(-m // case["each"])
    used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** requests)
    return dict(bytes=2 * m * k + 2 * m * n * size + 2 * used * r * (k + n), flops=2 * m * r * (k + n))


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_pages(s):
    """The stack and the table as lists, one sequence after the other."""
    page = s["case"]["page"]
    table, free, lens = s["table"].tolist(), s["free"].tolist(), s["lens"].tolist()
    n, asked, slots, positions = int(s["n_free"]), 0, [], []
    top = n
    for b, new in enumerate(s["new"].tolist()):
        held, now = -(-lens[b] // page), -(-(lens[b] + new) // page)
        asked += now - held
        ok = now == held or asked <= n
        for place in range(held, now if ok else held):
            top -= 1
            table[b][place] = free[top]
        for t in range(lens[b], lens[b] + new):
            slots.append(table[b][t // page] * page + t % page if ok else -1)
            positions.append(t if ok else -1)
    whole = lambda x, like: torch.tensor(x, dtype=like.dtype)
    return (torch.tensor(slots, dtype=torch.int64), torch.tensor(positions, dtype=torch.int64), whole(table, s["table"]),
            whole(lens, s["lens"]), whole(free, s["free"]), whole([n], s["n_free"]))


def _exact_rotary(s):
    c = s["case"]
    d = c["rot_dim"]
    i = torch.arange(d // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + d // 2)
    turn = torch.polar(torch.full_like(s["freqs"], s["amplitude"]).expand(c["tokens"], -1).contiguous(),
                       torch.outer(s["positions"].double(), s["freqs"]))[:, None]
    out = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_sample(s):
    import numpy as np
    z, u = s["z"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    n, v = z.shape
    of = lambda x, i, off: off if x is None else float(np.float32(x[i].item() if torch.is_tensor(x) else x))
    tokens, probs = np.zeros(n, np.int32), np.zeros((n, v))
    for i in range(n):
        t = of(s["temperature"], i, 1.0)
        order = np.lexsort((np.arange(v), -z[i]))
        k = int(of(s["top_k"], i, 0)) or v
        order = order[:1 if t <= 0 else min(k, v)]
        w = np.exp((z[i][order] - z[i][order[0]]) / (t if t > 0 else 1.0))
        top_p, min_p = of(s["top_p"], i, 1.0), of(s["min_p"], i, 0.0)
        last = len(w)
        if top_p < 1:
            last = min(last, max(1, int(np.searchsorted(np.cumsum(w), top_p * w.sum(), side="left")) + 1))
        last = min(last, max(1, int((w >= min_p).sum())))
        kept = np.sort(order[:last])
        w = np.exp((z[i][kept] - z[i].max()) / (t if t > 0 else 1.0))
        up = np.cumsum(w)
        tokens[i] = kept[min(int(np.searchsorted(up, u[i] * up[-1], side="right")), len(kept) - 1)]
        probs[i][kept] = w / up[-1]
    tokens = torch.from_numpy(tokens)
    return (tokens, torch.from_numpy(probs)) if s["case"]["probs"] else tokens


def _exact_lora(s):
    y = s["base"].double().clone()
    for a in range(s["case"]["adapters"]):
        rows = (s["ids"] == a).nonzero()[:, 0]
        if len(rows):
            h = s["x"][rows].double() @ s["a"][a].double().T.contiguous()
            y[rows] += s["scales"][a].double() * (h @ s["b"][a].double().T.contiguous())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "rotary": _exact_rotary, "sample": _exact_sample, "lora": _exact_lora}[case["kind"]](s)
