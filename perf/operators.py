"""The decode-side operators beside the linear layers, as cases to be timed and compared.

Four operators: a paged key-value cache's write (quantising), its read back, the attention
of new tokens over that cache, and the verification of drafted tokens.  ``run`` computes
them in plain torch operations, or (``own``) through the library's entry points.

Cache values are bf16, or e4m3 codes with one power-of-two scale per token and kv head:
with a = max|x| over the head, e is the smallest integer >= -110 with a <= 448 * 2^e, the
code is x * 2^-e rounded to e4m3 (ties to even), its value code * 2^e; the byte e + 127 is
stored.  Caches are [page][kv head][token of the page][head dim].
"""

import math

import torch

own = False

DEV = "cuda"
E_MIN = -110


def listed():
    return [
        # one token's keys and values as the GEMV gives them (fp32), kept as bf16
        dict(name="store_1_token_bf16", kind="store", seqs=1, tokens=1, kv_heads=8, head_dim=128, page=16,
             fmt="bf16", src="f32"),
        # a serving batch's new tokens, quantised
        dict(name="store_64_seqs_e4m3", kind="store", seqs=64, tokens=64, kv_heads=8, head_dim=128, page=48,
             fmt="e4m3", src="f32"),
        # the positions of a long prompt, quantised after the prefill GEMM
        dict(name="store_8192_prompt_e4m3", kind="store", seqs=1, tokens=8192, kv_heads=8, head_dim=128, page=64,
             fmt="e4m3", src="bf16"),
        # a conversation's prefix taken out of the cache, to be kept or moved
        dict(name="fetch_4224_e4m3", kind="fetch", seqs=1, tokens=4224, kv_heads=8, head_dim=128, page=16,
             fmt="e4m3", src="bf16"),
        # prefixes of a whole batch
        dict(name="fetch_32x2000_bf16", kind="fetch", seqs=32, tokens=64000, kv_heads=8, head_dim=128, page=24,
             fmt="bf16", src="f32"),
        # the first steps of one conversation, all in fp32 around the cache
        dict(name="attend_1x37_bf16", kind="attend", seqs=1, q_len=1, heads=40, kv_heads=8, head_dim=128, page=16,
             longest=37, ragged=False, window=0, fmt="bf16", src="f32"),
        # one long conversation: few heads, so the length has to be split
        dict(name="attend_1x8192_bf16", kind="attend", seqs=1, q_len=1, heads=48, kv_heads=8, head_dim=128, page=16,
             longest=8192, ragged=False, window=0, fmt="bf16", src="bf16"),
        # a serving batch of ragged lengths over a quantised cache
        dict(name="attend_32x8192_e4m3", kind="attend", seqs=32, q_len=1, heads=48, kv_heads=8, head_dim=128,
             page=64, longest=8192, ragged=True, window=0, fmt="e4m3", src="bf16"),
        # drafts verified in one sweep: four drafts and the token before them, odd pages
        dict(name="attend_16x4224_drafts_bf16", kind="attend", seqs=16, q_len=5, heads=40, kv_heads=8, head_dim=128,
             page=24, longest=4224, ragged=True, window=0, fmt="bf16", src="bf16"),
        # long documents
        dict(name="attend_8x32768_bf16", kind="attend", seqs=8, q_len=1, heads=40, kv_heads=8, head_dim=128,
             page=64, longest=32768, ragged=False, window=0, fmt="bf16", src="bf16"),
        # one conversation's drafts
        dict(name="verify_1x4", kind="verify", seqs=1, drafts=4, vocab=32000, one_hot=False, src="f32"),
        # a serving batch's drafts over a large vocabulary
        dict(name="verify_64x8", kind="verify", seqs=64, drafts=8, vocab=151937, one_hot=False, src="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["store", "fetch", "attend", "attend", "attend", "verify"])
    fmt = rng.choice(["bf16", "e4m3"])
    src = rng.choice(["f32", "bf16"])
    if kind == "verify":
        drafts = rng.randint(0, 12)
        vocab = _spread(rng, 500, 160000)
        return dict(kind=kind, seqs=_spread(rng, 1, 64), drafts=min(drafts, 8 if vocab > 80000 else 12), vocab=vocab,
                    one_hot=rng.random() < 0.3, src=src)
    head_dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128, 48, 24, 20, 1, 7])
    if kind in ("store", "fetch"):
        seqs, kv_heads = _spread(rng, 1, 64), rng.choice([1, 2, 3, 4, 8])
        most = (8192 if kind == "store" else 64000) * 8 * 128 // (kv_heads * head_dim * seqs)
        return dict(kind=kind, seqs=seqs, tokens=seqs * _spread(rng, 1, most), kv_heads=kv_heads, head_dim=head_dim,
                    page=page, fmt=fmt, src=src)
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 5, 6, 8, 12])
    seqs = _spread(rng, 1, 128)
    longest = _spread(rng, 1, 32768)
    while seqs * longest * kv_heads * head_dim > 8 * 32768 * 1024 // 2:
        longest = max(1, longest // 2)
    return dict(kind=kind, seqs=seqs, q_len=rng.choice([1, 1, 1, 2, 3, 5, 8]), heads=kv_heads * group,
                kv_heads=kv_heads, head_dim=head_dim, page=page, longest=longest, ragged=rng.random() < 0.6,
                window=rng.choice([0, 0, 0, 0, 1024]), fmt=fmt, src=src)


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _rows(gen, shape, dtype):
    """Keys or values as a projection gives them: normal, heads of different sizes, a few large channels."""
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((1,) * (len(shape) - 2) + (shape[-2], 1), generator=gen, device=DEV))
    x *= 1 + 5 * (torch.rand(shape[-1], generator=gen, device=DEV) < 0.03)
    return x.to(dtype)


def _places(gen, seqs, each, page):
    """Cache slots of `each` successive positions of every sequence, on pages in no order; and the page count."""
    pages = (each + page - 1) // page + 1
    table = torch.randperm(seqs * pages, generator=gen, device=DEV).view(seqs, pages)
    at = torch.randint(0, page, (seqs, 1), generator=gen, device=DEV) + torch.arange(each, device=DEV)
    return (table.gather(1, at // page) * page + at % page).reshape(-1), seqs * pages


def _encode(x):
    """e4m3 codes (as bytes) and scale bytes of x [..., head_dim] in float32."""
    a = x.abs().amax(-1)
    m, n = torch.frexp(a)
    e = torch.where(a == 0, E_MIN, n - 9 + (m > 0.875).to(n.dtype)).clamp(min=E_MIN)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _decode(codes, scale):
    """Values (float32) of e4m3 codes and their scale bytes."""
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), (scale.to(torch.int32) - 127)[..., None])


def _fill(gen, pages, case):
    """A cache holding drawn keys or values in every slot: (data, scale bytes or None)."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    data = torch.empty(shape, dtype=torch.uint8 if case["fmt"] == "e4m3" else torch.bfloat16, device=DEV)
    scale = torch.empty(shape[:3], dtype=torch.uint8, device=DEV) if case["fmt"] == "e4m3" else None
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pages, step):
        x = _rows(gen, (min(step, pages - i), case["page"], case["kv_heads"], case["head_dim"]), torch.float32)
        x = x.transpose(1, 2)
        if scale is None:
            data[i:i + step] = x.to(torch.bfloat16)
        else:
            data[i:i + step], scale[i:i + step] = _encode(x.to(torch.bfloat16).float())
    return data, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=dict(case))
    kind, dtype = case["kind"], _dtype(case["src"])
    if kind == "verify":
        n, d, v = case["seqs"], case["drafts"], case["vocab"]
        z = 2.5 * torch.randn((n, d + 1, v), generator=gen, device=DEV)
        near = z[:, :d] + 0.4 * torch.randn((n, d, v), generator=gen, device=DEV)
        q = torch.softmax(near, -1).to(dtype)
        noise = torch.rand((n, d, v), generator=gen, device=DEV).clamp_(min=1e-12).log_()
        s["p"] = torch.softmax(z, -1).to(dtype)
        s["drafts"] = (q.float() / -noise).argmax(-1).to(torch.int32) if d else torch.zeros(n, 0, dtype=torch.int32,
                                                                                           device=DEV)
        s["q"] = None if case["one_hot"] else q
        s["u"] = torch.rand((n, d + 1), generator=gen, device=DEV)
        return s
    if kind == "attend":
        n, longest, page = case["seqs"], case["longest"], case["page"]
        lens = torch.full((n,), longest, device=DEV)
        if case["ragged"]:      # lengths spread over a factor of eight, the first the longest
            lens[1:] = (longest * torch.exp2(-3 * torch.rand(n - 1, generator=gen, device=DEV))).long().clamp_(min=1)
        each = (longest + page - 1) // page
        s["table"] = torch.randperm(n * each, generator=gen, device=DEV).view(n, each).to(torch.int32)
        s["lens"] = lens.to(torch.int32)
        q = torch.randn((n, case["q_len"], case["heads"], case["head_dim"]), generator=gen, device=DEV)
        s["q"] = (1.5 * q).to(dtype)
        pages = n * each
    else:
        s["slots"], pages = _places(gen, case["seqs"], case["tokens"] // case["seqs"], case["page"])
        if kind == "store":
            shape = (case["tokens"], case["kv_heads"], case["head_dim"])
            s["new_k"], s["new_v"] = _rows(gen, shape, dtype), _rows(gen, shape, dtype)
    s["k"], s["k_scale"] = _fill(gen, pages, case)
    s["v"], s["v_scale"] = _fill(gen, pages, case)
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_put(data, scale, slots, x):
    """Writes rows x [token][kv head][head_dim] into a cache's slots."""
    page, at = slots // data.shape[2], slots % data.shape[2]
    if scale is None:
        data[page, :, at] = x.to(torch.bfloat16)
    else:
        data[page, :, at], scale[page, :, at] = _encode(x.float())


def _plain_get(data, scale, slots, dtype):
    """The values of a cache's slots, [token][kv head][head_dim]."""
    page, at = slots // data.shape[2], slots % data.shape[2]
    x = data[page, :, at]
    return (x if scale is None else _decode(x, scale[page, :, at])).to(dtype)


def _plain_pages(data, scale, table):
    """The tokens of whole sequences in order, float32 [sequence][kv head][token][head_dim]."""
    x = data[table]
    x = x.float() if scale is None else _decode(x, scale[table])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c, q = s["case"], s["q"].float()
    n, ql, heads, dim = q.shape
    kh, group = c["kv_heads"], heads // c["kv_heads"]
    k = _plain_pages(s["k"], s["k_scale"], s["table"])
    rows = q.view(n, ql, kh, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kh, ql * group, dim)
    logits = torch.matmul(rows, k.transpose(2, 3)) * (1 / math.sqrt(dim))
    del k
    t = torch.arange(logits.shape[-1], device=DEV)
    at = (s["lens"][:, None] - ql + torch.arange(ql, device=DEV)).repeat_interleave(group, 1)[:, None, :, None]
    seen = (t <= at) & (t > at - c["window"]) if c["window"] else t <= at
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    w = torch.exp(logits - top)
    total = w.sum(-1, keepdim=True)
    w = w / total.masked_fill(total == 0, 1)
    v = _plain_pages(s["v"], s["v_scale"], s["table"])
    v = v.masked_fill((t >= s["lens"][:, None])[:, None, :, None], 0)
    out = torch.matmul(w, v)
    return out.view(n, kh, ql, group, dim).permute(0, 2, 1, 3, 4).reshape(n, ql, heads, dim).to(s["q"].dtype)


def _plain_verify(s):
    c, p, drafts, u = s["case"], s["p"], s["drafts"].long(), s["u"].double()
    n, d, v = c["seqs"], c["drafts"], c["vocab"]
    px = p[:, :d].gather(2, drafts[..., None])[..., 0].double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(2, drafts[..., None])[..., 0].double()
    accepted = (u[:, :d] * qx < px).long().cumprod(1).sum(1)
    seq = torch.arange(n, device=DEV)
    top = p[seq, accepted].double()
    w = top
    if d:
        at = accepted.clamp(max=d - 1)
        if s["q"] is None:
            less = torch.zeros_like(top).scatter_(1, drafts.gather(1, at[:, None]), 1.0)
            less = torch.where(less > 0, top, torch.zeros_like(top))
        else:
            less = s["q"][seq, at].double()
        w = torch.where((accepted < d)[:, None], top - less, top)
    w = w.clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, top.clamp(min=0))
    up = w.cumsum(1)
    over = up > u[:, d:] * up[:, -1:]
    token = over.to(torch.uint8).argmax(1)
    i = torch.arange(d + 1, device=DEV)
    tokens = torch.where(i < accepted[:, None], torch.nn.functional.pad(drafts, (0, 1)), -1)
    tokens = torch.where(i == accepted[:, None], token[:, None], tokens)
    return accepted.to(torch.int32), tokens.to(torch.int32)


def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        import weight_streaming_linear_amd as wsl
        if kind == "verify":
            return wsl.verify_drafts(s["p"], s["q"], s["drafts"], s["u"])
        if "cache" not in s:        # the cache's handle: a program makes it with the cache
            e4m3 = torch.float8_e4m3fn
            data = (s["k"], s["v"]) if c["fmt"] == "bf16" else (s["k"].view(e4m3), s["v"].view(e4m3))
            s["cache"] = wsl.KVCache(*data, s["k_scale"], s["v_scale"])
        ofmt = wsl.WSL_OUT_F32 if c["src"] == "f32" else wsl.WSL_OUT_BF16
        if kind == "attend":
            return wsl.attn_decode(s["cache"], s["q"], s["table"], s["lens"], window=c["window"])
        if kind == "store":
            wsl.kv_cache_write(s["cache"], s["new_k"], s["new_v"], s["slots"])
        return wsl.kv_cache_read(s["cache"], s["slots"], ofmt=ofmt)
    if kind == "verify":
        return _plain_verify(s)
    if kind == "attend":
        return _plain_attend(s)
    if kind == "store":
        _plain_put(s["k"], s["k_scale"], s["slots"], s["new_k"])
        _plain_put(s["v"], s["v_scale"], s["slots"], s["new_v"])
    dtype = _dtype(c["src"])
    return (_plain_get(s["k"], s["k_scale"], s["slots"], dtype), _plain_get(s["v"], s["v_scale"], s["slots"], dtype))


def work(case):
    """One pass: every input read once and every output written once."""
    size = 4 if case["src"] == "f32" else 2
    if case["kind"] == "verify":    # one row of p, and of q where there is one, a sequence
        rows = 1 if case["one_hot"] or case["drafts"] == 0 else 2
        return dict(bytes=case["seqs"] * (rows * case["vocab"] * size + case["drafts"] * 20),
                    flops=3 * case["seqs"] * case["vocab"])
    cell = 2 if case["fmt"] == "bf16" else 1 + 1 / case["head_dim"]
    if case["kind"] == "attend":
        n, longest = case["seqs"], case["longest"]
        # the mean of longest * 2^-3x over x in 0..1 for every sequence but the first
        tokens = n * longest if not case["ragged"] else longest + (n - 1) * longest * (1 - 2 ** -3) / (3 * math.log(2))
        if case["window"]:
            tokens = min(tokens, n * (case["window"] + case["q_len"] - 1))
        rows = n * case["q_len"] * case["heads"] * case["head_dim"]
        return dict(bytes=2 * tokens * case["kv_heads"] * case["head_dim"] * cell + 2 * rows * size,
                    flops=4 * tokens * case["q_len"] * case["heads"] * case["head_dim"])
    cells = 2 * case["tokens"] * case["kv_heads"] * case["head_dim"]
    once = cells * (size + cell)
    return dict(bytes=2 * once if case["kind"] == "store" else once, flops=cells)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _e4m3_value(x):
    """x [..., head_dim] in float64, quantised with one power of two for the last axis."""
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(a / 448)).clamp(min=float(E_MIN))
    e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((a <= 448 * torch.exp2(e - 1)) & (e > E_MIN), e - 1, e)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _codes64(data, scale):
    """Values in float64 of e4m3 bytes, by sign, exponent and fraction."""
    if scale is None:
        return data.double()
    b = data.to(torch.int32)
    n, f = (b >> 3) & 15, (b & 7).double()
    x = torch.where(n == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2(n.double() - 7))
    return torch.where(b >= 128, -x, x) * torch.exp2(scale.double() - 127)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "store":
        x = [s["new_k"].double(), s["new_v"].double()]
        return tuple(_e4m3_value(y) if case["fmt"] == "e4m3" else y.to(torch.bfloat16).double() for y in x)
    if case["kind"] == "fetch":
        page, at = s["slots"] // case["page"], s["slots"] % case["page"]
        return tuple(_codes64(s[x][page, :, at], None if case["fmt"] == "bf16" else s[x + "_scale"][page, :, at])
                     for x in ("k", "v"))
    if case["kind"] == "attend":
        n, ql, heads, dim = s["q"].shape
        group = heads // case["kv_heads"]
        out = torch.zeros((n, ql, heads, dim), dtype=torch.float64, device=DEV)
        for b in range(n):
            length = int(s["lens"][b])
            for h in range(case["kv_heads"]):
                pages = s["table"][b].long()
                cell = lambda x: _codes64(s[x][pages, h], None if case["fmt"] == "bf16" else s[x + "_scale"][pages, h])
                k, v = cell("k").reshape(-1, dim), cell("v").reshape(-1, dim)
                for i in range(ql):
                    end = length - ql + i + 1
                    start = max(0, end - case["window"]) if case["window"] else 0
                    if end > start:
                        q = s["q"][b, i, h * group:(h + 1) * group].double()
                        w = torch.softmax(q @ k[start:end].T / math.sqrt(dim), -1)
                        out[b, i, h * group:(h + 1) * group] = w @ v[start:end]
        return out
    import numpy as np
    d, v = case["drafts"], case["vocab"]
    drafts, u = s["drafts"].cpu().numpy(), s["u"].cpu().numpy().astype(np.float64)
    counts = np.zeros(case["seqs"], np.int32)
    tokens = np.full((case["seqs"], d + 1), -1, np.int32)
    for b in range(case["seqs"]):
        r = 0
        while r < d:
            x = int(drafts[b, r])
            q = 1.0 if s["q"] is None else float(s["q"][b, r, x])
            if not u[b, r] * q < float(s["p"][b, r, x]):
                break
            tokens[b, r] = x
            r += 1
        p = s["p"][b, r].double().cpu().numpy()
        w = p.copy()
        if r < d and s["q"] is None:
            w[drafts[b, r]] = 0
        elif r < d:
            w = np.maximum(p - s["q"][b, r].double().cpu().numpy(), 0)
        w = w if w.sum() > 0 else p
        up = np.cumsum(w)
        counts[b], tokens[b, r] = r, min(int(np.searchsorted(up, u[b, d] * up[-1], side="right")), v - 1)
    return torch.from_numpy(counts), torch.from_numpy(tokens)
