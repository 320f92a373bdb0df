"""Attention inputs on which every step but a few counted roundings is exact, so that the bits of the weights
and of the queries show, and the bounds that those roundings give.

Keys are powers of two in one dimension each, values ones in one column each: a score is one product, an
output element one weight.  With eps = 2^-24 (half a step of fp32) and scale_log2 = scale * log2 e:
* a score in the log2 domain, x = (q k) * scale_log2: q k is exact where q's terms hold all its 24 bits;
  the constant and the product round once each: |x| * 2 eps.
* a weight exp2(x - m) for the maximum m: that difference rounds once, the exponential is good to 2^-22.
* the sum l of T weights: T eps, and each weight's own error once more; 1 / l and the last product round
  once each, the division being good to 2.5 steps: 6 eps.
"""

import numpy as np

EPS = 2.0 ** -24
DIM, TOKENS = 32, 8


def split(x, terms):
    """x (fp32) as a sum of bf16 numbers, each the nearest to what is left; what they add up to (float64)."""
    import torch
    left = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    total = torch.zeros_like(left, dtype=torch.float64)
    for _ in range(terms):
        t = left.to(torch.bfloat16).float()
        total += t.double()
        left = left - t
    return total.numpy()


def weight_case(seed, rows, f32_queries):
    """q [rows][DIM], keys, values [TOKENS][DIM]: scores within +-1, so that every weight counts."""
    import torch
    g = np.random.default_rng([2026, 13, seed])
    q = g.uniform(-1, 1, (rows, DIM)).astype(np.float32)
    if not f32_queries:
        q = torch.from_numpy(q).to(torch.bfloat16).float().numpy()
    k, v = np.zeros((TOKENS, DIM), np.float32), np.zeros((TOKENS, DIM), np.float32)
    for t in range(TOKENS):
        k[t, 3 * t] = 2.0 ** (t % 3 - 2)
        v[t, 4 * t + 1] = 1
    return q, k, v


def weight_bound(q, k, scale, out):
    x = np.abs(scale * (q.astype(np.float64) @ k.T.astype(np.float64))) * np.log2(np.e)
    top = x.max(-1, keepdims=True)
    ds = np.log(2) * (2 * top * 2 * EPS + 2 * top * EPS)       # of x - m, both with their roundings, and the difference's
    rel = 2 * (ds + 2.0 ** -22) + (TOKENS + 6) * EPS           # its own and those in the sum
    return np.abs(out) * rel * (1 + 1e-4)


def query_case(seed, rows):
    """Large fp32 queries over one token: the log of the sum is the score itself."""
    g = np.random.default_rng([2026, 14, seed])
    q = (g.uniform(20, 90, (rows, DIM)) * g.choice([-1, 1], (rows, DIM))).astype(np.float32)
    k = np.zeros((1, DIM), np.float32)
    k[0, 5] = 0.5
    return q, k


def query_bound(lse):
    return np.abs(lse) * 4 * EPS * (1 + 1e-4) + 1e-30          # two constants and two products round


def emulate(q, k, v, scale, q_terms, p_terms):
    """The documented computation in fp32 with so many bf16 terms: (out, lse)."""
    f = np.float32
    scale_log2 = f(np.float64(f(scale)) * 1.44269504088896340736)
    x = (split(q, q_terms) @ k.T.astype(np.float64)).astype(f) * scale_log2
    m = x.max(-1, keepdims=True)
    p = np.exp2((x - m).astype(f)).astype(f)
    l = p[:, :1].copy()
    for t in range(1, p.shape[1]):
        l = l + p[:, t:t + 1]
    out = (split(p, p_terms) @ v.astype(np.float64)).astype(f) * (f(1) / l)
    return out, ((m + np.log2(l)) * f(0.69314718055994530942))[:, 0]
