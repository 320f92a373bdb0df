"""fp64 references for the key-value cache, its attention and draft verification.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* e4m3 is taken from its table of 256 values (1 sign, 4 exponent bits with bias 7, 3 fraction
  bits, no infinities, all ones = NaN), and a number is encoded by search in that table: the
  nearest value, the even code on a tie.
* A cached row x has the scale 2^e, e the least integer >= -110 with max|x| <= 448 * 2^e.
* Attention: softmax over the tokens a query sees, computed from the definition per row.
* Verification: the definition, draft by draft and entry by entry.

Tolerances (``attn_bound``) count the roundings that the documented computation makes at most,
over all its variants (the weights' 16 bits beside bf16 queries among them); none is fitted to a
result.  Whether a variant has more bits than that shows on inputs where nearly nothing else rounds
(tests/precision_cases.py).
"""

import numpy as np

E_MIN = -110
EPS32 = 2.0 ** -24      # half a step of binary32


def e4m3_table():
    """The 256 values of e4m3, NaN at 0x7f and 0xff."""
    out = np.empty(256)
    for b in range(256):
        n, f = (b >> 3) & 15, b & 7
        x = f * 2.0 ** -9 if n == 0 else (1 + f / 8) * 2.0 ** (n - 7)
        if b & 0x7f == 0x7f:
            x = np.nan
        out[b] = -x if b & 0x80 else x
    return out


def e4m3_encode(x):
    """Codes of float64 numbers within +-448: nearest, ties to the even code; the sign is kept."""
    x = np.asarray(x, dtype=np.float64)
    grid = e4m3_table()[:0x7f]                       # 0 .. 448, ascending
    a = np.abs(x)
    hi = np.minimum(np.searchsorted(grid, a), 0x7e)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - grid[lo], grid[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)


def kv_scale_exponent(a):
    """The least integer e >= E_MIN with a <= 448 * 2^e (float64 a, finite), by trial."""
    a = np.asarray(a, dtype=np.float64)
    e = np.full(a.shape, E_MIN, dtype=np.int64)
    for _ in range(300):
        more = a > 448.0 * np.exp2(e.astype(np.float64))
        if not more.any():
            return e
        e = e + more
    raise ValueError("not finite")


def kv_encode(x):
    """(codes, scale bytes) of rows x [..., head_dim]; a row that is not finite is all NaN."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x).all(-1)
    y = np.where(fine[..., None], x, 0.0)
    e = kv_scale_exponent(np.abs(y).max(-1))
    codes = e4m3_encode(y * np.exp2(-e.astype(np.float64))[..., None])
    return np.where(fine[..., None], codes, 0x7f).astype(np.uint8), np.where(fine, e + 127, 127).astype(np.uint8)


def kv_decode(codes, scale):
    """Values (float64) of codes [..., head_dim] with scale bytes [...]."""
    return e4m3_table()[codes] * np.exp2(scale.astype(np.float64) - 127)[..., None]


def attn_ref(q, k, v, length, scale, window=0):
    """Attention of one sequence: q [q_len][n_heads][D], k, v [tokens][n_kv][D] (the first `length`
    count).  Returns (out, lse, weighted): out [q_len][n_heads][D], lse [q_len][n_heads] and, for
    the bound, {"pv": sum p |V|, "score": max sum |scale q k|} per row."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    ql, nh, dim = q.shape
    group = nh // k.shape[1]
    out, lse = np.zeros((ql, nh, dim)), np.full((ql, nh), -np.inf)
    pv, score = np.zeros((ql, nh, dim)), np.zeros((ql, nh))
    for i in range(ql):
        pos = length - ql + i
        lo = max(0, pos - window + 1) if window else 0
        if pos < 0:
            continue
        for h in range(nh):
            kk, vv = k[lo:pos + 1, h // group], v[lo:pos + 1, h // group]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (kk @ q[i, h])
                m = s.max()
                p = np.exp(s - m)
                out[i, h] = (p / p.sum()) @ vv
                lse[i, h] = m + np.log(p.sum())
                pv[i, h] = (p / p.sum()) @ np.abs(vv)
                score[i, h] = np.abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, {"pv": pv, "score": score}


def attn_bound(extra, dim, tokens, ref, half_step):
    """|out - ref| allowed for the documented computation, whatever the queries' type: products accumulated in binary32 over
    dim terms (queries in 24 bits), one multiplication by the scale, an exponential good to
    2^-22, weights in 16 bits, a sum over `tokens` terms in binary32 with at most one rescale per
    32 of them, one division, and the result's own rounding."""
    ds = extra["score"] * (dim + 8) * EPS32             # absolute error of a score
    rel = 2 * ds + 2.0 ** -15 + (2 * tokens + 64) * EPS32
    return rel[..., None] * extra["pv"] * 1.01 + np.abs(ref) * half_step + 1e-30


def lse_bound(extra, dim, tokens, ref):
    ds = extra["score"] * (dim + 8) * EPS32
    return 2 * ds + (2 * tokens + 64) * EPS32 + 8 * np.abs(np.where(np.isfinite(ref), ref, 0)) * EPS32


def verify_ref(p, q, drafts, u, n, vocab):
    """One sequence: p [width + 1][vocab], q [width][vocab] or None, drafts [width], u [width + 1];
    the first n drafts count.  Returns (accepted, tokens [width + 1])."""
    width = len(u) - 1
    n = min(max(int(n), 0), width)
    tokens = np.full(width + 1, -1, dtype=np.int32)
    r = 0
    while r < n:
        x = int(drafts[r])
        if not 0 <= x < vocab:
            break
        qx = 1.0 if q is None else float(q[r][x])
        if not float(u[r]) * qx < float(p[r][x]):
            break
        tokens[r] = x
        r += 1
    top = np.asarray(p[r], dtype=np.float64)
    top = np.where(top > 0, top, 0.0)
    w = top.copy()
    if r < n:
        if q is None:
            if 0 <= int(drafts[r]) < vocab:
                w[int(drafts[r])] = 0.0
        else:
            with np.errstate(invalid="ignore"):
                d = np.asarray(p[r], dtype=np.float64) - np.asarray(q[r], dtype=np.float64)
            w = np.where(d > 0, d, 0.0)
    if not w.sum() > 0:
        w = top
    total = w.sum()
    if not (total > 0 and np.isfinite(total)):
        return r, tokens
    target = max(float(u[width]) * total, 0.0) if u[width] == u[width] else np.inf
    up = np.cumsum(w)
    over = np.nonzero((up > target) & (w > 0))[0]
    tokens[r] = over[0] if len(over) else np.nonzero(w > 0)[0][-1]
    return r, tokens
