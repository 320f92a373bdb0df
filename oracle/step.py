"""fp64 references for what a decode step does beside its linear layers: pages, rotary positions,
sampling and low-rank adapters.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* Pages: lists and loops, one sequence and one page after the other.
* Rotary: a complex multiplication by amplitude * exp(i p f).
* Sampling: rows sorted by (logit descending, index ascending), the kept beginning counted out.
* Adapters: two products a row.

The bounds count the roundings that the documented computation makes at most; none is fitted to a
result.
"""

import math

import numpy as np

EPS32 = 2.0 ** -24      # half a step of binary32, relative
HALF_BF16 = 2.0 ** -8   # and of bf16
STATUS_INDEX, STATUS_PAGES = 4, 32


class Pages:
    """kv_pages_grow and kv_pages_trim over Python lists."""

    def __init__(self, table, lens, free, n_free, page_size):
        self.table = [list(map(int, r)) for r in table]
        self.lens, self.free = list(map(int, lens)), list(map(int, free))
        self.n_free, self.page = int(n_free), int(page_size)
        self.status = 0

    def room(self):
        return min(len(self.table[0]) * self.page, 2 ** 31 - 1) if self.table else 0

    def _stack(self):
        if not 0 <= self.n_free <= len(self.free):
            self.status |= STATUS_INDEX
            self.n_free = min(max(self.n_free, 0), len(self.free))

    def grow(self, new, n_tokens):
        """(slots, positions, starts) of lists of new tokens."""
        slots, positions, starts = [-1] * n_tokens, [-1] * n_tokens, []
        if self.table:
            self._stack()
        start, asked, top = 0, 0, self.n_free
        for b, w in enumerate(new):
            begins = start
            starts.append(min(begins, n_tokens))
            start += max(w, 0)
            n = self.lens[b]
            if n < 0 or w < 0 or n > self.room() or n + w > self.room() or (w > 0 and start > n_tokens):
                self.status |= STATUS_INDEX
                continue
            held, now = -(-n // self.page), -(-(n + w) // self.page)
            asked += now - held
            if now > held and asked > top:
                self.status |= STATUS_PAGES
                continue
            for place in range(held, now):
                self.n_free -= 1
                self.table[b][place] = self.free[self.n_free]
            for i in range(w):
                page = self.table[b][(n + i) // self.page]
                positions[begins + i] = n + i
                if 0 <= page < len(self.free):
                    slots[begins + i] = page * self.page + (n + i) % self.page
                else:
                    self.status |= STATUS_INDEX
            self.lens[b] += w
        return slots, positions, starts + [min(start, n_tokens)]

    def trim(self, to):
        back = []
        self._stack()
        for b, w in enumerate(to):
            n = self.lens[b]
            if n < 0 or n > self.room() or w < 0:
                self.status |= STATUS_INDEX
                continue
            if w < n:
                back += self.table[b][-(-w // self.page):-(-n // self.page)]
                self.lens[b] = w
        for i, page in enumerate(back):
            at = self.n_free + len(back) - 1 - i
            if at < len(self.free):
                self.free[at] = page
            else:
                self.status |= STATUS_INDEX
        self.n_free = min(self.n_free + len(back), len(self.free))


def rotary_ref(x, positions, freqs, interleaved=False, amplitude=1.0):
    """x [tokens][heads][dim] turned; returns (out, the bound's |a cos| + |b sin|)."""
    x = np.asarray(x, dtype=np.float64)
    half = len(freqs)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    # p * f in extended precision where there is one; the fp64 product is within 2^-53 of it
    angle = np.asarray(positions, dtype=np.longdouble)[:, None, None] * np.asarray(freqs, dtype=np.longdouble)
    c, s = (amplitude * np.cos(angle)).astype(np.float64), (amplitude * np.sin(angle)).astype(np.float64)
    out, parts = x.copy(), np.abs(x)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    parts[..., first], parts[..., second] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return out, parts


def rotary_bound(x, ref, parts, positions, freqs, interleaved, amplitude, bf16):
    """cos and sin: rounded to binary32 (half a step), their series and the angle before (2^-33, and
    2^-52 of |p f|) times the amplitude; two products and a sum rounded; then the output's type."""
    half = len(freqs)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    near = np.zeros(ref.shape)
    far = np.abs(np.asarray(positions, dtype=np.float64))[:, None, None] * np.asarray(freqs) * 2.0 ** -52 + 2.0 ** -32
    ab = (np.abs(x[..., first]) + np.abs(x[..., second])) * abs(amplitude) * far
    near[..., first] = near[..., second] = ab
    turned = np.zeros(ref.shape[-1], dtype=bool)
    turned[:2 * half] = True
    bound = np.where(turned, (3 * EPS32 * parts + near) * (1 + 2.0 ** -20) + 2.0 ** -148, 0)
    return bound + (HALF_BF16 * (np.abs(ref) + bound) if bf16 else 0)


def _two_pi(bits):
    """2 pi * 2^bits, cut off: pi = 16 atan(1/5) - 4 atan(1/239) (Machin), in whole numbers."""
    guard = 32

    def atan_inverse(n):
        term = (1 << (bits + guard)) // n
        total, k, sign = term, 1, -1
        while term:
            term //= n * n
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    return 2 * (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> guard


def turn_ref(positions, freqs):
    """(cos, sin) of position * frequency, [len(positions)][len(freqs)]: the product of the two as whole
    numbers and the angle left of whole turns of it, so that nothing is lost at any size (to 2^-52)."""
    bits = 320
    turn = _two_pi(bits)
    out = np.empty((2, len(positions), len(freqs)))
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            num, den = float(f).as_integer_ratio()
            angle = ((int(p) * num) << bits) // den % turn
            angle = math.ldexp(angle - turn if 2 * angle > turn else angle, -bits)
            out[:, i, j] = math.cos(angle), math.sin(angle)
    return out[0], out[1]


def sample_ref(z, u=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probabilities) of one row of logits (float64 values of its type); settings are floats
    that fp32 holds."""
    z = np.asarray(z, dtype=np.float64)
    v = len(z)
    probs = np.zeros(v)
    if np.isnan(z).any() or np.isposinf(z).any() or not np.isfinite(z).any():
        return -1, probs
    order = np.lexsort((np.arange(v), -z))
    order = order[np.isfinite(z[order])]
    if not temperature > 0 or top_p <= 0:
        order = order[:1]
    elif top_k > 0:
        order = order[:top_k]
    t = temperature if temperature > 0 else 1.0
    w = np.exp((z[order] - z[order[0]]) / t)
    keep = np.ones(len(w), dtype=bool)
    if top_p < 1:
        keep &= np.concatenate(([0.0], np.cumsum(w)[:-1])) < top_p * math.fsum(w)
    if min_p > 0:
        keep &= w >= min_p
    keep[0] = True
    assert not (np.diff(keep.astype(int)) > 0).any()       # a beginning of the order
    kept = np.sort(order[keep])
    w = np.exp((z[kept] - z[order[0]]) / t)
    probs[kept] = w / math.fsum(w)
    if u is None:
        return None, probs
    up = np.cumsum(w)
    over = np.nonzero((up > max(u, 0.0) * up[-1]) & (w > 0))[0]
    return int(kept[over[0]] if len(over) else kept[np.nonzero(w > 0)[0][-1]]), probs


def lora_ref(base, x, a, b, ids, scales=None):
    """(out, bound of the fp32 computation before the last rounding): sums in any order make at most
    (terms - 1) roundings a term, each relative EPS32 of what it has added up."""
    base, x, a, b = (np.asarray(t, dtype=np.float64) for t in (base, x, a, b))
    rank, k = a.shape[1:]
    out, bound = base.copy(), np.zeros(base.shape)
    for t, i in enumerate(ids):
        if not 0 <= i < len(a):
            continue
        s = 1.0 if scales is None else float(scales[i])
        h, h_abs = a[i] @ x[t], np.abs(a[i]) @ np.abs(x[t])
        out[t] += s * (b[i] @ h)
        # the scale and its product, and the three parts of h on the matrix cores (24 bits): 4 more
        h_err = (k + 4) * EPS32 * h_abs
        bound[t] = abs(s) * (np.abs(b[i]) @ (h_err * (1 + 2.0 ** -8) + (3 * rank + 2) * EPS32 * np.abs(h)))
        bound[t] += EPS32 * (np.abs(out[t]) + bound[t])
    return out, bound
