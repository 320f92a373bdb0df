"""The references for cache, attention and verification against other ways to the same numbers (CPU)."""

import numpy as np
import pytest
import torch

import oracle.decode as od
from decode_cases import probabilities


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, od.e4m3_table(), equal_nan=True)


def test_e4m3_encode_is_torchs_rounding():
    g = np.random.default_rng(1)
    x = np.concatenate([g.uniform(-448, 448, 4000), g.standard_normal(4000) * 0.01, od.e4m3_table()[:0x7f],
                        (od.e4m3_table()[:0x7e] + od.e4m3_table()[1:0x7f]) / 2, [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(od.e4m3_encode(x), want)


def test_scale_exponent_by_frexp():
    a = np.concatenate([np.exp2(np.random.default_rng(2).uniform(-126, 127, 3000)), [0.0, 448.0, 448.1, 1.75, 1.76]])
    m, n = np.frexp(a)
    want = np.where(a == 0, od.E_MIN, np.maximum(n - 9 + (m > 0.875), od.E_MIN))
    assert np.array_equal(od.kv_scale_exponent(a), want)


def test_encoded_rows_are_within_half_a_step():
    x = np.random.default_rng(3).standard_normal((200, 128)) * np.exp2(np.arange(200) - 100)[:, None]
    y = od.kv_decode(*od.kv_encode(x))
    # 2^-4 of the value, or half the smallest step of the row's scale
    assert (np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.abs(x).max(-1, keepdims=True) / 224 * 2.0 ** -10)).all()
    assert np.isnan(od.kv_decode(*od.kv_encode(np.array([[1.0, np.inf]])))).all()


@pytest.mark.parametrize("ql,length,window", [(1, 1, 0), (1, 50, 0), (3, 50, 0), (4, 2, 0), (5, 60, 16), (2, 0, 0)])
def test_attention_against_torch(ql, length, window):
    g = np.random.default_rng(4)
    q, k, v = g.standard_normal((ql, 6, 32)), g.standard_normal((80, 2, 32)), g.standard_normal((80, 2, 32))
    out, lse, _ = od.attn_ref(q, k, v, length, 0.2, window)
    tq, tk, tv = (torch.from_numpy(t).transpose(0, 1) for t in (q, k[:length], v[:length]))
    t = torch.arange(length)
    at = length - ql + torch.arange(ql)[:, None]
    see = (t <= at) & ((t > at - window) if window else True)
    s = (tq @ tk.repeat_interleave(3, 0).transpose(1, 2) * 0.2).masked_fill(~see, -np.inf)
    some = see.any(-1)
    want = (torch.softmax(s, -1) @ tv.repeat_interleave(3, 0)).transpose(0, 1)
    assert np.allclose(out[some.numpy()], want[some].numpy(), rtol=1e-12, atol=1e-12)
    assert (out[~some.numpy()] == 0).all() and np.isneginf(lse[~some.numpy()]).all()
    assert np.allclose(lse[some.numpy()], torch.logsumexp(s, -1).T[some].numpy(), rtol=1e-12)


def test_verification_gives_the_targets_distribution():
    """Over a grid of random numbers the token after 0 drafts, and after one, follows p exactly as
    finely as the grid: |share - p| <= a few grid steps."""
    g = np.random.default_rng(5)
    p, q = probabilities(g, 1, 2, 7, 1.0)[0], probabilities(g, 1, 1, 7, 1.0)[0]
    n = 64
    us = (np.arange(n) + 0.5) / n
    share = np.zeros(7)
    for x in range(7):                      # the draft, with its probability under q
        for a in us:
            for b in us:
                r, t = od.verify_ref(p, q, [x], np.array([a, b]), 1, 7)
                share[t[0]] += q[0][x] / (n * n)
    assert np.abs(share - p[0]).max() < 8 / n
    hits = np.bincount([od.verify_ref(p, None, [0], np.array([0.0, a]), 0, 7)[1][0] for a in us], minlength=7) / n
    assert np.abs(hits - p[0]).max() <= 1 / n


@pytest.mark.parametrize("what", ["scale_tie", "code_tie", "mask", "window", "accept", "residual"])
def test_a_planted_mistake_shows(monkeypatch, what):
    """Each reference is sharp: a mistake planted in it changes what it gives on these inputs."""
    g = np.random.default_rng(6)
    if what == "scale_tie":
        good = od.kv_encode(np.full((1, 16), 448.0))
        monkeypatch.setattr(od, "kv_scale_exponent", lambda a: np.floor(np.log2(np.maximum(a, 1e-30) / 448)).astype(int) + 1)
        assert not np.array_equal(good[1], od.kv_encode(np.full((1, 16), 448.0))[1])
    elif what == "code_tie":
        x = np.array([1.0625, 1.1875])      # halfway: down to 1.0, up to 1.25
        assert np.array_equal(od.e4m3_table()[od.e4m3_encode(x)], [1.0, 1.25])
    elif what in ("mask", "window"):
        q, k, v = g.standard_normal((2, 1, 16)), g.standard_normal((9, 1, 16)), g.standard_normal((9, 1, 16))
        good = od.attn_ref(q, k, v, 9, 0.25, 4)[0]
        other = od.attn_ref(q, k, v, 8 if what == "mask" else 9, 0.25, 4 if what == "mask" else 5)[0]
        assert np.abs(good - other).max() > 1e-3
    else:
        p, q = np.array([[0.5, 0.5], [0.5, 0.5]]), np.array([[0.5, 0.5]])
        if what == "accept":                # strict: u q < p
            assert od.verify_ref(p, q, [0], np.array([1.0, 0.1]), 1, 2)[0] == 0
            assert od.verify_ref(p, q, [0], np.array([0.99, 0.1]), 1, 2)[0] == 1
        else:                               # nothing left: p itself
            assert od.verify_ref(p, q, [0], np.array([1.0, 0.6]), 1, 2)[1].tolist() == [1, -1]
