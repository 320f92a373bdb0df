"""Calls at the edges of what the cache, attention and verification calls take, on the GPU."""

import numpy as np
import pytest

import oracle.decode as od
import weight_streaming_linear_amd as wsl
from decode_cases import CacheCase, f32_of, probabilities
from gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,width", [(2, 3), (1, 3), (4, 1), (1, 1)])
@pytest.mark.parametrize("vocab", [501, 40009])
def test_a_drafter_with_one_distribution_for_every_position(n, width, vocab):
    """A broadcast q is refused, never taken for no q at all; copied out it gives what the definition does."""
    import torch
    say(f"verify, one q for all: n={n} width={width} vocab={vocab}")
    g = np.random.default_rng([2026, 12, n, width])
    p = torch.from_numpy(probabilities(g, n, width + 1, vocab)).cuda()
    one = torch.from_numpy(probabilities(g, 1, 1, vocab)).cuda()
    q = one.expand(n, width, vocab)
    drafts = torch.from_numpy(g.integers(0, vocab, (n, width)).astype(np.int32)).cuda()
    u = torch.from_numpy(g.random((n, width + 1)).astype(np.float32)).cuda()
    if n * width > 1:
        for a, b in ((p, q), (p[:1, :1].expand(n, width + 1, vocab), q.contiguous())):
            with pytest.raises(ValueError):
                wsl.verify_drafts(a, b, drafts, u)
    acc, tok = wsl.verify_drafts(p, q.contiguous(), drafts, u)
    for b in range(n):
        r, t = od.verify_ref(f32_of(p)[b], f32_of(q)[b], drafts[b].cpu().numpy(), u[b].cpu().numpy(), width, vocab)
        assert acc[b].item() == r and np.array_equal(tok[b].cpu().numpy(), t)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ql", [1, 5])
@pytest.mark.parametrize("lens,window,page,wide", [
    ([500, 400, 385, 384, 383, 260, 129, 128, 90, 3], 100, 16, 0), ([511, 300, 257, 200], 33, 24, 0),
    ([1100, 1151, 1152, 1153, 1279, 1280, 1281, 1025, 1024, 700], 1024, 16, 0), ([130, 3000, 40, 555], 1, 7, 100),
    ([4099], 300, 16, 500)])
def test_pages_behind_the_window_may_be_gone(lens, window, page, wide, ql, e4m3):
    """Table entries of pages that no query sees any more are -1, wherever the window begins in a tile:
    nothing is reported.  A page that some query sees is; in whole items and in shares."""
    import torch
    heads, n_kv, dim = 4, 2, 64
    say(f"attn window {window} q_len={ql} page={page} e4m3={e4m3} lens={lens[:5]} wide={wide}")
    c = CacheCase(80 + ql, lens, n_kv, dim, page, e4m3, "cuda")
    lowest = [max(0, n - ql - window + 1) for n in lens]
    for b, lo in enumerate(lowest):
        c.table[b, :lo // page] = -1
    c.table = torch.cat((c.table, torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")), 1)
    q = torch.randn((len(lens), ql, heads, dim), device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(bad=None):
        out = f32_of(wsl.attn_decode(c.cache, q, c.table, c.kv_lens, window=window, status=st))
        for b, n in enumerate(lens):
            if b != bad:
                ref, _, extra = od.attn_ref(f32_of(q)[b], c.values[0][b], c.values[1][b], n, dim ** -0.5, window)
                assert (np.abs(out[b] - ref) <= od.attn_bound(extra, dim, n, ref, 2.0 ** -8)).all(), f"sequence {b}"

    check()
    assert st.item() == 0
    for b in range(len(lens)):      # the page of the lowest token that is seen, and that of the newest
        for at in (lowest[b] // page, (lens[b] - 1) // page):
            st.zero_()
            was, c.table[b, at] = c.table[b, at].item(), -1
            check(b)
            assert st.item() == wsl.WSL_STATUS_INDEX, f"sequence {b}"
            c.table[b, at] = was


def test_the_example_goes_past_a_thousand_tokens(monkeypatch, capsys):
    """All drafts of the target itself stand, so its sequences grow to about 100 + 1100 tokens."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    say("example: 1 layer, 2 sequences, 1100 tokens")
    monkeypatch.setattr("sys.argv", ["speculative_decode.py", "--tokens", "1100", "--width", "10", "--layers", "1",
                                     "--seqs", "2", "--e4m3"])
    ex.main()
    assert "the target itself" in capsys.readouterr().out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [0, 100])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 + 7, 2 ** 63 - 1, 2 ** 64 + 3])
def test_a_window_without_an_end(window, wide, e4m3):
    """Windows of any size, among them those larger than every position, beside sequences shorter than q_len."""
    import torch
    lens = [0, 1, 2, 3, 4, 5, 6, 9, 300]
    say(f"attn window {window} e4m3={e4m3} wide={wide}")
    c = CacheCase(90, lens, 2, 64, 16, e4m3, "cuda")
    c.table = torch.cat((c.table, torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")), 1)
    q = torch.randn((len(lens), 5, 4, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = wsl.attn_decode(c.cache, q, c.table, c.kv_lens, window=window, status=st)
    assert st.item() == 0
    assert torch.equal(got, wsl.attn_decode(c.cache, q, c.table, c.kv_lens))
    for b, n in enumerate(lens):
        ref, _, extra = od.attn_ref(f32_of(q)[b], c.values[0][b], c.values[1][b], n, 0.125)
        assert (np.abs(f32_of(got)[b] - ref) <= od.attn_bound(extra, 64, n, ref, 2.0 ** -8)).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), 1.0])
@pytest.mark.parametrize("wide", [0, 100])
def test_rows_whose_scores_are_all_minus_infinity_are_zero(f32, odd, wide):
    """Whatever the values are that they weigh with zero; other sequences beside them as ever."""
    import torch
    lens = [40, 700, 129]
    say(f"attn scores of -inf f32={f32} values {odd} wide={wide}")

    def kfill(b, x):
        if b < 2:
            x[:, :, 0] = -np.inf

    def vfill(b, x):
        if b < 2:
            x[:, :, 3] = odd

    c = CacheCase(95, lens, 2, 64, 16, False, "cuda", k_fill=kfill, v_fill=vfill)
    c.table = torch.cat((c.table, torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")), 1)
    q = torch.randn((3, 2, 4, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    q[..., 0] = q[..., 0].abs() + 0.5
    q = q if f32 else q.to(torch.bfloat16)
    lse = torch.zeros(q.shape[:3], device="cuda")
    out = wsl.attn_decode(c.cache, q, c.table, c.kv_lens, lse=lse)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    ref, rl, extra = od.attn_ref(f32_of(q)[2], c.values[0][2], c.values[1][2], 129, 0.125)
    assert (np.abs(f32_of(out)[2] - ref) <= od.attn_bound(extra, 64, 129, ref, 2.0 ** (-24 if f32 else -8))).all()


def _dyadic_cache(k, v, dim, e4m3):
    """A cache of one page that holds rows k, v (padded to dim) exactly."""
    import torch
    pad = [np.zeros((16, dim), np.float32) for _ in range(2)]
    for to, x in zip(pad, (k, v)):
        to[:len(x), :x.shape[1]] = x
    rows = [torch.from_numpy(x).cuda()[:, None] for x in pad]
    cache = wsl.KVCache.empty(1, 1, 16, dim, wsl.WSL_KV_E4M3 if e4m3 else wsl.WSL_KV_BF16)
    slots = torch.arange(16, device="cuda")
    wsl.kv_cache_write(cache, *rows, slots)
    back = wsl.kv_cache_read(cache, slots, ofmt=wsl.WSL_OUT_F32)
    assert all(torch.equal(a, b) for a, b in zip(rows, back))
    return cache


def _check_weights_bits(f32, dim, rows, wide, e4m3):
    import torch
    import precision_cases as pc
    say(f"attn weights' bits f32={f32} dim={dim} rows={rows} wide={wide} e4m3={e4m3}")
    q, k, v = pc.weight_case(dim + rows, rows, f32)
    cache = _dyadic_cache(k, v, dim, e4m3)
    qt = torch.zeros((1, 1, rows, dim), device="cuda")
    qt[0, 0, :, :pc.DIM] = torch.from_numpy(q)
    out = wsl.attn_decode(cache, qt if f32 else qt.to(torch.bfloat16), torch.zeros((1, wide), dtype=torch.int32, device="cuda"),
                          torch.tensor([pc.TOKENS], dtype=torch.int32, device="cuda"), scale=0.5, ofmt=wsl.WSL_OUT_F32)
    ref, _, _ = od.attn_ref(q[None], k[:, None], v[:, None], pc.TOKENS, 0.5)
    got = f32_of(out)[0, 0]
    assert (got[:, pc.DIM:] == 0).all()
    err, bound = np.abs(got[:, :pc.DIM] - ref[0]), pc.weight_bound(q, k, 0.5, ref[0])
    assert (err <= bound).all(), f"{(err[bound > 0] / bound[bound > 0]).max()} of the bound"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [32, 64, 128, 192, 256])
@pytest.mark.parametrize("rows", [5, 64])
@pytest.mark.parametrize("wide", [1, 4200])
def test_results_of_fp32_queries_have_the_weights_bits(dim, rows, wide, e4m3):
    _check_weights_bits(True, dim, rows, wide, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [32, 64, 128, 192, 256])
@pytest.mark.parametrize("rows", [5, 64])
@pytest.mark.parametrize("wide", [1, 4200])
def test_fp32_results_of_bf16_queries_have_the_weights_bits(dim, rows, wide, e4m3):
    _check_weights_bits(False, dim, rows, wide, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [32, 64, 128, 192, 256])
@pytest.mark.parametrize("rows", [5, 64])
def test_fp32_queries_keep_their_bits(dim, rows, e4m3):
    import torch
    import precision_cases as pc
    say(f"attn queries' bits dim={dim} rows={rows} e4m3={e4m3}")
    q, k = pc.query_case(dim + rows, rows)
    cache = _dyadic_cache(k, k, dim, e4m3)
    qt = torch.zeros((1, 1, rows, dim), device="cuda")
    qt[0, 0, :, :pc.DIM] = torch.from_numpy(q)
    lse = torch.zeros((1, 1, rows), device="cuda")
    wsl.attn_decode(cache, qt, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                    torch.ones(1, dtype=torch.int32, device="cuda"), scale=0.7, lse=lse)
    _, ref, _ = od.attn_ref(q[None], k[:, None], k[:, None], 1, np.float64(np.float32(0.7)))
    err, bound = np.abs(f32_of(lse)[0, 0] - ref[0]), pc.query_bound(ref[0])
    assert (err <= bound).all(), f"{(err / bound).max()} of the bound"


def _items_in_parts(lens, n_kv, workers, cost=2, tile=128):
    """How many (sequence, kv head) items lie in the shares of two workers or more, by the arithmetic of the
    split: an item is its tiles and `cost` units for its beginning, all items in a row are cut into equal shares."""
    units = [max(1, -(-n // tile)) + cost for n in lens for _ in range(n_kv)]
    each = -(-sum(units) // workers)
    at, parts = 0, 0
    for n in units:
        parts += (at + cost) // each != (at + n - 1) // each     # (a share that ends in the beginning holds no part)
        at += n
    return parts


def _some(n, *lens):
    return [int(x) for x in np.random.default_rng([2026, 15, n]).choice(lens, n)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,heads,n_kv,dim,ql", [
    (_some(786, 140, 700, 1100), 2, 1, 16, 1),      # one row tile: more items than the most workgroups (768)
    (_some(260, 300, 1300, 0, 77), 6, 3, 32, 1),
    (_some(80, 900, 130, 2000, 1), 128, 1, 16, 3),  # 384 rows: several row tiles, fewer workgroups for each
    (_some(90, 1500, 40, 700), 40, 2, 128, 8)])
def test_parts_of_more_items_than_workgroups(lens, heads, n_kv, dim, ql, e4m3):
    """What is to be joined is then kept by worker, not by item."""
    import torch
    row_tiles = -(-heads // n_kv * ql // 32)        # at least
    most = max(8, 768 // row_tiles)
    assert len(lens) > 64 and len(lens) * n_kv > most
    assert all(_items_in_parts(lens, n_kv, w) > 0 for w in range(8, most + 1, 8))
    say(f"attn {len(lens) * n_kv} items heads={heads}/{n_kv} dim={dim} q_len={ql} e4m3={e4m3}")
    c = CacheCase(100 + dim, lens, n_kv, dim, 16, e4m3, "cuda")
    c.table = torch.cat((c.table, torch.full((len(lens), 100), -1, dtype=torch.int32, device="cuda")), 1)
    q = torch.randn((len(lens), ql, heads, dim), device="cuda", generator=torch.Generator("cuda").manual_seed(8)).to(torch.bfloat16)
    n = wsl.attn_decode_workspace_bytes(1, len(lens), ql, heads, n_kv, dim, c.table.shape[1], 16)
    assert n > 0
    ws = torch.full((n // 4,), float("nan"), device="cuda")
    lse, st = torch.full(q.shape[:3], float("nan"), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    first = wsl.attn_decode(c.cache, q, c.table, c.kv_lens, lse=lse, workspace=ws, status=st)
    assert torch.equal(first, wsl.attn_decode(c.cache, q, c.table, c.kv_lens, workspace=ws)) and st.item() == 0
    got, glse, q64 = f32_of(first), f32_of(lse), f32_of(q)
    for b, length in enumerate(lens):
        if b % 3 and b > 40 and b < len(lens) - 20:         # (the reference takes the time here)
            continue
        ref, rl, extra = od.attn_ref(q64[b], c.values[0][b], c.values[1][b], length, dim ** -0.5)
        assert (np.abs(got[b] - ref) <= od.attn_bound(extra, dim, length, ref, 2.0 ** -8)).all(), f"sequence {b}"
        assert np.array_equal(np.isneginf(glse[b]), np.isneginf(rl))
        some = np.isfinite(rl)
        bound = od.lse_bound(extra, dim, length, rl) + 1e-6
        assert (np.abs(glse[b][some] - rl[some]) <= bound[some]).all(), f"lse of sequence {b}"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 300, 2 ** 31 - 600])
def test_a_table_with_room_for_more_than_2_to_the_31_tokens(window, e4m3):
    import torch
    page, pages, lens = 1 << 16, 1 << 16, [70000, 5, 0]
    say(f"attn room for 2^32 tokens, window {window}, e4m3={e4m3}")
    c = CacheCase(97, lens, 1, 16, page, e4m3, "cuda", spare=0)
    table = torch.full((len(lens), pages), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    q = torch.randn((len(lens), 2, 2, 16), device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = f32_of(wsl.attn_decode(c.cache, q, table, c.kv_lens, window=window, status=st))
    assert st.item() == 0
    for b, n in enumerate(lens):
        ref, _, extra = od.attn_ref(f32_of(q)[b], c.values[0][b], c.values[1][b], n, 0.25, window)
        assert (np.abs(got[b] - ref) <= od.attn_bound(extra, 16, n, ref, 2.0 ** -24)).all()
