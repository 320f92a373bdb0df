"""attn_decode on the GPU against the fp64 reference, within the bound that its documented
roundings give (oracle.decode.attn_bound)."""

import numpy as np
import pytest

import oracle.decode as od
import weight_streaming_linear_amd as wsl
from decode_cases import CacheCase, f32_of
from gpu_common import say

pytestmark = pytest.mark.gpu


def _q(seed, n, ql, heads, dim, f32, size=1.5):
    import torch
    g = np.random.default_rng([2026, 10, seed])
    q = torch.from_numpy((size * g.standard_normal((n, ql, heads, dim))).astype(np.float32))
    return (q if f32 else q.to(torch.bfloat16)).cuda()


def _check(c, q, out, lse, scale, window, where=""):
    dim, heads = q.shape[-1], q.shape[2]
    half = 2.0 ** -24 if str(out.dtype) == "torch.float32" else 2.0 ** -8
    q64, got, glse = f32_of(q), f32_of(out), None if lse is None else f32_of(lse)
    for b, n in enumerate(c.lens):
        ref, rl, extra = od.attn_ref(q64[b], c.values[0][b], c.values[1][b], n, scale, window)
        bound = od.attn_bound(extra, dim, n, ref, half)
        err = np.abs(got[b] - ref)
        assert np.isfinite(got[b]).all(), f"{where} sequence {b} ({n} tokens): not finite"
        assert (err <= bound).all(), f"{where} sequence {b} ({n} tokens): {(err / bound).max()} of the bound"
        if glse is not None:
            empty = np.isneginf(rl)
            assert np.array_equal(np.isneginf(glse[b]), empty)
            e = np.abs(np.where(empty, 0, glse[b]) - np.where(empty, 0, rl))
            assert (e <= od.lse_bound(extra, dim, n, rl) + 1e-6).all(), f"{where} lse of sequence {b}"


def _run(seed, lens, heads, n_kv, dim, page, e4m3, ql=1, f32=False, ofmt=None, window=0, order="phtd", scale=None, wide=0, **kw):
    """wide: entries (none of the cache's pages) behind each row of the table, as where lengths may yet
    grow: the split is decided by what a row has room for."""
    import torch
    say(f"attn lens={lens[:6]}.. heads={heads}/{n_kv} dim={dim} page={page} e4m3={e4m3} q_len={ql} f32={f32} "
        f"ofmt={ofmt} window={window} {order}")
    c = CacheCase(seed, lens, n_kv, dim, page, e4m3, "cuda", order=order, **kw)
    c.table = torch.cat((c.table, torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")), 1)
    q = _q(seed, len(lens), ql, heads, dim, f32)
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = wsl.attn_decode(c.cache, q, c.table, c.kv_lens, scale=scale, window=window, ofmt=ofmt, lse=lse, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    _check(c, q, out, lse, dim ** -0.5 if scale is None else scale, window)
    return c, q, out


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("wide", [0, 100])
def test_lengths_around_every_edge(e4m3, f32, page, wide):
    _run(1, EDGES, 10, 2, 128, page, e4m3, f32=f32, wide=wide)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ql", [2, 5, 8])
@pytest.mark.parametrize("wide", [0, 100])
def test_drafts_see_what_is_before_them(e4m3, ql, wide):
    """Lengths below q_len leave the first queries with nothing to see."""
    _run(2, EDGES, 6, 2, 64, 16, e4m3, ql=ql, wide=wide)


@pytest.mark.parametrize("heads,n_kv,dim,page,e4m3,ql,f32,order", [
    (1, 1, 16, 1, False, 1, False, "phtd"), (1, 1, 16, 7, True, 1, True, "pthd"),
    (8, 8, 32, 48, False, 1, True, "pthd"), (40, 8, 128, 20, True, 4, False, "phtd"),
    (48, 8, 128, 64, False, 3, False, "pthd"), (12, 1, 128, 16, True, 1, True, "phtd"),
    (16, 1, 128, 32, False, 4, False, "phtd"), (24, 1, 128, 16, False, 5, False, "phtd"),
    (4, 2, 80, 16, False, 1, False, "phtd"), (4, 2, 96, 24, True, 2, True, "pthd"),
    (6, 3, 192, 16, True, 1, False, "phtd"), (10, 2, 256, 40, False, 1, True, "phtd"),
    (64, 2, 256, 16, True, 2, False, "phtd"), (33, 3, 64, 5, False, 9, True, "phtd"),
    (128, 1, 64, 16, False, 3, False, "phtd"), (5, 1, 48, 16, True, 7, False, "pthd"),
    (2, 2, 144, 16, False, 17, True, "phtd"), (20, 4, 112, 128, True, 40, False, "phtd"),
    (24, 2, 192, 16, False, 2, False, "phtd"), (18, 1, 160, 7, False, 3, False, "pthd"), (17, 1, 192, 16, True, 2, False, "phtd"),
    (9, 1, 208, 16, False, 2, False, "phtd"), (3, 1, 240, 24, True, 6, True, "phtd"), (20, 1, 176, 16, True, 1, False, "pthd")])
@pytest.mark.parametrize("ofmt", [wsl.WSL_OUT_F32, wsl.WSL_OUT_BF16])
@pytest.mark.parametrize("room", [0, 70000])
def test_head_layouts(heads, n_kv, dim, page, e4m3, ql, f32, order, ofmt, room):
    """room: tokens that may yet come; with many, a workgroup takes two blocks of 16 rows."""
    _run(3, [130, 1, 517, 40], heads, n_kv, dim, page, e4m3, ql=ql, f32=f32, order=order, ofmt=ofmt, wide=room // page)


@pytest.mark.parametrize("e4m3,page", [(False, 16), (True, 24)])
@pytest.mark.parametrize("window", [1, 2, 31, 100, 128, 1000])
@pytest.mark.parametrize("wide", [0, 100])
def test_windows(e4m3, page, window, wide):
    _run(4, [0, 1, 99, 100, 101, 260, 500], 4, 2, 64, page, e4m3, ql=3, window=window, wide=wide)
    _run(4, [0, 1, 99, 100, 101, 260, 700], 4, 2, 64, page, e4m3, ql=3, window=window, wide=wide)


@pytest.mark.parametrize("n", [1, 63, 64, 65, 200, 4100])
def test_many_sequences_and_empty_ones(n):
    """The sequence of a share of the work is found by dividing the sequences among 64 lanes."""
    g = np.random.default_rng(n)
    lens = [int(x) if i % 5 else 0 for i, x in enumerate(g.integers(0, 40, n))]
    lens[n // 2] = 700
    _run(70, lens, 2, 1, 16, 16, False, wide=100)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,heads,n_kv", [(1, 8, 1), (1, 40, 8), (3, 4, 2), (300, 2, 1), (70, 16, 8)])
def test_long_and_many(e4m3, n, heads, n_kv):
    """From one sequence spread over the chip to more sequences than workgroups."""
    g = np.random.default_rng(n)
    longest = 6000 if n <= 3 else 400
    lens = [longest] + [int(x) for x in np.exp(g.uniform(0, np.log(longest), n - 1))]
    _run(5 + n, lens, heads, n_kv, 128, 16, e4m3)


def test_65535_sequences():
    """As many sequences as a call takes, on shared pages: three divisions among 64 lanes."""
    import torch
    n, pages, page = 65535, 40, 16
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn((pages, 1, page, 16), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randint(0, pages, (n, 36), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(0, 33, (n,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn((n, 1, 1, 16), generator=g, device="cuda").to(torch.bfloat16)
    cache = wsl.KVCache(k, v)
    for wide in (2, 36):        # 32 tokens of room: whole items; 576: shares
        out = wsl.attn_decode(cache, q, table[:, :wide].contiguous(), lens)
        kk, vv = (t[table[:, :2].long(), 0].flatten(1, 2).double() for t in (k, v))
        s = (kk @ q[:, 0, 0, :, None].double())[..., 0] * 0.25
        seen = torch.arange(32, device="cuda") < lens[:, None]
        s = s.masked_fill(~seen, -torch.inf)
        w = torch.softmax(s, -1).nan_to_num(0)
        ref = (w[:, None] @ vv)[:, 0]
        extra = {"pv": (w[:, None] @ vv.abs())[:, 0].cpu().numpy(),
                 "score": (kk.abs() @ q[:, 0, 0, :, None].double().abs())[..., 0].amax(-1).mul(0.25).cpu().numpy()}
        ref = ref.cpu().numpy()
        bound = od.attn_bound(extra, 16, 32, ref, 2.0 ** -8)
        assert (np.abs(f32_of(out)[:, 0, 0] - ref) <= bound).all()


def test_scales_and_large_scores():
    """Negative and zero scales, and scores far apart (one token takes all)."""
    for scale in (-0.3, 0.0, 1e-30, 4.0):
        _run(6, [200, 3], 4, 2, 64, 16, False, f32=True, scale=scale)


def test_masked_places_may_hold_anything():
    """Every unused slot holds NaN already; here also the drafts' own values are NaN or infinite:
    only the queries that see them take them."""
    import torch

    def fill(b, x):
        x[95 + b, 0, 3] = [np.nan, np.inf, -np.inf][b]

    for e4m3 in (False, True):
        if e4m3:
            def fill(b, x):     # noqa: F811  (an e4m3 row with a NaN is NaN as a whole)
                x[95 + b, 0, 3] = np.nan
        lens = [100, 101, 102]
        c = CacheCase(7, lens, 1, 64, 16, e4m3, "cuda", v_fill=fill)
        q = _q(7, 3, 8, 3, 64, False)
        got = f32_of(wsl.attn_decode(c.cache, q, c.table, c.kv_lens))
        for b, n in enumerate(lens):
            ref, _, extra = od.attn_ref(f32_of(q)[b], c.values[0][b], c.values[1][b], n, 0.125)
            fine = np.isfinite(ref)
            assert fine[:3].all() and not fine[3:, :, 3].any()
            assert np.array_equal(np.isnan(got[b]), np.isnan(ref)) and np.array_equal(np.isinf(got[b]), np.isinf(ref))
            assert np.array_equal(got[b][np.isinf(ref)], ref[np.isinf(ref)])
            bound = od.attn_bound({k: np.where(np.isfinite(x), x, 0) for k, x in extra.items()}, 64, n, ref, 2.0 ** -8)
            assert (np.abs(got[b] - ref)[fine] <= bound[fine]).all()

    # an infinite key makes the softmax of the queries that see it NaN, and no other
    def kfill(b, x):
        x[97, 0] = np.inf

    c = CacheCase(8, [100], 1, 64, 24, False, "cuda", k_fill=kfill)
    q = _q(8, 1, 6, 2, 64, False)
    got = f32_of(wsl.attn_decode(c.cache, q, c.table, c.kv_lens))[0]
    assert np.isfinite(got[:3]).all() and np.isnan(got[3:]).any()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dim,heads,n_kv,ql,window,f32,e4m3,page", [
    (128, 5, 1, 5, 0, False, False, 16), (128, 5, 1, 5, 0, True, False, 24), (128, 40, 2, 3, 100, False, True, 16),
    (256, 4, 1, 4, 0, False, False, 16), (256, 4, 1, 4, 60, True, True, 7), (192, 6, 2, 2, 0, False, True, 16),
    (80, 12, 1, 5, 33, False, False, 16), (64, 16, 1, 4, 0, False, False, 48), (48, 2, 2, 6, 0, True, False, 1)])
@pytest.mark.parametrize("room", [0, 70000])
def test_odd_values_reach_only_what_sees_them(dim, heads, n_kv, ql, window, f32, e4m3, page, room):
    """NaNs among the values: in the newest positions (seen by the last queries alone) and before the
    window's reach of the last ones; sequences of one and of many parts.  What sees none is as exact as
    ever; what sees one is NaN in that element and exact in the others."""
    import torch
    say(f"attn odd dim={dim} heads={heads}/{n_kv} q_len={ql} window={window} f32={f32} e4m3={e4m3} page={page}")
    lens = [130, 3000, 9]

    def fill(b, x):
        n = lens[b]
        x[n - 1, :, dim - 1] = np.nan
        if ql > 2:
            x[n - 2, 0, 1] = np.nan
        if window:
            x[max(0, n - ql - window + 1), :, 7] = np.nan      # seen by the first query alone

    c = CacheCase(40 + ql, lens, n_kv, dim, page, e4m3, "cuda", v_fill=fill)
    c.table = torch.cat((c.table, torch.full((3, room // page), -1, dtype=torch.int32, device="cuda")), 1)
    q = _q(40, 3, ql, heads, dim, f32)
    got = f32_of(wsl.attn_decode(c.cache, q, c.table, c.kv_lens, window=window))
    for b, n in enumerate(lens):
        ref, _, extra = od.attn_ref(f32_of(q)[b], c.values[0][b], c.values[1][b], n, dim ** -0.5, window)
        assert np.array_equal(np.isnan(got[b]), np.isnan(ref))
        fine = ~np.isnan(ref)
        assert not fine.all()
        extra = {k: np.where(np.isnan(x), 0, x) for k, x in extra.items()}
        bound = od.attn_bound(extra, dim, n, ref, 2.0 ** -24 if f32 else 2.0 ** -8)
        assert (np.abs(got[b] - ref)[fine] <= bound[fine]).all()


def test_rows_whose_pages_are_all_bad_are_zero():
    import torch
    for n, lens_heads in ((60, 4), (3000, 24)):
        c = CacheCase(60, [n, n], 2, 64, 16, False, "cuda")
        q = _q(60, 2, 2, lens_heads, 64, False)
        table = c.table.clone()
        table[0] = -1
        st, lse = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(q.shape[:3], device="cuda")
        out = wsl.attn_decode(c.cache, q, table, c.kv_lens, lse=lse, status=st)
        assert st.item() == wsl.WSL_STATUS_INDEX
        assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
        ref, _, extra = od.attn_ref(f32_of(q)[1], c.values[0][1], c.values[1][1], n, 0.125)
        assert (np.abs(f32_of(out)[1] - ref) <= od.attn_bound(extra, 64, n, ref, 2.0 ** -8)).all()


def test_bad_pages_and_lengths_are_reported():
    import torch
    for page in (16, 10):
        c = CacheCase(9, [200, 200], 2, 64, page, False, "cuda")
        q = _q(9, 2, 1, 4, 64, True)
        per = c.table.shape[1]
        bad_at = 3
        for bad in (-1, int(c.cache.n_pages), 2 ** 31 - 1, -2 ** 31):
            table = c.table.clone()
            table[1, bad_at] = bad
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = f32_of(wsl.attn_decode(c.cache, q, table, c.kv_lens, status=st))
            assert st.item() == wsl.WSL_STATUS_INDEX
            keep = np.ones(200, bool)
            keep[bad_at * page:(bad_at + 1) * page] = False
            for b in range(2):
                k, v = (c.values[i][b][keep if b else slice(None)] for i in range(2))
                ref, _, extra = od.attn_ref(f32_of(q)[b], k, v, len(k), 0.125)
                assert (np.abs(out[b] - ref) <= od.attn_bound(extra, 64, 200, ref, 2.0 ** -24)).all()
        # lengths outside the table are clamped
        table = c.table[:, :5].contiguous()
        for lens, used in (([-7, 200], [0, 5 * page]), ([2 ** 31 - 1, 3], [5 * page, 3])):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = f32_of(wsl.attn_decode(c.cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), status=st))
            assert st.item() == wsl.WSL_STATUS_INDEX
            for b in range(2):
                ref, _, extra = od.attn_ref(f32_of(q)[b], c.values[0][b], c.values[1][b], used[b], 0.125)
                assert (np.abs(out[b] - ref) <= od.attn_bound(extra, 64, 200, ref, 2.0 ** -24)).all()
        assert per == c.table.shape[1]


def test_offsets_past_32_bits():
    """Pages at the far end of a cache of more than 2^32 elements."""
    heads, dim, page = 8, 128, 16
    n_pages = (1 << 32) // (heads * dim * page) + 100
    c = CacheCase(10, [300, 70], heads, dim, page, False, "cuda", total_pages=n_pages)
    q = _q(10, 2, 1, 16, dim, False)
    out = wsl.attn_decode(c.cache, q, c.table, c.kv_lens)
    _check(c, q, out, None, dim ** -0.5, 0)


def test_strided_queries_outputs_and_tables():
    import torch
    c = CacheCase(11, [70, 300, 9], 2, 64, 16, True, "cuda")
    fused = torch.zeros(3, 2, 4 + 2 + 2, 64, device="cuda")
    fused[:, :, :4] = _q(11, 3, 2, 4, 64, True)
    wide = torch.full((3, c.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    out = torch.full((3, 2, 6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    wsl.attn_decode(c.cache, fused[:, :, :4], wide[:, :c.table.shape[1]], c.kv_lens, out=out[:, :, 1:5])
    _check(c, fused[:, :, :4], out[:, :, 1:5], None, 0.125, 0)
    assert (out[:, :, 0] == 5).all() and (out[:, :, 5] == 5).all()


def test_same_bits_every_time_and_streams():
    import torch
    c = CacheCase(12, [5000, 37, 800], 2, 128, 16, False, "cuda")
    q = _q(12, 3, 1, 8, 128, False)
    first = wsl.attn_decode(c.cache, q, c.table, c.kv_lens)
    ws = torch.full((wsl.attn_decode_workspace_bytes(1, 3, 1, 8, 2, 128, c.table.shape[1], 16) // 4,), float("nan"),
                    device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        out = wsl.attn_decode(c.cache, q, c.table, c.kv_lens, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("heads,n_kv,dim,ql", [(1, 1, 64, 1), (6, 1, 128, 1), (5, 1, 128, 3), (7, 1, 128, 1), (40, 1, 64, 2),
                                               (24, 2, 128, 5), (3, 1, 256, 3), (12, 1, 192, 2), (1, 1, 16, 1)])
def test_parts_are_joined(heads, n_kv, dim, ql):
    """Few and many rows (one and several row tiles, fewer and more elements than threads), two and
    many parts, fewer and more items than workgroups; on a workspace of NaNs."""
    import torch
    for lens in ([3000], [4099, 700, 129], [300, 1, 0, 5000] + [257] * 90, [140] * 600):
        say(f"attn join heads={heads}/{n_kv} dim={dim} q_len={ql} {len(lens)} sequences")
        c = CacheCase(20 + ql, lens, n_kv, dim, 16, False, "cuda")
        q = _q(20, len(lens), ql, heads, dim, False)
        n = wsl.attn_decode_workspace_bytes(1, len(lens), ql, heads, n_kv, dim, c.table.shape[1], 16)
        ws = torch.full((n // 4,), float("nan"), device="cuda")
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        for _ in range(2):
            out = wsl.attn_decode(c.cache, q, c.table, c.kv_lens, lse=lse, workspace=ws)
        _check(c, q, out, lse, dim ** -0.5, 0)


def test_a_captured_step_follows_growing_lengths():
    """Write, attend and advance, captured once; lengths grow on the device."""
    import torch
    n, n_kv, heads, dim, page, start = 3, 2, 4, 64, 16, 120
    c = CacheCase(13, [start + 40] * n, n_kv, dim, page, False, "cuda")
    lens = torch.tensor([start, start - 100, 1], dtype=torch.int32, device="cuda")
    begin = lens.clone()
    new = [torch.zeros(n, n_kv, dim, device="cuda") for _ in range(2)]
    q = torch.zeros(n, 1, heads, dim, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(max(16, wsl.attn_decode_workspace_bytes(0, n, 1, heads, n_kv, dim, c.table.shape[1], page)),
                     dtype=torch.uint8, device="cuda")

    def step():
        at = lens.long()
        slots = c.table.gather(1, (at // page)[:, None])[:, 0].long() * page + at % page
        wsl.kv_cache_write(c.cache, *new, slots)
        lens.add_(1)
        wsl.attn_decode(c.cache, q, c.table, lens, out=out, workspace=ws)

    step()
    lens.copy_(begin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = np.random.default_rng(13)
    for i in range(5):
        for w in range(2):
            x = torch.from_numpy(g.standard_normal((n, n_kv, dim)).astype(np.float32)).to(torch.bfloat16).float()
            new[w].copy_(x)
            for b in range(n):
                c.values[w][b][int(begin[b]) + i] = x[b].numpy()
        q.copy_(_q(50 + i, n, 1, heads, dim, True))
        graph.replay()
        torch.cuda.synchronize()
        c.lens = [int(x) for x in lens]
        assert c.lens == [int(x) + i + 1 for x in begin]
        _check(c, q, out, None, dim ** -0.5, 0, f"replay {i}")


def test_refusals():
    import torch
    c = CacheCase(14, [20, 30], 2, 64, 16, False, "cuda")
    q = _q(14, 2, 1, 4, 64, False)
    ok = dict(q=q, block_table=c.table, kv_lens=c.kv_lens)
    wsl.attn_decode(c.cache, **ok)
    lse = torch.zeros(2, 1, 4, device="cuda")
    for bad in (dict(q=q[0]), dict(q=q.half()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q.repeat(1, 1, 1, 2)[..., ::2]),
                dict(block_table=c.table.long()), dict(block_table=c.table[:1]), dict(block_table=c.table.t()),
                dict(kv_lens=c.kv_lens.long()), dict(kv_lens=c.kv_lens[:1]), dict(out=torch.zeros(2, 1, 4, 32, device="cuda")),
                dict(out=torch.zeros_like(q).half()), dict(out=q, ofmt=wsl.WSL_OUT_F32), dict(ofmt=7),
                dict(lse=lse.double()), dict(lse=lse[:1]), dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            wsl.attn_decode(c.cache, **{**ok, **bad})
    for bad, code in ((dict(q=q[:, :, :3].contiguous()), 2), (dict(window=-1), 2), (dict(scale=float("nan")), 2)):
        with pytest.raises(wsl.WSLError) as e:
            wsl.attn_decode(c.cache, **{**ok, **bad})
        assert e.value.code == code
    assert wsl.attn_decode(c.cache, q[:0], c.table[:0], c.kv_lens[:0]).shape == (0, 1, 4, 64)
