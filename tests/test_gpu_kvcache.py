"""kv_cache_write / kv_cache_read on the GPU against the fp64 reference, bit for bit: both are exact
given their one documented rounding."""

import numpy as np
import pytest

import oracle.decode as od
import weight_streaming_linear_amd as wsl
from decode_cases import f32_of
from gpu_common import say

pytestmark = pytest.mark.gpu

BF16, E4M3 = wsl.WSL_KV_BF16, wsl.WSL_KV_E4M3


def _rows(seed, count, heads, dim, f32):
    """Rows of very different sizes, some of them zero."""
    import torch
    g = np.random.default_rng([2026, 8, seed])
    x = g.standard_normal((count, heads, dim)) * np.exp2(g.integers(-60, 60, (count, heads, 1)))
    x[g.random((count, heads)) < 0.05] = 0
    t = torch.from_numpy(x.astype(np.float32))
    return t if f32 else t.to(torch.bfloat16)


def _empty(fmt, n_pages, heads, page, dim, order="phtd"):
    """A cache of marker bytes."""
    import torch
    shape = (n_pages, heads, page, dim) if order == "phtd" else (n_pages, page, heads, dim)
    dt = torch.uint8 if fmt == E4M3 else torch.int16
    raw = [torch.full(shape, 0x55, dtype=dt, device="cuda") for _ in range(2)]
    exps = [torch.full((n_pages, heads, page), 0x55, dtype=torch.uint8, device="cuda") if fmt == E4M3 else None
            for _ in range(2)]
    if order == "pthd":
        raw = [t.transpose(1, 2) for t in raw]
    views = [t.view(torch.float8_e4m3fn if fmt == E4M3 else torch.bfloat16) for t in raw]
    return wsl.KVCache(*views, *exps), raw, exps


def _want(x, fmt):
    """(stored integers, scale bytes, values) of rows x."""
    import torch
    if fmt == E4M3:
        codes, exps = od.kv_encode(f32_of(x))
        return codes, exps, od.kv_decode(codes, exps)
    b = x.float().to(torch.bfloat16)
    return b.view(torch.int16).numpy(), None, f32_of(b)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("count,heads,dim,page,order", [
    (1, 8, 128, 16, "phtd"), (1, 1, 16, 1, "phtd"), (77, 8, 128, 24, "pthd"), (300, 3, 80, 7, "phtd"),
    (65, 2, 256, 64, "pthd"), (33, 5, 48, 16, "phtd"), (1000, 4, 64, 48, "phtd"), (5, 1, 192, 3, "pthd"),
    (9, 2, 144, 128, "phtd"), (40, 1, 32, 5, "pthd")])
def test_write_then_read(fmt, f32, count, heads, dim, page, order):
    import torch
    say(f"kv write fmt={fmt} f32={f32} {count}x{heads}x{dim} page={page} {order}")
    g = np.random.default_rng([2026, 9, count])
    n_pages = (count + page - 1) // page + 4
    cache, raw, exps = _empty(fmt, n_pages, heads, page, dim, order)
    k, v = _rows(count, count, heads, dim, f32), _rows(count + 1, count, heads, dim, f32)
    slots = torch.from_numpy(g.permutation(n_pages * page)[:count].astype(np.int64))
    wsl.kv_cache_write(cache, k.cuda(), v.cuda(), slots.cuda())
    ks, vs = [wsl.kv_cache_read(cache, slots.cuda(), ofmt=o) for o in (wsl.WSL_OUT_F32, wsl.WSL_OUT_BF16)]
    torch.cuda.synchronize()
    at = (slots // page).numpy(), slice(None), (slots % page).numpy()
    untouched = np.ones((n_pages, page), bool)
    untouched[at[0], at[2]] = False
    for i, x in enumerate((k, v)):
        ints, ex, values = _want(x, fmt)
        got = raw[i].cpu().numpy()
        assert np.array_equal(got[at], ints)
        assert (got.transpose(0, 2, 1, 3)[untouched] == 0x55).all()
        if fmt == E4M3:
            gex = exps[i].cpu().numpy()
            assert np.array_equal(gex[at], ex)
            assert (gex.transpose(0, 2, 1)[untouched] == 0x55).all()
        assert np.array_equal(f32_of(ks[i]), values) and np.array_equal(f32_of(vs[i]), values)
        assert ks[i].dtype == torch.float32 and vs[i].dtype == torch.bfloat16


def test_views_of_a_fused_projection():
    """k and v inside rows of [q | k | v], read back into views of wider rows."""
    import torch
    heads, dim, count = 2, 64, 37
    cache, _, _ = _empty(E4M3, 8, heads, 16, dim)
    fused = _rows(5, count, 8 + 2 * heads, dim, False).cuda()
    slots = torch.randperm(128, device="cuda")[:count]
    wsl.kv_cache_write(cache, fused[:, 8:8 + heads], fused[:, 8 + heads:], slots)
    out = torch.full((count, 3 * heads, dim), 7.0, device="cuda")
    wsl.kv_cache_read(cache, slots, out[:, :heads], out[:, 2 * heads:], ofmt=wsl.WSL_OUT_F32)
    for i, at in ((8, 0), (8 + heads, 2 * heads)):
        want = _want(fused[:, i:i + heads].cpu(), E4M3)[2]
        assert np.array_equal(f32_of(out[:, at:at + heads]), want)
    assert (out[:, heads:2 * heads] == 7).all()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_slots_outside_and_skipped(fmt):
    import torch
    heads, dim, page = 2, 32, 5
    cache, raw, _ = _empty(fmt, 3, heads, page, dim)
    x = _rows(6, 6, heads, dim, True).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wsl.kv_cache_write(cache, x[:2], x[:2], torch.tensor([-1, 4], device="cuda"), status=st)
    assert st.item() == 0
    for bad in (15, -2, 1 << 40, -(1 << 62)):
        st.zero_()
        slots = torch.tensor([0, bad, 14], device="cuda")
        wsl.kv_cache_write(cache, x[:3], x[3:], slots, status=st)
        assert st.item() == wsl.WSL_STATUS_INDEX
        st.zero_()
        k, v = wsl.kv_cache_read(cache, slots, ofmt=wsl.WSL_OUT_F32, status=st)
        assert st.item() == wsl.WSL_STATUS_INDEX
        assert (k[1] == 0).all() and (v[1] == 0).all()
        assert np.array_equal(f32_of(k[[0, 2]]), _want(x[[0, 2]].cpu(), fmt)[2])
    got = raw[0].cpu().numpy().transpose(0, 2, 1, 3).reshape(15, -1)
    assert (got[[1, 2, 3, 5, 6, 7, 8, 9, 10, 11, 12, 13]] == 0x55).all()
    st.zero_()
    k, _ = wsl.kv_cache_read(cache, torch.tensor([-1, 4, 4], device="cuda"), status=st)
    assert st.item() == 0 and (k[0] == 0).all() and torch.equal(k[1], k[2])
    wsl.kv_cache_write(cache, x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device="cuda"))


def test_rows_that_are_not_finite_or_tiny():
    import torch
    dim = 48
    x = torch.zeros(8, 1, dim)
    x[0, 0, 3] = float("nan")
    x[1, 0, 47] = float("inf")
    x[2, 0, 0] = -float("inf")
    x[3] = 3e38
    x[4] = torch.full((dim,), 1e-45)
    x[5, 0, 7] = 2.0 ** -120
    x[6, 0, 1], x[6, 0, 2] = 448.0, 2.0 ** -10        # the second: halfway to the least code, ties to zero
    x[7] = -0.0
    cache, raw, exps = _empty(E4M3, 1, 1, 8, dim)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.arange(8, device="cuda")
    wsl.kv_cache_write(cache, x.cuda(), x.cuda(), slots, status=st)
    assert st.item() == wsl.WSL_STATUS_NONFINITE
    codes, ex, values = _want(x, E4M3)
    assert np.array_equal(raw[1].cpu().numpy()[0, 0], codes[:, 0]) and np.array_equal(exps[1].cpu().numpy()[0, 0], ex[:, 0])
    k, _ = wsl.kv_cache_read(cache, slots)
    assert np.array_equal(f32_of(k), values, equal_nan=True)
    assert np.isnan(f32_of(k)[:3]).all()
    st.zero_()
    bf = _empty(BF16, 1, 1, 8, dim)[0]
    wsl.kv_cache_write(bf, x.cuda(), x.cuda(), slots, status=st)
    assert st.item() == 0
    assert np.array_equal(f32_of(wsl.kv_cache_read(bf, slots)[1]), f32_of(x.to(torch.bfloat16)), equal_nan=True)


def test_every_code_reads_back():
    """All 256 codes under every scale byte that a write can store, in both output types; what is past
    the largest finite number of the output's type (from 2^128 on, in both) is an infinity there."""
    import torch
    ex = torch.arange(17, 248, dtype=torch.uint8)
    codes = torch.arange(256, dtype=torch.uint8).repeat(len(ex), 1)[:, None, None].contiguous()
    exps = ex[:, None, None].contiguous()
    c = codes.cuda().view(torch.float8_e4m3fn)
    cache = wsl.KVCache(c, c.clone(), exps.cuda(), exps.cuda())
    slots = torch.arange(len(ex), device="cuda")
    with np.errstate(over="ignore"):
        want = od.kv_decode(codes.numpy(), exps.numpy())[:, 0, 0].astype(np.float32)
    assert np.isinf(want).sum() == 2 * 7 and np.isinf(want[-1]).sum() == 2 * 7      # 256 .. 448 times 2^120
    for o in (wsl.WSL_OUT_F32, wsl.WSL_OUT_BF16):
        k, v = wsl.kv_cache_read(cache, slots, ofmt=o)
        assert np.array_equal(f32_of(k)[:, 0], want, equal_nan=True) and np.array_equal(f32_of(v)[:, 0], want, equal_nan=True)


def test_offsets_past_32_bits():
    """A bf16 cache of more than 2^32 elements each for k and v; slots at its far end."""
    import torch
    heads, dim, page = 8, 128, 16
    n_pages = (1 << 32) // (heads * dim * page) + 100
    cache = wsl.KVCache.empty(n_pages, heads, page, dim)
    slots = torch.tensor([n_pages * page - 1 - 997 * i for i in range(50)] + [3, 0], device="cuda")
    k, v = _rows(11, 52, heads, dim, False).cuda(), _rows(12, 52, heads, dim, False).cuda()
    wsl.kv_cache_write(cache, k, v, slots)
    rk, rv = wsl.kv_cache_read(cache, slots)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    assert torch.equal(cache.tensors[0].flatten()[-dim:], k[0, -1])


def test_another_stream_and_a_graph():
    import torch
    heads, dim, page, count = 4, 64, 16, 96
    cache, _, _ = _empty(E4M3, 10, heads, page, dim)
    x = _rows(13, count, heads, dim, True).cuda()
    slots = torch.randperm(160, device="cuda")[:count]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    wsl.kv_cache_write(cache, x, x, slots, stream=s)
    k, v = wsl.kv_cache_read(cache, slots, ofmt=wsl.WSL_OUT_F32, stream=s)
    s.synchronize()
    want = _want(x.cpu(), E4M3)[2]
    assert np.array_equal(f32_of(k), want) and np.array_equal(f32_of(v), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wsl.kv_cache_write(cache, x, x, slots)
        wsl.kv_cache_read(cache, slots, k, v, ofmt=wsl.WSL_OUT_F32)
    for i in range(4):
        x.copy_(_rows(20 + i, count, heads, dim, True))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f32_of(v), _want(x.cpu(), E4M3)[2])


def test_refusals():
    import torch
    cache, _, _ = _empty(BF16, 4, 2, 16, 64)
    x = torch.zeros(3, 2, 64, device="cuda")
    slots = torch.arange(3, device="cuda")
    ok = (cache, x, x, slots)
    wsl.kv_cache_write(*ok)
    for i, bad in ((1, x.half()), (1, x.cpu()), (1, x[:2]), (1, x[:, :1]), (2, x.bfloat16()), (3, slots.int()),
                   (3, slots[:2]), (3, slots.cpu()), (1, x.transpose(0, 1).contiguous().transpose(0, 1)),
                   (1, torch.zeros(3, 2, 128, device="cuda")[..., ::2])):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            wsl.kv_cache_write(*args)
    with pytest.raises(ValueError):
        wsl.kv_cache_read(cache, slots, k=x.bfloat16(), ofmt=wsl.WSL_OUT_F32)
    with pytest.raises(wsl.WSLError) as e:     # rows that start off 16 bytes
        wsl.kv_cache_write(cache, torch.zeros(3 * 129 + 8, device="cuda")[1:1 + 3 * 128].view(3, 2, 64), x, slots)
    assert e.value.code == 3
    d = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    f = d.to(torch.float8_e4m3fn)
    b = torch.zeros(4, 2, 16, dtype=torch.uint8, device="cuda")
    for args in ((d, d.float()), (d, d[:3]), (d[0], d[0]), (f, f), (f, f, b, b[:3]), (d, d, b, b), (f, f, b, b.int()),
                 (d, d.transpose(1, 2).contiguous().transpose(1, 2)), (d.transpose(2, 3), d.transpose(2, 3))):
        with pytest.raises(ValueError):
            wsl.KVCache(*args)
