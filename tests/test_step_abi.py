"""kv_pages_*, rotary_embed, sample_logits and lora_add without a GPU: what they refuse, workspace sizes,
frequencies, and the references against each other."""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle.step as ref
import weight_streaming_linear_amd as wsl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, FORMAT, RANGE, FLAGS = 0, 1, 2, 3, 4, 7, 10
A, ODD = 4096, 4097         # addresses, never dereferenced: validation fails first


def pages(**over):
    d = dict(table=A, lens=A, free_pages=A, n_free=A, n_seq=3, pages_per_seq=8, ld_table=8, n_pages=24, page_size=16)
    d.update(over)
    return wsl.WslKvPages(*(d[n] for n, _ in wsl.WslKvPages._fields_))


@pytest.mark.parametrize("over,code", [
    (dict(n_seq=-1), SHAPE), (dict(n_seq=65536), SHAPE), (dict(pages_per_seq=0), SHAPE), (dict(ld_table=7), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=(1 << 30) + 1), SHAPE),
    (dict(ld_table=1 << 62), SHAPE), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(free_pages=None), NULL),
    (dict(n_free=None), NULL), (dict(table=ODD), ALIGN), (dict(lens=4098), ALIGN), (dict(free_pages=ODD), ALIGN),
    (dict(n_free=ODD), ALIGN)])
def test_bad_pages_are_refused(over, code):
    L, p = wsl.lib(), ctypes.byref(pages(**over))
    assert L.kv_pages_grow(p, None, 1, 3, A, A, None, A, 1 << 20, None, None) == code
    assert L.kv_pages_trim(p, A, None, None) == code


def test_pages_refusals():
    L = wsl.lib()

    def grow(p=None, new=None, each=1, n=3, slots=A, positions=A, starts=None, ws=A, nb=1 << 30):
        return L.kv_pages_grow(ctypes.byref(p or pages()), new, each, n, slots, positions, starts, ws, nb, None, None)

    assert L.kv_pages_grow(None, None, 1, 3, A, A, None, A, 1 << 20, None, None) == NULL
    assert L.kv_pages_trim(None, A, None, None) == NULL and L.kv_pages_trim(ctypes.byref(pages()), None, None, None) == NULL
    assert L.kv_pages_trim(ctypes.byref(pages()), ODD, None, None) == ALIGN
    none = pages(n_seq=0, table=None, lens=None, free_pages=None, n_free=None)
    assert grow(none, n=0, slots=None, positions=None) == OK and L.kv_pages_trim(ctypes.byref(none), None, None, None) == OK
    assert grow(each=-1) == SHAPE and grow(each=(1 << 30) + 1) == SHAPE and grow(n=-1) == SHAPE and grow(n=(1 << 30) + 1) == SHAPE
    assert grow(slots=None) == NULL
    assert grow(slots=4100) == ALIGN and grow(positions=4100) == ALIGN and grow(starts=ODD) == ALIGN and grow(new=4098) == ALIGN
    need = wsl.kv_pages_grow_workspace_bytes(3, 1 << 20)
    assert need > 0 and wsl.kv_pages_grow_workspace_bytes(3, 3) == 0 and wsl.kv_pages_grow_workspace_bytes(-1, 1 << 20) == 0
    assert wsl.kv_pages_grow_workspace_bytes(65535, 3) > 0
    assert grow(n=1 << 20, ws=None) == NULL and grow(n=1 << 20, nb=need - 1) == RANGE and grow(n=1 << 20, ws=4104) == ALIGN


def test_rotary_refusals():
    L = wsl.lib()

    def call(q=A, heads=4, ld_q=512, k=A, kv=2, ld_k=256, xfmt=0, count=3, dim=128, rot=128, pos=A, freqs=A, amp=1.0, flags=0,
             qo=A, ld_qo=512, ko=A, ld_ko=256, ofmt=1):
        return L.rotary_embed(q, heads, ld_q, k, kv, ld_k, xfmt, count, dim, rot, pos, freqs, amp, flags, qo, ld_qo, ko, ld_ko,
                              ofmt, None)

    assert call(count=0, q=None, pos=None, freqs=None, qo=None) == OK
    assert call(xfmt=2) == FORMAT and call(ofmt=-1) == FORMAT and call(flags=2) == FLAGS
    assert call(count=-1) == SHAPE and call(heads=0) == SHAPE and call(heads=65537) == SHAPE and call(kv=0) == SHAPE
    assert call(dim=24) == SHAPE and call(dim=272, ld_q=2048) == SHAPE and call(dim=0) == SHAPE
    assert call(rot=0) == SHAPE and call(rot=130) == SHAPE and call(rot=63) == SHAPE
    assert call(amp=float("nan")) == SHAPE and call(amp=float("inf")) == SHAPE
    assert call(count=1 << 40) == SHAPE
    assert call(q=None) == NULL and call(qo=None) == NULL and call(pos=None) == NULL and call(freqs=None) == NULL
    assert call(ko=None) == NULL
    assert call(ld_q=508) == SHAPE and call(ld_qo=504) == SHAPE and call(ld_k=252) == SHAPE and call(ld_ko=248) == SHAPE
    assert call(ld_q=514) == ALIGN and call(ld_qo=516) == ALIGN and call(ld_k=258) == ALIGN and call(ld_ko=260) == ALIGN
    assert call(q=4104) == ALIGN and call(qo=4104) == ALIGN and call(k=4104) == ALIGN and call(ko=4104) == ALIGN
    assert call(pos=4100) == ALIGN and call(freqs=4100) == ALIGN


def test_sampling_refusals():
    L = wsl.lib()

    def call(z=A, fmt=0, n=2, vocab=100, ld=100, how=None, u=A, tok=A, probs=None, ld_p=100, ws=A, nb=1 << 30):
        return L.sample_logits(z, fmt, n, vocab, ld, how, u, tok, probs, ld_p, ws, nb, None, None)

    assert call(n=0, z=None, u=None) == OK
    assert call(fmt=2) == FORMAT
    assert call(n=-1) == SHAPE and call(n=65536) == SHAPE and call(vocab=0) == SHAPE and call(vocab=(1 << 22) + 1, ld=1 << 23) == SHAPE
    assert call(z=None) == NULL and call(u=None) == NULL and call(tok=None) == NULL
    assert call(ld=99) == SHAPE and call(probs=A, ld_p=99) == SHAPE and call(ld=1 << 62) == SHAPE and call(probs=A, ld_p=1 << 62) == SHAPE
    assert call(z=4098) == ALIGN and call(z=ODD, fmt=1) == ALIGN and call(u=ODD) == ALIGN and call(tok=4098) == ALIGN
    assert call(probs=4098) == ALIGN
    for name in ("d_temperature", "d_top_k", "d_top_p", "d_min_p"):
        assert call(how=ctypes.byref(wsl.WslSampling(**{name: 4098}))) == ALIGN
    f = wsl.sample_logits_workspace_bytes
    assert f(3, 8192) == 0 == f(0, 151937) == f(3, 0) == f(3, 1 << 23)
    need = f(3, 151937)
    assert need > 0
    assert call(n=3, vocab=151937, ld=151937, ws=None) == NULL
    assert call(n=3, vocab=151937, ld=151937, nb=need - 1) == RANGE
    assert call(n=3, vocab=151937, ld=151937, ws=4104) == ALIGN


def test_lora_refusals():
    L = wsl.lib()

    def call(a=A, b=A, count=3, rank=16, n_out=100, k=64, ids=A, scales=A, x=A, m=2, ldx=64, base=A, ld_b=100, out=A, ld_o=100,
             fmt=0, ws=A, nb=1 << 30):
        return L.lora_add(a, b, count, rank, n_out, k, ids, scales, x, m, ldx, base, ld_b, out, ld_o, fmt, ws, nb, None, None)

    assert call(m=0, a=None, x=None, out=None) == OK
    assert call(fmt=2) == FORMAT
    for bad in (dict(m=-1), dict(m=(1 << 20) + 1), dict(rank=0), dict(rank=12), dict(rank=136), dict(k=0), dict(k=60), dict(k=1 << 23, ldx=1 << 23),
                dict(n_out=0), dict(n_out=(1 << 22) + 1, ld_b=1 << 23, ld_o=1 << 23), dict(count=0), dict(count=(1 << 20) + 1),
                dict(ldx=56), dict(ld_b=99), dict(ld_o=99), dict(ldx=1 << 62), dict(ld_b=1 << 62), dict(ld_o=1 << 62)):
        assert call(**bad) == SHAPE, bad
    for name in ("a", "b", "ids", "x", "base", "out"):
        assert call(**{name: None}) == NULL
    for bad in (dict(a=4104), dict(b=4104), dict(x=4104), dict(ids=4098), dict(scales=4098), dict(base=4098), dict(out=4098),
                dict(base=ODD, fmt=1), dict(ldx=68)):
        assert call(**bad) == ALIGN, bad
    need = wsl.lora_add_workspace_bytes(2, 16, 64)
    assert need == 2 * 16 * 4
    assert call(ws=None) == NULL and call(nb=need - 1) == RANGE and call(ws=4104) == ALIGN
    f = wsl.lora_add_workspace_bytes
    assert f(0, 16, 64) == 0 == f(2, 12, 64) == f(2, 16, 60) == f(-1, 16, 64)
    assert f(1, 16, 5120) <= f(64, 16, 5120) <= 64 * 16 * 16 * 4


def test_binding_refuses_what_the_abi_would_misread():
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="GPU"):
        wsl.sample_logits(z, torch.zeros(2))
    with pytest.raises(ValueError, match="GPU"):
        wsl.rotary_embed(torch.zeros(2, 1, 16), torch.zeros(2, dtype=torch.int64), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="GPU"):
        wsl.lora_add(z, z.bfloat16(), torch.zeros(1, 8, 8), torch.zeros(1, 8, 8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        i = torch.zeros(2, dtype=torch.int32)
        wsl.KVPages(torch.zeros(2, 3, dtype=torch.int32), i, i, i[:1], 16)
    with pytest.raises(ValueError, match="lie 0 apart"):
        wsl._logit_rows(torch.zeros(8).expand(2, 8), "logits", 2)
    with pytest.raises(ValueError, match="stride 1"):
        wsl._logit_rows(torch.zeros(8, 2).t(), "logits", 2)
    assert wsl._logit_rows(torch.zeros(3, 9)[:, :8], "logits", 3) == 9
    assert wsl._logit_rows(torch.zeros(3, 9)[:1, 1:8], "logits", 1) == 7
    with pytest.raises(ValueError, match="shape"):
        wsl._token_rows(z, "x", 2, 9)


def test_frequencies():
    f = wsl.rotary_freqs(64, device="cpu")
    assert f.dtype is torch.float64 and f.shape == (32,)
    assert torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-14)
    assert torch.equal(wsl.rotary_freqs(64, scaling="linear", factor=4.0, device="cpu") * 4, f)
    slow = wsl.rotary_freqs(64, scaling="base", factor=8.0, device="cpu")
    assert slow[0] == 1 and math.isclose(float(f[-1] / slow[-1]), 8.0, rel_tol=1e-12)
    bands = wsl.rotary_freqs(128, base=500000.0, scaling="bands", factor=8.0, trained=8192, device="cpu")
    g = wsl.rotary_freqs(128, base=500000.0, device="cpu")
    turns = 8192 * g / (2 * math.pi)
    assert torch.equal(bands[turns >= 4], g[turns >= 4]) and torch.equal(bands[turns <= 1], g[turns <= 1] / 8)
    between = (turns > 1) & (turns < 4)
    assert between.any() and (bands[between] < g[between]).all() and (bands[between] > g[between] / 8).all()
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, base=0.0), dict(rot_dim=8, factor=0.0), dict(rot_dim=8, scaling="x"),
                dict(rot_dim=2, scaling="base"), dict(rot_dim=8, scaling="bands", low=4.0, high=4.0),
                dict(rot_dim=8, scaling="bands", trained=0)):
        with pytest.raises(ValueError):
            wsl.rotary_freqs(**bad, device="cpu")


def test_references():
    """By hand: ties, borders, masked entries, pages that run out, a quarter turn."""
    z = np.array([1.0, 3.0, 3.0, -np.inf, 2.0])
    assert ref.sample_ref(z, 0.0, temperature=0.0)[0] == 1
    assert (ref.sample_ref(z, top_k=2)[1] == [0, 0.5, 0.5, 0, 0]).all()
    assert ref.sample_ref(z, 0.5, top_k=2)[0] == 2 and ref.sample_ref(z, 0.499, top_k=2)[0] == 1
    assert (ref.sample_ref(np.zeros(8), top_p=0.5)[1] == [0.25] * 4 + [0] * 4).all()
    assert (ref.sample_ref(z, min_p=1.0)[1] == [0, 0.5, 0.5, 0, 0]).all()
    assert ref.sample_ref(z, 1.0)[0] == 4 and ref.sample_ref(z, float("nan"))[0] == 4
    assert ref.sample_ref(np.array([0.0, np.nan]), 0.5)[0] == -1 and ref.sample_ref(np.array([-np.inf]), 0.5)[0] == -1
    p = ref.Pages([[0, 0], [5, 0]], [0, 3], [1, 2, 9], 2, 4)
    assert p.grow([5, 2], 7) == ([8, 9, 10, 11, 4, -1, -1], [0, 1, 2, 3, 4, -1, -1], [0, 5, 7])
    assert p.status == ref.STATUS_PAGES and p.lens == [5, 3] and p.n_free == 0
    p.trim([0, 3])
    assert p.n_free == 2 and p.free[:2] == [1, 2] and p.lens == [0, 3]
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    out, _ = ref.rotary_ref(x, [1], [math.pi / 2, 0.0])
    assert np.allclose(out, [[[-3, 2, 1, 4, 9]]])
    out, _ = ref.rotary_ref(x, [1], [math.pi / 2, 0.0], interleaved=True, amplitude=2.0)
    assert np.allclose(out, [[[-4, 2, 6, 8, 9]]])
    one = np.ones((1, 2))
    out, bound = ref.lora_ref(one, one * 3, np.ones((1, 1, 2)), np.array([[[2.0], [4.0]]]), [0], [0.5])
    assert (out == [[7.0, 13.0]]).all() and (0 < bound).all() and (bound < 1e-5).all()
    assert (ref.lora_ref(one, one, np.ones((1, 1, 2)), np.ones((1, 2, 1)), [-1])[0] == 1).all()


def test_validation_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "validate_step")
    srcs = [os.path.join(ROOT, "tests", "cpp", "validate_step_main.cpp"),
            os.path.join(ROOT, "weight_streaming_linear_amd", "csrc", "validate.cpp")]
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", *srcs, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("rank", [8, 16, 40, 64, 128])
@pytest.mark.parametrize("k", [8, 1024, 5120, 16384, 1 << 20])
def test_a_workspace_for_many_tokens_serves_fewer(rank, k):
    sizes = [wsl.lora_add_workspace_bytes(m, rank, k) for m in [*range(1, 3000), 4096, 5000, 70000, 1 << 20]]
    assert sizes == sorted(sizes) and sizes[0] >= 4 * rank


@pytest.mark.parametrize("vocab", [8193, 32000, 65536, 131072, 131073, 151937])
def test_a_workspace_for_many_rows_serves_fewer(vocab):
    sizes = [wsl.sample_logits_workspace_bytes(n, vocab) for n in range(1, 300)]
    assert sizes == sorted(sizes)
