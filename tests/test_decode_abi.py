"""kv_cache_*, attn_decode and verify_drafts without a GPU: what they refuse, and workspace sizes."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import weight_streaming_linear_amd as wsl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, FORMAT, RANGE = 0, 1, 2, 3, 4, 7
A, ODD = 4096, 4097         # addresses, never dereferenced: validation fails first


def cache(**over):
    d = dict(k=A, v=A, k_exp=A, v_exp=A, fmt=wsl.WSL_KV_BF16, n_pages=4, n_kv=2, page_size=16, head_dim=64,
             page_stride=2048, head_stride=1024, token_stride=64)
    d.update(over)
    return wsl.WslKvCache(*(d[n] for n, _ in wsl.WslKvCache._fields_))


CACHE_FAULTS = [(dict(fmt=2), FORMAT), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=4104), ALIGN),
                (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE), (dict(n_kv=0), SHAPE), (dict(page_size=0), SHAPE),
                (dict(head_dim=24), SHAPE), (dict(head_dim=272), SHAPE), (dict(head_dim=0), SHAPE),
                (dict(token_stride=48), SHAPE), (dict(token_stride=68), ALIGN), (dict(page_stride=-2048), SHAPE),
                (dict(page_stride=1 << 60), SHAPE), (dict(fmt=wsl.WSL_KV_E4M3, k_exp=None), NULL),
                (dict(fmt=wsl.WSL_KV_E4M3, v_exp=None), NULL), (dict(fmt=wsl.WSL_KV_E4M3, token_stride=72), ALIGN)]


@pytest.mark.parametrize("over,code", CACHE_FAULTS)
def test_bad_caches_are_refused_everywhere(over, code):
    L, c = wsl.lib(), cache(**over)
    r = ctypes.byref(c)
    assert L.kv_cache_write(r, A, A, 0, 3, 128, 128, A, None, None) == code
    assert L.kv_cache_read(r, A, 3, A, A, 0, 128, 128, None, None) == code
    assert L.attn_decode(r, A, 1, 2, 1, 4, 256, A, 8, 8, A, 0.1, 0, A, 1, 256, None, A, 1 << 30, None, None) == code


def test_kv_rows_refusals():
    L = wsl.lib()
    r = ctypes.byref(cache())

    def both(k=A, v=A, fmt=0, count=3, ld_k=128, ld_v=128, slots=A):
        w = L.kv_cache_write(r, k, v, fmt, count, ld_k, ld_v, slots, None, None)
        assert w == L.kv_cache_read(r, slots, count, k, v, fmt, ld_k, ld_v, None, None)
        return w

    assert L.kv_cache_write(None, A, A, 0, 3, 128, 128, A, None, None) == NULL
    assert both(count=0, k=None, slots=None) == OK
    assert both(count=-1) == SHAPE
    assert both(fmt=2) == FORMAT
    assert both(k=None) == NULL and both(v=None) == NULL and both(slots=None) == NULL
    assert both(ld_k=124) == SHAPE and both(ld_v=127) == SHAPE
    assert both(ld_k=130) == ALIGN and both(fmt=1, ld_v=132) == ALIGN
    assert both(k=4104) == ALIGN and both(slots=4100) == ALIGN
    assert both(count=(1 << 26) // 2 + 1) == SHAPE


def test_attn_refusals():
    L = wsl.lib()

    def call(c=None, q=A, qfmt=1, n=2, ql=1, heads=4, ld_q=256, table=A, ld_t=8, pages=8, lens=A, scale=0.1, window=0,
             out=A, ofmt=1, ld_o=256, lse=None, ws=A, nb=1 << 30):
        return L.attn_decode(ctypes.byref(c or cache()), q, qfmt, n, ql, heads, ld_q, table, ld_t, pages, lens, scale,
                             window, out, ofmt, ld_o, lse, ws, nb, None, None)

    assert L.attn_decode(None, A, 1, 2, 1, 4, 256, A, 8, 8, A, 0.1, 0, A, 1, 256, None, A, 1 << 30, None, None) == NULL
    assert call(n=0, q=None, table=None, lens=None, out=None, ws=None, nb=0) == OK
    assert call(n=-1) == SHAPE and call(n=65536) == SHAPE
    assert call(ql=0) == SHAPE and call(ql=257) == SHAPE
    assert call(heads=3) == SHAPE and call(heads=0) == SHAPE
    assert call(heads=2 * 65536, ql=2, ld_q=1 << 24, ld_o=1 << 24) == SHAPE
    assert call(qfmt=2) == FORMAT and call(ofmt=5) == FORMAT
    assert call(q=None) == NULL and call(table=None) == NULL and call(lens=None) == NULL and call(out=None) == NULL
    assert call(pages=0) == SHAPE and call(ld_t=7) == SHAPE and call(window=-1) == SHAPE
    assert call(scale=float("nan")) == SHAPE and call(scale=float("inf")) == SHAPE
    assert call(ld_q=255) == SHAPE and call(ld_q=260) == ALIGN and call(ld_o=248) == SHAPE and call(ld_o=257) == ALIGN
    assert call(q=4104) == ALIGN and call(out=4100) == ALIGN and call(table=4098) == ALIGN and call(lens=ODD) == ALIGN
    assert call(lse=4097) == ALIGN
    # tiles of 128 tokens and four more over all sequences and kv heads: at most 2^30, just below 2 * 1024 * 2^19
    most = cache(page_size=1 << 17, page_stride=1 << 24, head_stride=1 << 23)
    assert call(c=most, n=1023, pages=1 << 9, ld_t=1 << 9, ws=None) == NULL
    assert call(c=most, n=1024, pages=1 << 9, ld_t=1 << 9, ws=None) == SHAPE
    need = wsl.attn_decode_workspace_bytes(1, 2, 1, 4, 2, 64, 64, 16)
    assert need > 0
    assert call(pages=64, ld_t=64, ws=None) == NULL
    assert call(pages=64, ld_t=64, nb=need - 1) == RANGE
    assert call(pages=64, ld_t=64, ws=4104, nb=need) == ALIGN


def test_attn_workspace_sizes():
    f = wsl.attn_decode_workspace_bytes
    assert f(1, 1, 1, 40, 8, 128, 2, 16) == 0              # one tile of tokens: nothing to join
    assert f(1, 0, 1, 40, 8, 128, 64, 16) == 0
    assert f(1, 1, 1, 41, 8, 128, 64, 16) == 0 and f(3, 1, 1, 40, 8, 128, 64, 16) == 0
    assert 0 < f(1, 1, 1, 40, 8, 128, 512, 16) <= f(1, 64, 1, 40, 8, 128, 512, 16) <= 256 << 20


def test_verify_refusals():
    L = wsl.lib()

    def call(p=A, q=A, fmt=0, n=2, width=3, vocab=100, ld_p=100000, ld_q=100000, drafts=A, nd=None, u=A, acc=A, tok=A,
             ws=A, nb=1 << 20):
        return L.verify_drafts(p, q, fmt, n, width, vocab, ld_p, ld_q, drafts, nd, u, acc, tok, ws, nb, None, None)

    assert call(n=0, p=None, u=None) == OK
    assert call(fmt=2) == FORMAT
    assert call(n=-1) == SHAPE and call(n=65536) == SHAPE and call(width=-1) == SHAPE and call(width=65) == SHAPE
    assert call(vocab=0) == SHAPE and call(vocab=(1 << 30) + 1) == SHAPE
    assert call(p=None) == NULL and call(drafts=None) == NULL and call(u=None) == NULL
    assert call(acc=None) == NULL and call(tok=None) == NULL
    assert call(ld_p=99) == SHAPE and call(ld_q=99) == SHAPE and call(vocab=100001) == SHAPE
    assert call(p=4098) == ALIGN and call(q=ODD) == ALIGN and call(drafts=4098) == ALIGN and call(nd=ODD) == ALIGN
    big = 100000
    assert call(vocab=big, ws=None) == NULL and call(vocab=big, ws=4104) == ALIGN
    assert call(vocab=big, nb=wsl.verify_drafts_workspace_bytes(2, big) - 1) == RANGE
    assert wsl.verify_drafts_workspace_bytes(2, 100) == 0       # one launch, nothing to keep between two
    assert wsl.verify_drafts_workspace_bytes(0, 100) == 0 == wsl.verify_drafts_workspace_bytes(3, 0)


def test_binding_refuses_what_the_abi_would_misread():
    """CPU tensors, wrong types, shapes and strides are refused before any pointer is taken."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        wsl.KVCache(k, k)
    with pytest.raises(ValueError):
        wsl.KVCache.empty(4, 2, 16, 64, fmt=9, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        wsl.verify_drafts(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))


def test_validation_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "validate_decode")
    srcs = [os.path.join(ROOT, "tests", "cpp", "validate_decode_main.cpp"),
            os.path.join(ROOT, "weight_streaming_linear_amd", "csrc", "validate.cpp")]
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", *srcs, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
