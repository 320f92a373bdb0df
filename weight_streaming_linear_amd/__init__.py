"""Weight-streaming linear layers for AMD Instinct MI355X (gfx950).

A thin ctypes binding over the C ABI of ``libwsl.so`` (declared in
``include/wsl.h``).  Every step of the computation runs in the library's HIP
kernels; this module only marshals arguments: it takes torch tensors (device
memory) and the current torch stream, passes raw pointers and sizes, and turns
status codes into exceptions.  There is no fallback: if the library is not
built, every call raises.

Entry points (same names as the C ABI):
  nf4_packed_bytes, nf4_codebook, nf4_pack, nf4_dequant_tile,
  linear_gemv, linear_gemm, linear_gemm_workspace_bytes, nf4_embed_rows, wsl_strerror;
  linear_gemm_noalloc; linear_gemv_multi; GemvSweep (linear_gemv_sweep,
  linear_gemv_sweep_workspace_bytes);
  KVCache (wsl_kv_cache) with kv_cache_write, kv_cache_read, attn_decode and
  attn_decode_workspace_bytes; verify_drafts and verify_drafts_workspace_bytes;
  stream_read (wsl_stream_read); CopyRing.gemv / CopyRing.gemm (linear_gemv_streamed /
  linear_gemm_streamed, weights streamed from page-locked host memory, see to_pinned).
"""

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwsl.so")

WSL_OK = 0
WSL_W_BF16 = 0
WSL_W_NF4 = 1
WSL_OUT_F32 = 0
WSL_OUT_BF16 = 1
WSL_KV_BF16 = 0
WSL_KV_E4M3 = 1
WSL_STATUS_NONFINITE = 1
WSL_STATUS_OVERFLOW = 2
WSL_STATUS_INDEX = 4

EXPORTED = [
    "nf4_packed_bytes", "nf4_codebook", "nf4_pack", "nf4_dequant_tile", "linear_gemv",
    "linear_gemm_workspace_bytes", "linear_gemm", "nf4_embed_rows", "linear_gemv_streamed",
    "linear_gemm_streamed", "wsl_stream_read", "wsl_strerror", "linear_gemm_noalloc",
    "linear_gemv_sweep_workspace_bytes", "linear_gemv_sweep", "linear_gemv_multi",
    "kv_cache_write", "kv_cache_read", "attn_decode_workspace_bytes", "attn_decode",
    "verify_drafts_workspace_bytes", "verify_drafts",
]
WSL_STATUS_SWEEP_TIMEOUT = 8
WSL_STATUS_DESCRIPTOR = 16
SWEEP_STATUS_OFFSET = 1280      # byte offset of the status word in the sweep workspace
WSL_E_SCRATCH = 9
WSL_E_FLAGS = 10
WSL_RING_PACE = 1               # linear_*_streamed: the host keeps the copies two matrices ahead
NOALLOC_SCRATCH_BYTES = 4 << 20


class WSLError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: status {code} ({wsl_strerror(code)})")


_lib = None


def lib():
    """The loaded libwsl.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libwsl.so is not built ({LIB_PATH}); run __graft_entry__.build() "
                           "or python -m weight_streaming_linear_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    L.nf4_packed_bytes.argtypes = [i64, i64]
    L.nf4_packed_bytes.restype = sz
    L.nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.nf4_codebook.restype = ctypes.c_int
    L.nf4_pack.argtypes = [vp, i64, i64, vp, vp, vp]
    L.nf4_pack.restype = ctypes.c_int
    L.nf4_dequant_tile.argtypes = [vp, i64, i64, i64, i64, i64, i64, vp, i64, vp]
    L.nf4_dequant_tile.restype = ctypes.c_int
    L.linear_gemv.argtypes = [ctypes.c_int, vp, i64, i64, vp, vp, vp]
    L.linear_gemv.restype = ctypes.c_int
    L.linear_gemm_workspace_bytes.argtypes = [ctypes.c_int, i64, i64, i64]
    L.linear_gemm_workspace_bytes.restype = sz
    L.linear_gemm.argtypes = [ctypes.c_int, vp, i64, i64, vp, i64, i64, vp, ctypes.c_int, i64, vp, sz, vp]
    L.linear_gemm.restype = ctypes.c_int
    L.linear_gemv_sweep_workspace_bytes.argtypes = []
    L.linear_gemv_sweep_workspace_bytes.restype = sz
    L.linear_gemv_sweep.argtypes = [ctypes.c_int, i64, vp, vp, vp, sz, vp]
    L.linear_gemv_sweep.restype = ctypes.c_int
    L.linear_gemv_multi.argtypes = [ctypes.c_int, i64, vp, vp]
    L.linear_gemv_multi.restype = ctypes.c_int
    L.linear_gemm_noalloc.argtypes = [ctypes.c_int, vp, i64, i64, vp, i64, i64, vp, ctypes.c_int, i64, vp]
    L.linear_gemm_noalloc.restype = ctypes.c_int
    L.nf4_embed_rows.argtypes = [vp, i64, i64, vp, i64, vp, ctypes.c_int, i64, vp, vp]
    L.nf4_embed_rows.restype = ctypes.c_int
    L.linear_gemv_streamed.argtypes = [ctypes.c_int, i64, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, ctypes.c_int]
    L.linear_gemv_streamed.restype = ctypes.c_int
    L.linear_gemm_streamed.argtypes = [ctypes.c_int, i64, vp, vp, vp, vp, i64, i64, vp, ctypes.c_int, i64, vp, sz, vp,
                                       sz, vp, vp, vp, ctypes.c_int]
    L.linear_gemm_streamed.restype = ctypes.c_int
    ci = ctypes.c_int
    L.kv_cache_write.argtypes = [vp, vp, vp, ci, i64, i64, i64, vp, vp, vp]
    L.kv_cache_write.restype = ci
    L.kv_cache_read.argtypes = [vp, vp, i64, vp, vp, ci, i64, i64, vp, vp]
    L.kv_cache_read.restype = ci
    L.attn_decode_workspace_bytes.argtypes = [ci] + [i64] * 7
    L.attn_decode_workspace_bytes.restype = sz
    L.attn_decode.argtypes = [vp, vp, ci, i64, i64, i64, i64, vp, i64, i64, vp, ctypes.c_float, i64, vp, ci, i64, vp,
                              vp, sz, vp, vp]
    L.attn_decode.restype = ci
    L.verify_drafts_workspace_bytes.argtypes = [i64, i64]
    L.verify_drafts_workspace_bytes.restype = sz
    L.verify_drafts.argtypes = [vp, vp, ci, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.verify_drafts.restype = ci
    L.wsl_stream_read.argtypes = [vp, sz, vp, vp]
    L.wsl_stream_read.restype = ctypes.c_int
    L.wsl_strerror.argtypes = [ctypes.c_int]
    L.wsl_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def wsl_strerror(code):
    return lib().wsl_strerror(int(code)).decode()


def _check(rc, where):
    if rc != WSL_OK:
        raise WSLError(rc, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(t, name, dtypes, device=None, contiguous=False, ndim=None):
    """Raise ValueError unless t is a device tensor of one of ``dtypes`` whose last
    dimension is unit-stride (whole tensor contiguous if ``contiguous``), on ``device``.
    The C ABI reads raw row-major memory, so a transposed or sliced view, or a tensor of
    another element type, must be refused here rather than misread."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a GPU tensor, got one on {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {[str(d) for d in dtypes]}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.dim() > 0 and t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: last dimension must have stride 1 (got strides {t.stride()})")


def _weight(w, wfmt, n_out, k, name="w"):
    """Check a weight tensor against its format and shape: bf16 [n_out][k] contiguous, or a
    contiguous uint8 buffer of at least nf4_packed_bytes(n_out, k) bytes."""
    import torch
    if wfmt == WSL_W_NF4:
        _require(w, name, (torch.uint8,), contiguous=True)
        need = nf4_packed_bytes(n_out, k)
        if need and w.numel() < need:
            raise ValueError(f"{name}: {w.numel()} bytes, a packed {n_out}x{k} matrix needs {need}")
    elif wfmt == WSL_W_BF16:
        _require(w, name, (torch.bfloat16,), contiguous=True)
        if w.numel() < n_out * k:
            raise ValueError(f"{name}: {w.numel()} elements, a {n_out}x{k} bf16 matrix needs {n_out * k}")
    else:
        raise ValueError(f"{name}: unknown weight format {wfmt}")


def _stream(stream):
    """The handle of a stream, or of the current one.  That one is asked for as a number: making a
    Stream object of it takes 2.7 us of the host, as long as a launch."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(_device())


def _raw_stream(device):
    """torch's own function of this kind, which takes this one's place at the first call (as does _device's):
    the module itself loads without torch."""
    global _raw_stream, _device
    from torch import _C
    _raw_stream, _device = _C._cuda_getCurrentRawStream, _C._cuda_getDevice
    return _raw_stream(device)


def _device():
    from torch import _C
    return _C._cuda_getDevice()


# ---------------------------------------------------------------- format helpers
def nf4_packed_bytes(n_out, k):
    return int(lib().nf4_packed_bytes(int(n_out), int(k)))


def nf4_codebook():
    """The 16 binary32 levels the kernels use (a Python list of floats)."""
    buf = (ctypes.c_float * 16)()
    _check(lib().nf4_codebook(buf), "nf4_codebook")
    return [float(v) for v in buf]


# ---------------------------------------------------------------- entry points
def nf4_pack(w, packed=None, status=None, stream=None):
    """Encode a bf16 [n_out][k] device tensor into a packed NF4 uint8 device tensor."""
    import torch
    _require(w, "w", (torch.bfloat16,), contiguous=True, ndim=2)
    n_out, k = w.shape
    nbytes = nf4_packed_bytes(n_out, k)
    if packed is not None:
        _require(packed, "packed", (torch.uint8,), device=w.device, contiguous=True)
        if packed.numel() < nbytes:
            raise ValueError(f"packed: {packed.numel()} bytes, {n_out}x{k} needs {nbytes}")
    if status is not None:
        _require(status, "status", (torch.int32, torch.uint32), device=w.device)
    if packed is None:
        packed = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w.device)
    rc = lib().nf4_pack(_ptr(w), n_out, k, _ptr(packed), _ptr(status), _stream(stream))
    _check(rc, "nf4_pack")
    return packed


def nf4_dequant_tile(packed, n_out, k, row0, k0, rows, cols, tile=None, ld_tile=None, stream=None):
    """Restore the bf16 tile [rows][cols] at (row0, k0) of a packed NF4 matrix."""
    import torch
    _weight(packed, WSL_W_NF4, n_out, k, "packed")
    if tile is None:
        tile = torch.empty((rows, cols), dtype=torch.bfloat16, device=packed.device)
        ld_tile = cols
    _require(tile, "tile", (torch.bfloat16,), device=packed.device)
    if ld_tile is None:
        ld_tile = tile.stride(0)
    rc = lib().nf4_dequant_tile(_ptr(packed), n_out, k, row0, k0, rows, cols, _ptr(tile), ld_tile, _stream(stream))
    _check(rc, "nf4_dequant_tile")
    return tile


def nf4_embed_rows(packed, n_rows, k, ids, out=None, ofmt=WSL_OUT_BF16, status=None, stream=None):
    """Restore rows ids (int64 device tensor) of a packed NF4 [n_rows][k] matrix into out [count][>= k]."""
    import torch
    _weight(packed, WSL_W_NF4, n_rows, k, "packed")
    _require(ids, "ids", (torch.int64,), device=packed.device, contiguous=True)
    count = int(ids.numel())
    dt = torch.bfloat16 if ofmt == WSL_OUT_BF16 else torch.float32
    if out is None:
        out = torch.empty((count, k), dtype=dt, device=packed.device)
    _require(out, "out", (dt,), device=packed.device, ndim=2)
    if status is not None:
        _require(status, "status", (torch.int32, torch.uint32), device=packed.device)
    rc = lib().nf4_embed_rows(_ptr(packed), n_rows, k, _ptr(ids), count, _ptr(out), int(ofmt), out.stride(0),
                              _ptr(status), _stream(stream))
    _check(rc, "nf4_embed_rows")
    return out


def linear_gemv(w, x, y=None, wfmt=None, n_out=None, k=None, stream=None):
    """y = W x (fp32).  w: bf16 [n_out][k] or packed NF4 uint8 (give n_out and k)."""
    import torch
    if wfmt is None:
        wfmt = WSL_W_NF4 if w.dtype == torch.uint8 else WSL_W_BF16
    if n_out is None or k is None:
        n_out, k = w.shape
    _weight(w, wfmt, n_out, k)
    _require(x, "x", (torch.bfloat16,), device=w.device, contiguous=True)
    if x.numel() < k:
        raise ValueError(f"x: {x.numel()} elements, k = {k}")
    if y is None:
        y = torch.empty(n_out, dtype=torch.float32, device=x.device)
    _require(y, "y", (torch.float32,), device=w.device, contiguous=True)
    if y.numel() < n_out:
        raise ValueError(f"y: {y.numel()} elements, n_out = {n_out}")
    rc = lib().linear_gemv(int(wfmt), _ptr(w), n_out, k, _ptr(x), _ptr(y), _stream(stream))
    _check(rc, "linear_gemv")
    return y


def linear_gemm_workspace_bytes(wfmt, n_out, k, m):
    return int(lib().linear_gemm_workspace_bytes(int(wfmt), int(n_out), int(k), int(m)))


def linear_gemm(w, x, y=None, wfmt=None, n_out=None, k=None, ofmt=WSL_OUT_F32, workspace=None, stream=None):
    """Y = X W^T.  x: bf16 [m][k] (row stride = x.stride(0)); y fp32 or bf16 [m][n_out]."""
    import torch
    if wfmt is None:
        wfmt = WSL_W_NF4 if w.dtype == torch.uint8 else WSL_W_BF16
    if n_out is None or k is None:
        n_out, k = w.shape
    _weight(w, wfmt, n_out, k)
    _require(x, "x", (torch.bfloat16,), device=w.device, ndim=2)
    if x.shape[1] < k:
        raise ValueError(f"x: shape {tuple(x.shape)}, k = {k}")
    m = x.shape[0]
    dt = torch.float32 if ofmt == WSL_OUT_F32 else torch.bfloat16
    if y is None:
        y = torch.empty((m, n_out), dtype=dt, device=x.device)
    _require(y, "y", (dt,), device=w.device, ndim=2)
    if y.shape[0] < m or y.shape[1] < n_out:
        raise ValueError(f"y: shape {tuple(y.shape)}, need at least ({m}, {n_out})")
    if workspace is not None:
        _require(workspace, "workspace", (workspace.dtype,), device=w.device, contiguous=True)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().linear_gemm(int(wfmt), _ptr(w), n_out, k, _ptr(x), m, x.stride(0), _ptr(y), int(ofmt), y.stride(0),
                           _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "linear_gemm")
    return y


def linear_gemm_noalloc(w, x, y, wfmt=None, n_out=None, k=None, ofmt=WSL_OUT_F32, stream=None):
    """linear_gemm without a workspace argument and without allocating: the split partials use
    the library's per-device scratch (linear_gemm_noalloc).  y must be given (nothing is
    allocated here either)."""
    import torch
    if wfmt is None:
        wfmt = WSL_W_NF4 if w.dtype == torch.uint8 else WSL_W_BF16
    if n_out is None or k is None:
        n_out, k = w.shape
    _weight(w, wfmt, n_out, k)
    _require(x, "x", (torch.bfloat16,), device=w.device, ndim=2)
    if x.shape[1] < k:
        raise ValueError(f"x: shape {tuple(x.shape)}, k = {k}")
    m = x.shape[0]
    dt = torch.float32 if ofmt == WSL_OUT_F32 else torch.bfloat16
    _require(y, "y", (dt,), device=w.device, ndim=2)
    if y.shape[0] < m or y.shape[1] < n_out:
        raise ValueError(f"y: shape {tuple(y.shape)}, need at least ({m}, {n_out})")
    rc = lib().linear_gemm_noalloc(int(wfmt), _ptr(w), n_out, k, _ptr(x), m, x.stride(0), _ptr(y), int(ofmt),
                                   y.stride(0), _stream(stream))
    _check(rc, "linear_gemm_noalloc")
    return y


class WslGemvStage(ctypes.Structure):
    """struct wsl_gemv_stage of the C ABI."""
    _fields_ = [("w", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n_out", ctypes.c_int64), ("k", ctypes.c_int64)]


class GemvSweep:
    """A decode sweep for linear_gemv_sweep: NF4 GEMVs run in order in one launch.

    stages: [(packed NF4 uint8 tensor, x bf16 [k], y fp32 [n_out], n_out, k)].  The host and
    device descriptor arrays and the zeroed synchronization workspace are built once here;
    each call enqueues the one launch on the current (or given) stream."""

    def __init__(self, stages):
        import torch
        if not stages:
            raise ValueError("a sweep needs at least one stage")
        dev = stages[0][0].device
        self.h = (WslGemvStage * len(stages))()
        for i, (w, x, y, n_out, k) in enumerate(stages):
            _weight(w, WSL_W_NF4, n_out, k, f"w[{i}]")
            _require(x, f"x[{i}]", (torch.bfloat16,), device=dev, contiguous=True)
            _require(y, f"y[{i}]", (torch.float32,), device=dev, contiguous=True)
            if x.numel() < k or y.numel() < n_out:
                raise ValueError(f"stage {i}: x has {x.numel()} of {k}, y {y.numel()} of {n_out} elements")
            self.h[i] = WslGemvStage(w.data_ptr(), x.data_ptr(), y.data_ptr(), int(n_out), int(k))
        self.count = len(stages)
        self.tensors = [t for st in stages for t in st[:3]]      # keep the buffers alive
        raw = bytes(self.h)
        self.d = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(dev)
        self.ws_bytes = int(lib().linear_gemv_sweep_workspace_bytes())
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)

    def __call__(self, stream=None):
        rc = lib().linear_gemv_sweep(WSL_W_NF4, self.count, ctypes.byref(self.h), _ptr(self.d), _ptr(self.ws),
                                     self.ws_bytes, _stream(stream))
        _check(rc, "linear_gemv_sweep")

    def status(self):
        """The workspace's status word (reads the device: for tests and diagnostics)."""
        return int(self.ws[SWEEP_STATUS_OFFSET:SWEEP_STATUS_OFFSET + 4].view(__import__("torch").int32).item())


GEMV_MULTI_MAX = 8


def linear_gemv_multi(mats, stream=None):
    """Independent bf16 GEMVs of one k in one launch (linear_gemv_multi): mats is a list of
    (w bf16 [n_out][k], x bf16 [k], y fp32 [n_out] or None); returns the ys."""
    import torch
    if not mats:
        return []
    if len(mats) > GEMV_MULTI_MAX:
        raise ValueError(f"{len(mats)} matrices, at most {GEMV_MULTI_MAX}")
    dev = mats[0][0].device
    h = (WslGemvStage * len(mats))()
    ys = []
    for i, (w, x, y) in enumerate(mats):
        n_out, k = w.shape
        _weight(w, WSL_W_BF16, n_out, k, f"w[{i}]")
        _require(x, f"x[{i}]", (torch.bfloat16,), device=dev, contiguous=True)
        if x.numel() < k:
            raise ValueError(f"x[{i}]: {x.numel()} elements, k = {k}")
        if y is None:
            y = torch.empty(n_out, dtype=torch.float32, device=dev)
        _require(y, f"y[{i}]", (torch.float32,), device=dev, contiguous=True)
        if y.numel() < n_out:
            raise ValueError(f"y[{i}]: {y.numel()} elements, n_out = {n_out}")
        h[i] = WslGemvStage(w.data_ptr(), x.data_ptr(), y.data_ptr(), int(n_out), int(k))
        ys.append(y)
    rc = lib().linear_gemv_multi(WSL_W_BF16, len(mats), ctypes.byref(h), _stream(stream))
    _check(rc, "linear_gemv_multi")
    return ys


# ---------------------------------------------------------------- key-value cache, attention, drafts
class WslKvCache(ctypes.Structure):
    """struct wsl_kv_cache of the C ABI."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("fmt", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("n_kv", ctypes.c_int64), ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class KVCache:
    """The handle of one layer's paged key-value cache (wsl_kv_cache), over tensors that the caller owns.

    k, v: [n_pages][n_kv][page_size][head_dim] of bfloat16, or of float8_e4m3fn with k_exp and
    v_exp, uint8 [n_pages][n_kv][page_size] (see include/wsl.h for the 8-bit form).  k and v may
    be views with other orders of pages, heads and tokens (a transposed [page][token][head] pool,
    the halves of one tensor), both with the same strides and head_dim contiguous.  The handle
    keeps the tensors alive."""

    def __init__(self, k, v, k_exp=None, v_exp=None):
        import torch
        e4m3 = k.dtype == torch.float8_e4m3fn
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        _require(k, "k", (dtype,), ndim=4)
        _require(v, "v", (dtype,), device=k.device, ndim=4)
        if v.shape != k.shape or v.stride() != k.stride():
            raise ValueError(f"k and v differ: {tuple(k.shape)} {k.stride()}, {tuple(v.shape)} {v.stride()}")
        if e4m3:
            if k_exp is None or v_exp is None:
                raise ValueError("an e4m3 cache needs k_exp and v_exp")
            for t, name in ((k_exp, "k_exp"), (v_exp, "v_exp")):
                _require(t, name, (torch.uint8,), device=k.device, contiguous=True)
                if t.shape != k.shape[:3]:
                    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(k.shape[:3])}")
        elif k_exp is not None or v_exp is not None:
            raise ValueError("a bf16 cache has no scale bytes")
        n_pages, n_kv, page_size, dim = k.shape
        # a dimension of one entry is never stepped over: any stride serves
        strides = [s if n > 1 else -(-dim // 16) * 16 for s, n in zip(k.stride()[:3], k.shape[:3])]
        self.tensors = (k, v, k_exp, v_exp)
        self.device = k.device
        self.fmt = WSL_KV_E4M3 if e4m3 else WSL_KV_BF16
        self.n_pages, self.n_kv, self.page_size, self.head_dim = n_pages, n_kv, page_size, dim
        self.desc = WslKvCache(k.data_ptr(), v.data_ptr(), k_exp.data_ptr() if e4m3 else None,
                               v_exp.data_ptr() if e4m3 else None, self.fmt, n_pages, n_kv, page_size, dim, *strides)
        self.ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, n_pages, n_kv, page_size, head_dim, fmt=WSL_KV_BF16, device="cuda"):
        """A cache over new tensors (uninitialised: a slot is read only once it has been written)."""
        import torch
        shape = (int(n_pages), int(n_kv), int(page_size), int(head_dim))
        if fmt not in (WSL_KV_BF16, WSL_KV_E4M3):
            raise ValueError(f"unknown cache format {fmt}")
        dtype = torch.float8_e4m3fn if fmt == WSL_KV_E4M3 else torch.bfloat16
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if fmt == WSL_KV_BF16:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)))


def _float_format(t, name):
    """WSL_OUT_F32 or WSL_OUT_BF16 of a tensor."""
    import torch
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return WSL_OUT_BF16
    if dtype is torch.float32:
        return WSL_OUT_F32
    raise ValueError(f"{name}: dtype {dtype} is neither float32 nor bfloat16")


def _float_dtype(fmt):
    import torch
    if fmt not in (WSL_OUT_F32, WSL_OUT_BF16):
        raise ValueError(f"unknown element format {fmt}")
    return torch.float32 if fmt == WSL_OUT_F32 else torch.bfloat16


def _new(shape, dtype, device, stream):
    """A new tensor whose memory belongs to the stream that the call runs on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _status(status, device):
    import torch
    if status is not None:
        _require(status, "status", (torch.int32, torch.uint32), device=device)
        if status.numel() < 1:
            raise ValueError("status: empty")


def _head_rows(t, name, device, shape):
    """Check a [..., heads, head_dim] tensor whose leading dimensions step as one (a view of a wider
    row of tokens serves); returns the elements from token to token."""
    if t.device == device and t.shape == shape and t.is_contiguous():      # the common case, in 0.3 us
        return shape[-2] * shape[-1]
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    st = t.stride()
    heads, dim = shape[-2:]
    if (dim > 1 and st[-1] != 1) or (heads > 1 and st[-2] != dim):
        raise ValueError(f"{name}: heads and their elements must be contiguous (strides {st})")
    if len(shape) == 4:
        if shape[1] == 1:
            return st[0] if shape[0] > 1 else heads * dim
        if shape[0] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError(f"{name}: the first two dimensions must step as one (strides {st})")
        return st[1]
    return st[0] if shape[0] > 1 else heads * dim


def _plain(t, name, dtype, device, shape):
    """Check a contiguous tensor of one type and shape."""
    if t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return
    _require(t, name, (dtype,), device=device, contiguous=True)
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _slots(cache, slots):
    import torch
    if slots.dim() != 1:
        raise ValueError(f"slots: expected 1 dimension, got shape {tuple(slots.shape)}")
    _plain(slots, "slots", torch.int64, cache.device, slots.shape)
    return slots.numel()


def kv_cache_write(cache, k, v, slots, status=None, stream=None):
    """Put k, v [count][n_kv][head_dim] (fp32 or bf16; views of a fused projection serve) into the
    slots (int64 [count]: page * page_size + place, -1 for none) of a KVCache."""
    dev = cache.device
    count = _slots(cache, slots)
    shape = (count, cache.n_kv, cache.head_dim)
    xfmt = _float_format(k, "k")
    if v.dtype is not k.dtype:
        raise ValueError(f"v: dtype {v.dtype}, k has {k.dtype}")
    ld_k, ld_v = _head_rows(k, "k", dev, shape), _head_rows(v, "v", dev, shape)
    if status is not None:
        _status(status, dev)
    rc = lib().kv_cache_write(cache.ref, k.data_ptr(), v.data_ptr(), xfmt, count, ld_k, ld_v, slots.data_ptr(),
                              _ptr(status), _stream(stream))
    if rc:
        _check(rc, "kv_cache_write")


def kv_cache_read(cache, slots, k=None, v=None, ofmt=WSL_OUT_BF16, status=None, stream=None):
    """The keys and values held in slots, [count][n_kv][head_dim] each of ofmt's type (new ones are
    the halves of one tensor)."""
    dev = cache.device
    count = _slots(cache, slots)
    shape, dtype = (count, cache.n_kv, cache.head_dim), _float_dtype(ofmt)
    ld_k = ld_v = shape[1] * shape[2]
    if k is None and v is None:
        k, v = _new((2, *shape), dtype, dev, stream).unbind(0)
    else:
        if k is None:
            k = _new(shape, dtype, dev, stream)
        if v is None:
            v = _new(shape, dtype, dev, stream)
        if k.dtype is not dtype or v.dtype is not dtype:
            raise ValueError(f"k, v: dtypes {k.dtype}, {v.dtype}, expected {dtype}")
        ld_k, ld_v = _head_rows(k, "k", dev, shape), _head_rows(v, "v", dev, shape)
    if status is not None:
        _status(status, dev)
    rc = lib().kv_cache_read(cache.ref, slots.data_ptr(), count, k.data_ptr(), v.data_ptr(), ofmt, ld_k, ld_v,
                             _ptr(status), _stream(stream))
    if rc:
        _check(rc, "kv_cache_read")
    return k, v


@functools.lru_cache(maxsize=256)
def attn_decode_workspace_bytes(qfmt, n_seq, q_len, n_heads, n_kv, head_dim, pages_per_seq, page_size):
    return int(lib().attn_decode_workspace_bytes(int(qfmt), int(n_seq), int(q_len), int(n_heads), int(n_kv),
                                                 int(head_dim), int(pages_per_seq), int(page_size)))


def attn_decode(cache, q, block_table, kv_lens, scale=None, window=0, out=None, ofmt=None, lse=None, workspace=None,
                status=None, stream=None):
    """Attention of each sequence's q_len newest tokens over its cached tokens (their own included).

    q: [n_seq][q_len][n_heads][head_dim], fp32 or bf16; block_table: int32 [n_seq][pages];
    kv_lens: int32 [n_seq]; scale: 1 / sqrt(head_dim) unless given; window: the last positions a
    query sees, 0 for all; ofmt: q's type unless given; lse: fp32 [n_seq][q_len][n_heads] to be
    written; workspace: a device tensor of attn_decode_workspace_bytes (allocated unless given)."""
    import torch
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q: expected 4 dimensions, got shape {tuple(shape)}")
    n_seq, q_len, n_heads, dim = shape
    dev = cache.device
    qfmt = _float_format(q, "q")
    ld_q = _head_rows(q, "q", dev, (n_seq, q_len, n_heads, cache.head_dim))
    if block_table.dtype is not torch.int32 or block_table.device != dev or block_table.dim() != 2 or \
            not (block_table.is_contiguous() or block_table.stride(1) == 1) or block_table.shape[0] != n_seq:
        _require(block_table, "block_table", (torch.int32,), device=dev, ndim=2)
        raise ValueError(f"block_table: shape {tuple(block_table.shape)}, {n_seq} sequences")
    pages = block_table.shape[1]
    _plain(kv_lens, "kv_lens", torch.int32, dev, (n_seq,))
    ofmt = (qfmt if out is None else _float_format(out, "out")) if ofmt is None else int(ofmt)
    if out is None:
        if ofmt == qfmt and stream is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            out = _new(shape, _float_dtype(ofmt), dev, stream)
        ld_out = n_heads * dim
    else:
        if out.dtype is not _float_dtype(ofmt):
            raise ValueError(f"out: dtype {out.dtype}, expected {_float_dtype(ofmt)}")
        ld_out = _head_rows(out, "out", dev, tuple(shape))
    if lse is not None:
        _require(lse, "lse", (torch.float32,), device=dev, contiguous=True)
        if lse.shape != shape[:3]:
            raise ValueError(f"lse: shape {tuple(lse.shape)}, expected {tuple(shape[:3])}")
    if status is not None:
        _status(status, dev)
    if workspace is None:
        ws_bytes = attn_decode_workspace_bytes(qfmt, n_seq, q_len, n_heads, cache.n_kv, dim, pages, cache.page_size)
        if ws_bytes:
            workspace = _new(ws_bytes, torch.uint8, dev, stream)
    else:
        _require(workspace, "workspace", (workspace.dtype,), device=dev, contiguous=True)
        ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().attn_decode(cache.ref, q.data_ptr(), qfmt, n_seq, q_len, n_heads, ld_q, block_table.data_ptr(),
                           block_table.stride(0) if n_seq > 1 else pages, pages, kv_lens.data_ptr(),
                           dim ** -0.5 if scale is None else float(scale), min(int(window), 2 ** 63 - 1), out.data_ptr(), ofmt, ld_out,
                           _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream))
    if rc:
        _check(rc, "attn_decode")
    return out


@functools.lru_cache(maxsize=256)
def verify_drafts_workspace_bytes(n_seq, vocab):
    return int(lib().verify_drafts_workspace_bytes(int(n_seq), int(vocab)))


def _prob_rows(t, name, device, shape):
    """Check probability rows [n_seq][rows][vocab]; returns the elements from row to row."""
    if t.device == device and t.shape == shape and t.is_contiguous():
        return shape[2]
    if t.device != device or t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} on {t.device}, expected {shape} on {device}")
    st = t.stride()
    if shape[2] > 1 and st[2] != 1:
        raise ValueError(f"{name}: last dimension must have stride 1 (got strides {st})")
    ld = st[1] if shape[1] > 1 else (st[0] if shape[0] > 1 else shape[2])
    if shape[0] > 1 and st[0] != shape[1] * ld:
        raise ValueError(f"{name}: the first two dimensions must step as one (strides {st})")
    if ld < shape[2]:
        raise ValueError(f"{name}: rows of {shape[2]} entries lie {ld} apart (a broadcast tensor needs .contiguous())")
    return ld


def verify_drafts(p, q, drafts, u, n_drafts=None, accepted=None, tokens=None, workspace=None, status=None,
                  stream=None):
    """Which drafts stand, and the token after them, from given random numbers.

    p: [n_seq][width + 1][vocab] target probabilities, q: [n_seq][width][vocab] the drafter's, or
    None where each draft was certain (fp32 or bf16, the same; every row in memory of its own, none
    broadcast); drafts: int32 [n_seq][width]; u: fp32 [n_seq][width + 1] in [0, 1); n_drafts: int32
    [n_seq], width unless given.  Returns (accepted int32 [n_seq], tokens int32 [n_seq][width + 1]: the drafts that stand, the next
    token, -1s)."""
    import torch
    if p.dim() != 3 or not p.is_cuda:
        raise ValueError(f"p: expected a GPU tensor of 3 dimensions, got shape {tuple(p.shape)} on {p.device}")
    dev = p.device
    n_seq, rows, vocab = p.shape
    width = rows - 1
    if width < 0:
        raise ValueError("p: no rows")
    pfmt = _float_format(p, "p")
    ld_p, ld_q = _prob_rows(p, "p", dev, (n_seq, rows, vocab)), 0
    has_q = q is not None and width > 0
    if has_q:
        if q.dtype is not p.dtype:
            raise ValueError(f"q: dtype {q.dtype}, p has {p.dtype}")
        ld_q = _prob_rows(q, "q", dev, (n_seq, width, vocab))
    if drafts is None or u is None:
        raise ValueError("drafts, u: missing")
    _plain(drafts, "drafts", torch.int32, dev, (n_seq, width))
    _plain(u, "u", torch.float32, dev, (n_seq, rows))
    if n_drafts is not None:
        _plain(n_drafts, "n_drafts", torch.int32, dev, (n_seq,))
    if status is not None:
        _status(status, dev)
    if accepted is None:
        accepted = drafts.new_empty((n_seq,)) if stream is None else _new((n_seq,), torch.int32, dev, stream)
    else:
        _plain(accepted, "accepted", torch.int32, dev, (n_seq,))
    if tokens is None:
        tokens = drafts.new_empty((n_seq, rows)) if stream is None else _new((n_seq, rows), torch.int32, dev, stream)
    else:
        _plain(tokens, "tokens", torch.int32, dev, (n_seq, rows))
    if workspace is None:
        ws_bytes = verify_drafts_workspace_bytes(n_seq, vocab)
        if ws_bytes:
            workspace = _new(ws_bytes, torch.uint8, dev, stream)
    else:
        _require(workspace, "workspace", (workspace.dtype,), device=dev, contiguous=True)
        ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().verify_drafts(p.data_ptr(), q.data_ptr() if has_q else None, pfmt, n_seq, width, vocab, ld_p, ld_q,
                             drafts.data_ptr(), _ptr(n_drafts), u.data_ptr(), accepted.data_ptr(), tokens.data_ptr(),
                             _ptr(workspace), ws_bytes, _ptr(status), _stream(stream))
    if rc:
        _check(rc, "verify_drafts")
    return accepted, tokens


def stream_read(buf, sink, stream=None):
    """Read every byte of the device tensor ``buf`` once (wsl_stream_read): the
    streaming-read ceiling probe.  ``sink`` is a device int32/uint32 tensor of one
    element, written only if a lane's words XOR to 0x9e3779b9."""
    nbytes = buf.numel() * buf.element_size()
    _check(lib().wsl_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)), "wsl_stream_read")


# ---------------------------------------------------------------- copy ring
def to_pinned(t):
    """A page-locked host copy (uint8) of a device or host tensor's bytes."""
    import torch
    src = t.contiguous().view(torch.uint8).reshape(-1)
    h = torch.empty(src.numel(), dtype=torch.uint8, pin_memory=True)
    h.copy_(src)
    return h


def _ptr_array(items):
    arr = (ctypes.c_void_p * max(1, len(items)))()
    for i, t in enumerate(items):
        arr[i] = t if isinstance(t, int) else t.data_ptr()
    return arr


def _i64_array(vals):
    arr = (ctypes.c_int64 * max(1, len(vals)))()
    for i, v in enumerate(vals):
        arr[i] = int(v)
    return arr


class CopyRing:
    """Two device slots, a copy stream and four events for linear_*_streamed.

    Matrices stay in page-locked host memory (see to_pinned); each call copies them one
    by one into the slots on the ring's copy stream while the kernels run on the compute
    stream (torch's current stream unless given).  pace=True (WSL_RING_PACE) keeps the
    host at most two matrices ahead of the kernels, so a call returns shortly before its
    last kernels finish; pace=False enqueues everything without waiting (capturable)."""

    def __init__(self, slot_bytes, device="cuda"):
        import torch
        self.slot_bytes = int(slot_bytes)
        self.slots = [torch.empty(max(self.slot_bytes, 16), dtype=torch.uint8, device=device) for _ in range(2)]
        self.copy_stream = torch.cuda.Stream(device=device)
        self.events = [torch.cuda.Event() for _ in range(4)]
        for e in self.events:
            e.record()          # creates the events; a recorded, completed event is a no-op to wait on

    def _common(self, mats, xs, ys, x_dtype, y_dtypes):
        import torch
        if not (len(mats) == len(xs) == len(ys)):
            raise ValueError(f"{len(mats)} matrices, {len(xs)} inputs, {len(ys)} outputs")
        dev = self.slots[0].device
        for i, ((h, _, _), x, y) in enumerate(zip(mats, xs, ys)):
            if h.is_cuda or not h.is_contiguous():
                raise ValueError(f"matrix {i}: expected a contiguous host tensor (see to_pinned)")
            _require(x, f"x[{i}]", (x_dtype,), device=dev)
            _require(y, f"y[{i}]", y_dtypes, device=dev)
        hs = _ptr_array([h for h, _, _ in mats])
        ns = _i64_array([n for _, n, _ in mats])
        ks = _i64_array([k for _, _, k in mats])
        slots = _ptr_array(self.slots)
        evs = _ptr_array([e.cuda_event for e in self.events])
        return hs, ns, ks, slots, evs

    def gemv(self, mats, xs, ys, wfmt=WSL_W_NF4, stream=None, pace=True):
        """mats: [(pinned host tensor, n_out, k)]; xs: bf16 [k] device tensors; ys: fp32 [n_out]."""
        import torch
        hs, ns, ks, slots, evs = self._common(mats, xs, ys, torch.bfloat16, (torch.float32,))
        rc = lib().linear_gemv_streamed(int(wfmt), len(mats), hs, ns, ks, _ptr_array(xs), _ptr_array(ys), slots,
                                        self.slot_bytes, ctypes.c_void_p(self.copy_stream.cuda_stream),
                                        _stream(stream), evs, WSL_RING_PACE if pace else 0)
        _check(rc, "linear_gemv_streamed")
        return ys

    def gemm(self, mats, xs, ys, m, ldx, ldy, wfmt=WSL_W_NF4, ofmt=WSL_OUT_F32, workspace=None, stream=None,
             pace=True):
        import torch
        ydt = torch.float32 if ofmt == WSL_OUT_F32 else torch.bfloat16
        hs, ns, ks, slots, evs = self._common(mats, xs, ys, torch.bfloat16, (ydt,))
        nb = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib().linear_gemm_streamed(int(wfmt), len(mats), hs, ns, ks, _ptr_array(xs), int(m), int(ldx),
                                        _ptr_array(ys), int(ofmt), int(ldy), _ptr(workspace), nb, slots,
                                        self.slot_bytes, ctypes.c_void_p(self.copy_stream.cuda_stream),
                                        _stream(stream), evs, WSL_RING_PACE if pace else 0)
        _check(rc, "linear_gemm_streamed")
        return ys

