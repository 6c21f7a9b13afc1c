"""B200-native (sm_100a) exact IO-aware attention: a thin Python binding over the C ABI of ``libfa.so``.

Every step of the computation runs in the library's CUDA kernels; this module only marshals arguments
(PyTorch tensors -> device pointers, sizes and a CUDA stream) and turns status codes into exceptions. There is
no fallback: if the library is missing or fails to load, every call raises.

    fwd(q, k, v, causal=False, scale=None, window=(-1, -1), sinks=0) -> (out, lse)
    bwd(q, k, v, out, lse, dout, causal=False, scale=None, window=(-1, -1), sinks=0) -> (dq, dk, dv)

    cache_append(k, v, k_pages, v_pages, k_scale, v_scale, table, lens, counts=None)
    fwd_cache(q, k_pages, v_pages, k_scale, v_scale, table, lens, window_left=-1, sinks=0) -> (out, lse)

Layouts follow the C header (include/fa.h): q/out/dout [B, Sq, H, D], k/v [B, Sk, Hkv, D] (Hkv divides H:
grouped or multi-query K/V heads), fp16 or bf16, contiguous, on one CUDA device; lse is fp32 [B, H, Sq].
``scale=None`` means 1/sqrt(D); ``window=(left, right)`` limits each query to keys within left before and
right after its aligned key (-1 = unbounded side); the first ``sinks`` keys stay visible left of the window.

Every operand (inputs and caller-passed outputs alike) is checked against these shapes, dtypes and the
device of ``q`` before anything is launched; a mismatch raises ``ValueError`` or ``TypeError``. Each call
runs with ``q``'s device current and, unless a stream is given, on that device's current stream. What a call makes
itself comes from the memory of the stream it runs on, and may be freed on the current stream at any time.
"""
import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa.so")

FA_F16, FA_BF16 = 0, 1
FA_OK = 0
STATUS_NAMES = {0: "FA_OK", -1: "FA_ERR_INVALID", -2: "FA_ERR_UNSUPPORTED", -3: "FA_ERR_CUDA",
                -4: "FA_ERR_TIMEOUT", -5: "FA_ERR_WORKSPACE"}
EXPORTS = ("fa_fwd", "fa_fwd_ex", "fa_fwd_fp8", "fa_fwd_dropout", "fa_fwd_sink", "fa_bwd_dropout", "fa_bwd",
           "fa_bwd_ex", "fa_bwd_sink", "fa_bwd_sink_workspace_size", "fa_bwd_stage", "fa_bwd_noalloc",
           "fa_bwd_workspace_size", "fa_cache_append", "fa_cache_fwd", "fa_cache_workspace_size", "fa_status_string",
           "fa_device_status")

_lib = None


class FAError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: %s (%s)" % (what, status_string(status), STATUS_NAMES.get(status, status)))


def lib():
    """The loaded ``libfa.so`` (ctypes.CDLL). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libfa.so not found at %s; build it with `python -m exact_io_aware_76_b200.build`"
                          % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    u32, u64 = ctypes.c_uint32, ctypes.c_uint64
    L.fa_fwd.restype = i
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
    L.fa_bwd.restype = i
    L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, sz, vp]
    L.fa_bwd_stage.restype = i
    L.fa_bwd_stage.argtypes = [i] + L.fa_bwd.argtypes
    L.fa_bwd_noalloc.restype = i
    L.fa_bwd_noalloc.argtypes = [vp] * 9 + [i] * 6 + [f, i, vp]
    L.fa_fwd_ex.restype = i
    L.fa_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i, vp]
    L.fa_fwd_fp8.restype = i
    L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, f, f, f, vp]
    L.fa_fwd_dropout.restype = i
    L.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i, f, u64, u32, vp]
    L.fa_bwd_dropout.restype = i
    L.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i, f, u64, u32,
                                 vp, sz, vp]
    L.fa_bwd_ex.restype = i
    L.fa_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, i, vp, sz, vp]
    L.fa_fwd_sink.restype = i
    L.fa_fwd_sink.argtypes = [vp] * 5 + [i] * 10 + [f, i, vp]
    L.fa_bwd_sink.restype = i
    L.fa_bwd_sink.argtypes = [vp] * 9 + [i] * 10 + [f, i, vp, sz, vp]
    L.fa_bwd_sink_workspace_size.restype = sz
    L.fa_bwd_sink_workspace_size.argtypes = [i] * 10
    L.fa_cache_append.restype = i
    L.fa_cache_append.argtypes = [vp] * 9 + [i] * 8 + [vp]
    L.fa_cache_workspace_size.restype = sz
    L.fa_cache_workspace_size.argtypes = [i] * 5
    L.fa_cache_fwd.restype = i
    L.fa_cache_fwd.argtypes = [vp] * 9 + [i] * 10 + [f, i, vp, sz, vp]
    L.fa_bwd_workspace_size.restype = sz
    L.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_status_string.argtypes = [i]
    L.fa_device_status.restype = i
    L.fa_device_status.argtypes = [i]
    _lib = L
    return L


def status_string(status):
    return lib().fa_status_string(int(status)).decode()


# ------------------------------------------------------------------------------------------ operand checks
def _dtype_code(t):
    import torch

    if t.dtype == torch.float16:
        return FA_F16
    if t.dtype == torch.bfloat16:
        return FA_BF16
    raise TypeError("expected float16 or bfloat16, got %s" % t.dtype)


def _check(name, t, dev, shape=None, dtype=None):
    """``t`` must be a contiguous tensor on ``dev``, which the callers have found to be a CUDA device (and have
    ``shape`` / ``dtype`` if given)."""
    d = getattr(t, "device", None)
    if (d == dev and (shape is None or t.shape == shape) and (dtype is None or t.dtype == dtype)
            and t.is_contiguous()):
        return
    if d is None or d.type != "cuda" or d != dev:
        raise ValueError("%s must be a CUDA tensor on %s, got %s" % (name, dev, d))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def check_qkv(q, k, v, dtypes):
    """Shapes of the inputs: q [B, Sq, H, D], k and v [B, Sk, Hkv, D] with Hkv >= 1 dividing H, one dtype (from
    ``dtypes``) for all three, one CUDA device. Returns (B, Sq, Sk, H, Hkv, D, device)."""
    dev = getattr(q, "device", None)
    if dev is None or dev.type != "cuda":
        raise ValueError("q must be a CUDA tensor, got device %s" % dev)
    if len(q.shape) != 4:
        raise ValueError("q must be a [B, Sq, H, D] tensor, got shape %s" % (tuple(q.shape),))
    if q.dtype not in dtypes:
        raise TypeError("q must be one of %s, got %s" % (tuple(str(x) for x in dtypes), q.dtype))
    _check("q", q, dev)
    B, Sq, H, D = q.shape
    if len(k.shape) != 4 or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k must be [B=%d, Sk, Hkv, D=%d], got %s" % (B, D, tuple(k.shape)))
    Sk, Hkv = k.shape[1], k.shape[2]
    if Hkv < 1 or H % Hkv != 0:
        raise ValueError("the K/V head count %d must divide the query head count %d" % (Hkv, H))
    _check("k", k, dev, dtype=q.dtype)
    _check("v", v, dev, shape=k.shape, dtype=q.dtype)
    return B, Sq, Sk, H, Hkv, D, dev


def check_fwd_outputs(out, lse, B, Sq, H, D, dev, out_dtype):
    import torch

    _check("out", out, dev, shape=(B, Sq, H, D), dtype=out_dtype)
    _check("lse", lse, dev, shape=(B, H, Sq), dtype=torch.float32)


def check_bwd_operands(q, k, out, lse, dout, dq, dk, dv, workspace, ws_bytes, B, Sq, H, D, dev):
    check_fwd_outputs(out, lse, B, Sq, H, D, dev, q.dtype)
    _check("dout", dout, dev, shape=q.shape, dtype=q.dtype)
    _check("dq", dq, dev, shape=q.shape, dtype=q.dtype)
    _check("dk", dk, dev, shape=k.shape, dtype=q.dtype)
    _check("dv", dv, dev, shape=k.shape, dtype=q.dtype)
    if workspace is not None:
        _check("workspace", workspace, dev)
        if workspace.numel() * workspace.element_size() < ws_bytes:
            raise ValueError("workspace must hold at least %d bytes" % ws_bytes)


def _bound(w):
    """A window bound as the library's 32-bit integer; one beyond it hides nothing, as the largest does."""
    return max(-1, min(int(w), 2 ** 31 - 1))


def check_sinks(sinks, dropout_p):
    if int(sinks) != sinks or not 0 <= sinks < 2 ** 31:
        raise ValueError("sinks must be a number of keys (a 32-bit integer >= 0), got %r" % (sinks,))
    if sinks and dropout_p:
        raise ValueError("sinks and dropout do not go together")


def check_cache(k_pages, v_pages, k_scale, v_scale, table, lens, B, Hkv, D, dev):
    """The cache's operands against B sequences, Hkv heads of D. Returns (num_pages, page, max_pages)."""
    import torch

    if len(k_pages.shape) != 4 or k_pages.shape[1] != Hkv or k_pages.shape[3] != D:
        raise ValueError("k_pages must be [num_pages, Hkv=%s, page, D=%d], got %s" % (Hkv, D, tuple(k_pages.shape)))
    num_pages, page = k_pages.shape[0], k_pages.shape[2]
    if page not in (16, 32, 64, 128):
        raise ValueError("a page must hold 16, 32, 64 or 128 tokens, got %d" % page)
    _check("k_pages", k_pages, dev, dtype=torch.float8_e4m3fn)
    _check("v_pages", v_pages, dev, shape=k_pages.shape, dtype=torch.float8_e4m3fn)
    _check("k_scale", k_scale, dev, shape=(num_pages, Hkv), dtype=torch.float32)
    _check("v_scale", v_scale, dev, shape=(num_pages, Hkv), dtype=torch.float32)
    if len(table.shape) != 2 or table.shape[0] != B:
        raise ValueError("table must be [B=%d, max_pages], got %s" % (B, tuple(table.shape)))
    _check("table", table, dev, dtype=torch.int32)
    _check("lens", lens, dev, shape=(B,), dtype=torch.int32)
    return num_pages, page, table.shape[1]


_NOTHING = contextlib.nullcontext()


class _OnStream:
    """Makes a stream the current one of its device (which is current)."""

    def __init__(self, stream, caller):
        import torch

        self.set, self.stream, self.caller = torch.cuda.set_stream, stream, caller

    def __enter__(self):
        self.set(self.stream)

    def __exit__(self, *exc):
        self.set(self.caller)


def _memory_of(stream, caller):
    """The context in which a call makes its tensors: they come from the memory of the stream it runs on. (With a stream
    given, what the current one gave back its own earlier work may still be using.)"""
    return _NOTHING if stream is None else _OnStream(stream, caller)


def _caller(stream, dev):
    """The current stream where it is not the one that a call runs on: see ``_returned``."""
    if stream is None:
        return None
    import torch

    return torch.cuda.current_stream(dev)


def _returned(t, caller):
    """A tensor that a call made and returns: the caller goes on with it on the current stream, and may free it there."""
    if caller is not None:
        t.record_stream(caller)
    return t


def _stream(stream, dev):
    import torch

    if stream is None:
        return torch.cuda.current_stream(dev.index).cuda_stream
    if stream.device != dev:
        raise ValueError("stream is on %s but the tensors are on %s" % (stream.device, dev))
    return stream.cuda_stream


def _device(dev):
    import torch

    if torch.cuda.current_device() == dev.index:
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


# ------------------------------------------------------------------------------------------ entry points
def fwd(q, k, v, causal=False, scale=None, out=None, lse=None, stream=None, window=(-1, -1), dropout_p=0.0, seed=0,
        offset=0, sinks=0):
    """Forward attention. Returns (out [B,Sq,H,D] in q's dtype, lse fp32 [B,H,Sq]).

    ``sinks`` > 0 keeps the first ``sinks`` keys visible left of the window (``fa_fwd_sink``; not together with
    dropout). ``dropout_p`` > 0 drops attention probabilities with the Philox mask of ``fa_fwd_dropout`` (include/fa.h),
    keyed by ``seed`` (64-bit) and ``offset`` (32-bit); the backward must get the same three values."""
    import torch

    B, Sq, Sk, H, Hkv, D, dev = check_qkv(q, k, v, (torch.float16, torch.bfloat16))
    check_sinks(sinks, dropout_p)
    ptr, caller = _stream(stream, dev), _caller(stream, dev)
    with _device(dev), _memory_of(stream, caller):
        if out is None:
            out = _returned(torch.empty_like(q), caller)
        if lse is None:
            lse = _returned(q.new_empty((B, H, Sq), dtype=torch.float32), caller)
        check_fwd_outputs(out, lse, B, Sq, H, D, dev, q.dtype)
        shape = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Sq, Sk, H, Hkv, D,
                 int(bool(causal)), _bound(window[0]), _bound(window[1]))
        sc = (float(0.0 if scale is None else scale), _dtype_code(q))
        if dropout_p:
            rc = lib().fa_fwd_dropout(*shape, *sc, float(dropout_p), int(seed), int(offset), ptr)
        elif sinks:
            rc = lib().fa_fwd_sink(*shape, int(sinks), *sc, ptr)
        else:
            rc = lib().fa_fwd_ex(*shape, *sc, ptr)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_dropout" if dropout_p else "fa_fwd_sink" if sinks else "fa_fwd_ex")
    return out, lse


def fwd_fp8(q, k, v, causal=False, scale=None, descale=(1.0, 1.0, 1.0), out=None, lse=None, stream=None,
            window=(-1, -1)):
    """Forward attention on float8_e4m3fn inputs (D = 64 or 128). The real inputs are q * descale[0],
    k * descale[1], v * descale[2]. Returns (out bf16 [B,Sq,H,D], lse fp32 [B,H,Sq])."""
    import torch

    B, Sq, Sk, H, Hkv, D, dev = check_qkv(q, k, v, (torch.float8_e4m3fn,))
    ptr, caller = _stream(stream, dev), _caller(stream, dev)
    with _device(dev), _memory_of(stream, caller):
        if out is None:
            out = _returned(q.new_empty((B, Sq, H, D), dtype=torch.bfloat16), caller)
        if lse is None:
            lse = _returned(q.new_empty((B, H, Sq), dtype=torch.float32), caller)
        check_fwd_outputs(out, lse, B, Sq, H, D, dev, torch.bfloat16)
        rc = lib().fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Sq, Sk,
                              H, Hkv, D, int(bool(causal)), _bound(window[0]), _bound(window[1]),
                              float(0.0 if scale is None else scale), float(descale[0]), float(descale[1]),
                              float(descale[2]), ptr)
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_fp8")
    return out, lse


def workspace_size(B, Sq, H, D):
    return int(lib().fa_bwd_workspace_size(B, Sq, H, D))


def sink_workspace_size(B, Sq, Sk, H, Hkv, D, causal, window, sinks):
    """Bytes of workspace the backward with ``sinks`` needs."""
    return int(lib().fa_bwd_sink_workspace_size(B, Sq, Sk, H, Hkv, D, int(bool(causal)), _bound(window[0]),
                                                _bound(window[1]), int(sinks)))


def bwd(q, k, v, out, lse, dout, causal=False, scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None,
        stage=-1, window=(-1, -1), dropout_p=0.0, seed=0, offset=0, sinks=0):
    """Backward attention (P recomputed from lse). Returns (dq, dk, dv) in q's dtype.

    ``stage`` selects one of the three launches (0 preprocess, 1 main, 2 dQ conversion; -1 all), see
    ``fa_bwd_stage`` in include/fa.h; a caller running the stages separately must pass the same workspace."""
    import torch

    B, Sq, Sk, H, Hkv, D, dev = check_qkv(q, k, v, (torch.float16, torch.bfloat16))
    check_sinks(sinks, dropout_p)
    if stage != -1 and (dropout_p or Hkv != H or tuple(window) != (-1, -1) or sinks):
        raise ValueError("single backward stages are available for plain attention only")
    ptr, caller = _stream(stream, dev), _caller(stream, dev)
    with _device(dev), _memory_of(stream, caller):
        dq = _returned(torch.empty_like(q), caller) if dq is None else dq
        dk = _returned(torch.empty_like(k), caller) if dk is None else dk
        dv = _returned(torch.empty_like(v), caller) if dv is None else dv
        if sinks:
            ws_bytes = sink_workspace_size(B, Sq, Sk, H, Hkv, D, causal, window, sinks)
        else:
            ws_bytes = workspace_size(B, Sq, H, D)
        check_bwd_operands(q, k, out, lse, dout, dq, dk, dv, workspace, ws_bytes, B, Sq, H, D, dev)
        if workspace is None:
            workspace = q.new_empty(max(ws_bytes, 1), dtype=torch.uint8)
        sc = float(0.0 if scale is None else scale)
        bounds = (_bound(window[0]), _bound(window[1]))
        ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr())
        ws_args = (workspace.data_ptr(), workspace.numel() * workspace.element_size(), ptr)
        if dropout_p:
            rc = lib().fa_bwd_dropout(*ptrs, B, Sq, Sk, H, Hkv, D, int(bool(causal)), *bounds, sc,
                                      _dtype_code(q), float(dropout_p), int(seed), int(offset), *ws_args)
        elif sinks:
            rc = lib().fa_bwd_sink(*ptrs, B, Sq, Sk, H, Hkv, D, int(bool(causal)), *bounds, int(sinks), sc,
                                   _dtype_code(q), *ws_args)
        elif stage == -1:
            rc = lib().fa_bwd_ex(*ptrs, B, Sq, Sk, H, Hkv, D, int(bool(causal)), *bounds, sc,
                                 _dtype_code(q), *ws_args)
        else:
            rc = lib().fa_bwd_stage(int(stage), *ptrs, B, Sq, Sk, H, D, int(bool(causal)), sc, _dtype_code(q),
                                    *ws_args)
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_sink" if sinks else "fa_bwd")
    return dq, dk, dv


def bwd_noalloc(q, k, v, out, lse, dout, causal=False, scale=None, dq=None, dk=None, dv=None, stream=None):
    """``fa_bwd_noalloc``: the plain backward with the library's fixed device scratch instead of a workspace
    (problems up to FA_NOALLOC_SCRATCH_BYTES of workspace; see include/fa.h). Returns (dq, dk, dv)."""
    import torch

    B, Sq, Sk, H, Hkv, D, dev = check_qkv(q, k, v, (torch.float16, torch.bfloat16))
    if Hkv != H:
        raise ValueError("the no-alloc backward takes as many K/V heads as query heads")
    ptr, caller = _stream(stream, dev), _caller(stream, dev)
    with _device(dev), _memory_of(stream, caller):
        dq = _returned(torch.empty_like(q), caller) if dq is None else dq
        dk = _returned(torch.empty_like(k), caller) if dk is None else dk
        dv = _returned(torch.empty_like(v), caller) if dv is None else dv
        check_bwd_operands(q, k, out, lse, dout, dq, dk, dv, None, 0, B, Sq, H, D, dev)
        rc = lib().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                  dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Sq, Sk, H, D,
                                  int(bool(causal)), float(0.0 if scale is None else scale), _dtype_code(q), ptr)
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_noalloc")
    return dq, dk, dv


def cache_append(k, v, k_pages, v_pages, k_scale, v_scale, table, lens, counts=None, stream=None):
    """Rounds new tokens to e4m3 and writes them into a paged cache (``fa_cache_append`` in include/fa.h).

    k, v [B, T, Hkv, D] fp16 or bf16; k_pages, v_pages [num_pages, Hkv, page, D] float8_e4m3fn; k_scale, v_scale
    [num_pages, Hkv] fp32; table [B, max_pages] and lens [B] int32: page numbers, and lengths with the new tokens.
    The last ``counts[b]`` (int32 [B]; default T) of sequence b's rows are its new tokens. Changes the cache in place."""
    import torch

    dev = getattr(k, "device", None)
    if dev is None or dev.type != "cuda" or len(k.shape) != 4:
        raise ValueError("k must be a [B, T, Hkv, D] CUDA tensor")
    if k.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("k must be float16 or bfloat16, got %s" % k.dtype)
    B, T, Hkv, D = k.shape
    _check("k", k, dev)
    _check("v", v, dev, shape=k.shape, dtype=k.dtype)
    num_pages, page, max_pages = check_cache(k_pages, v_pages, k_scale, v_scale, table, lens, B, Hkv, D, dev)
    if counts is not None:
        _check("counts", counts, dev, shape=(B,), dtype=torch.int32)
    with _device(dev):
        rc = lib().fa_cache_append(k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                   k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                   None if counts is None else counts.data_ptr(), B, T, Hkv, D, num_pages, page,
                                   max_pages, _dtype_code(k), _stream(stream, dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_cache_append")


def cache_workspace_size(B, Sq, H, Hkv, D):
    return int(lib().fa_cache_workspace_size(B, Sq, H, Hkv, D))


def fwd_cache(q, k_pages, v_pages, k_scale, v_scale, table, lens, scale=None, window_left=-1, sinks=0, out=None,
              lse=None, workspace=None, stream=None):
    """Attention of each sequence's last Sq tokens over a paged e4m3 cache (``fa_cache_fwd`` in include/fa.h).

    q [B, Sq, H, D] fp16 or bf16; the cache as in ``cache_append``. Causal; ``window_left`` >= 0 hides keys more than
    that far before a query's own, except the first ``sinks``. Returns (out [B,Sq,H,D], lse fp32 [B,H,Sq])."""
    import torch

    dev = getattr(q, "device", None)
    if dev is None or dev.type != "cuda" or len(q.shape) != 4:
        raise ValueError("q must be a [B, Sq, H, D] CUDA tensor")
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q must be float16 or bfloat16, got %s" % q.dtype)
    _check("q", q, dev)
    B, Sq, H, D = q.shape
    Hkv = k_pages.shape[1] if len(k_pages.shape) == 4 else 0
    if Hkv < 1 or H % Hkv != 0:
        raise ValueError("the K/V head count %d must divide the query head count %d" % (Hkv, H))
    num_pages, page, max_pages = check_cache(k_pages, v_pages, k_scale, v_scale, table, lens, B, Hkv, D, dev)
    check_sinks(sinks, 0.0)
    ptr, caller = _stream(stream, dev), _caller(stream, dev)
    with _device(dev), _memory_of(stream, caller):
        if out is None:
            out = _returned(torch.empty_like(q), caller)
        if lse is None:
            lse = _returned(q.new_empty((B, H, Sq), dtype=torch.float32), caller)
        check_fwd_outputs(out, lse, B, Sq, H, D, dev, q.dtype)
        ws_bytes = cache_workspace_size(B, Sq, H, Hkv, D)
        if workspace is None:
            workspace = q.new_empty(max(ws_bytes, 1), dtype=torch.uint8)
        _check("workspace", workspace, dev)
        if workspace.numel() * workspace.element_size() < ws_bytes:
            raise ValueError("workspace must hold at least %d bytes" % ws_bytes)
        rc = lib().fa_cache_fwd(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), table.data_ptr(), lens.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, Sq, H, Hkv, D, num_pages, page, max_pages, _bound(window_left), int(sinks),
                                float(0.0 if scale is None else scale), _dtype_code(q), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), ptr)
    if rc != FA_OK:
        raise FAError(rc, "fa_cache_fwd")
    return out, lse


def device_status(reset=False, device=None):
    """The device-side sticky status word (FA_OK, or FA_ERR_TIMEOUT after a kernel gave up on a wait) of
    ``device`` (default: the current device)."""
    import torch

    if device is None:
        return int(lib().fa_device_status(int(bool(reset))))
    with torch.cuda.device(device):
        return int(lib().fa_device_status(int(bool(reset))))
