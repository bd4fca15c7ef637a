"""Python binding of librq.so, the GB300 quantized linear layer.

Thin ctypes marshalling over the C ABI declared in ``include/rq.h``; every
step of the computation runs in the library's CUDA kernels.  PyTorch only
supplies device memory (``tensor.data_ptr()``) and the current CUDA stream.
There is no fallback: if ``librq.so`` has not been built, importing this
package raises ImportError.

Function names are those of the C ABI (``rq_absmax``, ``rq_quant_e4m3``,
``rq_q4k_gemv``, ``rq_q6k_gemv``, ``rq_fp8_weight_cache``, ``rq_fp8_gemm``,
``rq_linear``...); ``Context`` wraps ``rq_ctx``.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "librq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "rq.h")

RQ_Q4K = 12
RQ_Q6K = 14
RQ_F32, RQ_F16, RQ_BF16 = 0, 1, 2
RQ_KV_E4M3, RQ_KV_I8 = 0, 1
STATUS = {0: "RQ_OK", 1: "RQ_ERR_NULL", 2: "RQ_ERR_SHAPE", 3: "RQ_ERR_QTYPE",
          4: "RQ_ERR_NOT_CACHED", 5: "RQ_ERR_ALLOC", 6: "RQ_ERR_CUDA",
          7: "RQ_ERR_TIMEOUT", 8: "RQ_ERR_ARCH", 9: "RQ_ERR_INDEX"}


class RqError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (%d)" % (where, STATUS.get(status, "?"), status))


if not os.path.exists(LIB_PATH):
    raise ImportError(
        "librq.so is not built (expected %s); run "
        "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64
_SIGS = {
    "rq_abi_version": ([], _i32),
    "rq_status_string": ([_i32], ctypes.c_char_p),
    "rq_ctx_create": ([ctypes.POINTER(_vp)], _i32),
    "rq_ctx_destroy": ([_vp], None),
    "rq_ctx_set_gemm_threshold": ([_vp, _i32], _i32),
    "rq_ctx_get_gemm_threshold": ([_vp], _i32),
    "rq_ctx_get_stats": ([_vp, _vp, _vp, _vp, _vp], _i32),
    "rq_absmax": ([_vp, _i64, _vp, _vp], _i32),
    "rq_quant_e4m3": ([_vp, _i64, _vp, _vp, _vp, _vp], _i32),
    "rq_q4k_gemv": ([_vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "rq_q6k_gemv": ([_vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "rq_fp8_weight_cache": ([_vp, _i32, _vp, _i32, _i32, ctypes.POINTER(_vp),
                             ctypes.POINTER(_vp), _vp], _i32),
    "rq_fp8_gemm": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "rq_fp8_act_cache": ([_vp, _vp, _i32, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                          _vp], _i32),
    "rq_linear": ([_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "rq_linear_group": ([_vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp], _i32),
    "rq_fp8_linear_noalloc": ([_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "rq_act_cache_invalidate": ([_vp], _i32),
    "rq_ctx_trace_begin": ([_vp, _i32], _i32),
    "rq_ctx_trace_end": ([_vp, _vp, _vp], _i32),
    "rq_ctx_trace_kinds": ([_vp, ctypes.c_uint], _i32),
    "rq_get_device_status": ([_vp], _i32),
    "rq_debug_wait_timeout": ([_i64, _vp], _i32),
    "rq_gemv_exact_outputs": ([_vp, ctypes.POINTER(_i64)], _i32),
    "rq_qk_norm_rope": ([_vp, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp], _i32),
    "rq_qkv_to_cache": ([_vp, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i32,
                         _vp], _i32),
    "rq_kv_write": ([_vp, _i32, _vp, _i64, _vp, _i64, _vp, _i32, _vp], _i32),
    "rq_kv_read": ([_vp, _i32, _vp, _vp, _vp, _i32, _vp], _i32),
    "rq_cache_attention": ([_vp, _vp, _i32, _vp, _i64, _vp, _i32, _i32, _i32, _vp, _i32, _vp,
                            _vp, ctypes.c_float, _vp], _i32),
    "rq_ctx_attention_launches": ([_vp, _vp, _vp], _i32),
    "rq_verify_chain": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "rq_verify_tree": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)


def lib():
    return _lib


def _check(status, where):
    if status != 0:
        raise RqError(status, where)


def _ptr(t):
    """Device (or host) address of a tensor, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


class _Kinds(dict):
    """Names of torch dtypes, "|" between them -> a tuple of those."""

    def __missing__(self, kind):
        import torch
        self[kind] = tuple(getattr(torch, name) for name in kind.split("|"))
        return self[kind]


_kinds = _Kinds()


def _dense(t, kind, where):
    """Address of a dense tensor of torch's dtype `kind`, or None."""
    try:
        if t.dtype in _kinds[kind] and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        return _ptr(t)
    if t.dtype in _kinds[kind]:
        raise RqError(2, where + " is not dense")
    raise RqError(3, "%s is not %s" % (where, kind))


_raw_stream = None      # torch's current-stream handle without a Stream object


def _current_stream():
    """Handle of torch's current stream on its current device.  Building the
    Stream object of torch.cuda.current_stream() takes about 3 us, more than a
    kernel launch; torch hands out the bare handle in 0.1 us."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        handle = torch.cuda.current_stream().cuda_stream      # brings CUDA up
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if raw is None or device is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            _raw_stream = lambda: raw(device())                # noqa: E731
        return handle
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream() if _raw_stream is None else _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def rq_abi_version():
    return _lib.rq_abi_version()


def rq_absmax(x, n, absmax_bits, stream=None):
    _check(_lib.rq_absmax(_ptr(x), n, _ptr(absmax_bits), _stream(stream)), "rq_absmax")


def rq_quant_e4m3(x, n, absmax_bits, out, dequant_out, stream=None):
    _check(_lib.rq_quant_e4m3(_ptr(x), n, _ptr(absmax_bits), _ptr(out),
                              _ptr(dequant_out), _stream(stream)), "rq_quant_e4m3")


def rq_q4k_gemv(w, x, y, M, N, K, stream=None):
    _check(_lib.rq_q4k_gemv(_ptr(w), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "rq_q4k_gemv")


def rq_q6k_gemv(w, x, y, M, N, K, stream=None):
    _check(_lib.rq_q6k_gemv(_ptr(w), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "rq_q6k_gemv")


def rq_fp8_gemm(x_fp8, x_dequant, w_fp8, w_dequant, y, M, N, K, stream=None):
    _check(_lib.rq_fp8_gemm(_ptr(x_fp8), _ptr(x_dequant), _ptr(w_fp8), _ptr(w_dequant),
                            _ptr(y), M, N, K, _stream(stream)), "rq_fp8_gemm")


NOALLOC_MAX_ACT_BYTES = 8 * 1024 * 1024


def rq_fp8_linear_noalloc(x, w_fp8, w_dequant, y, M, N, K, stream=None):
    """FP8 linear layer that allocates nothing (for callers that may not call
    cudaMalloc while serving): the activation's E4M3 copy lives in a fixed
    array inside the library, so (M rounded up to 16) * K must not exceed
    NOALLOC_MAX_ACT_BYTES.  w_fp8 / w_dequant are device tensors or the
    addresses Context.rq_fp8_weight_cache returns."""
    _check(_lib.rq_fp8_linear_noalloc(_ptr(x), _ptr(w_fp8), _ptr(w_dequant), _ptr(y), M, N,
                                      K, _stream(stream)), "rq_fp8_linear_noalloc")


def rq_get_device_status(stream=None):
    """Synchronise the stream; return the status code (0 = ok, 7 = timeout)."""
    return _lib.rq_get_device_status(_stream(stream))


def rq_debug_wait_timeout(limit_ns, stream=None):
    _check(_lib.rq_debug_wait_timeout(limit_ns, _stream(stream)), "rq_debug_wait_timeout")


def rq_gemv_exact_outputs(stream=None):
    """Synchronise the stream; return (and reset) how many GEMV outputs were
    recomputed on the exact fp64 path since the last call."""
    n = _i64()
    _check(_lib.rq_gemv_exact_outputs(_stream(stream), ctypes.byref(n)),
           "rq_gemv_exact_outputs")
    return n.value


def _is_f32(t):
    return t.element_size() == 4 and t.is_floating_point()


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("pages", _i64),
                ("page_size", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("format", _i32)]


class _QKParamsStruct(ctypes.Structure):
    _fields_ = [("q_weight", _vp), ("k_weight", _vp), ("cos_table", _vp), ("sin_table", _vp),
                ("positions", _i64), ("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32),
                ("rotary_dim", _i32), ("interleaved", _i32), ("eps", ctypes.c_float)]


class KVCache:
    """A paged quantized K/V cache (rq_kv_cache): codes k, v
    [pages, kv_heads, page_size, head_dim] of one byte and f32 scales k_scale,
    v_scale [pages, kv_heads, page_size].  The constructor allocates them;
    from_tensors takes the caller's."""

    def __init__(self, pages, page_size, kv_heads, head_dim, format=RQ_KV_E4M3, device="cuda"):
        import torch
        code = torch.float8_e4m3fn if format == RQ_KV_E4M3 else torch.int8
        shape = (pages, kv_heads, page_size)
        self._set(torch.zeros(shape + (head_dim,), dtype=torch.uint8, device=device).view(code),
                  torch.zeros(shape + (head_dim,), dtype=torch.uint8, device=device).view(code),
                  torch.zeros(shape, dtype=torch.float32, device=device),
                  torch.zeros(shape, dtype=torch.float32, device=device), format)

    @classmethod
    def from_tensors(cls, k, v, k_scale, v_scale, format=None):
        """The format follows from the codes' type: float8_e4m3fn or int8; bytes
        of another type hold `format`, E4M3 unless it is given."""
        import torch
        named = {torch.float8_e4m3fn: RQ_KV_E4M3, torch.int8: RQ_KV_I8}.get(k.dtype)
        if v.dtype is not k.dtype or named is not None and format not in (None, named):
            raise RqError(3, "KVCache: codes are not of the format")
        if format is None:
            format = RQ_KV_E4M3 if named is None else named
        c = cls.__new__(cls)
        c._set(k, v, k_scale, v_scale, format)
        return c

    def _set(self, k, v, k_scale, v_scale, format):
        for t in (k, v, k_scale, v_scale):
            if not t.is_contiguous():
                raise RqError(2, "KVCache: tensors must be dense")
        if (k.dim() != 4 or v.shape != k.shape or k_scale.shape != k.shape[:3] or
                v_scale.shape != k.shape[:3] or k.element_size() != 1 or v.element_size() != 1 or
                not _is_f32(k_scale) or not _is_f32(v_scale)):
            raise RqError(2, "KVCache")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.format = format
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.struct = _KVCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                     v_scale.data_ptr(), self.pages, self.page_size,
                                     self.kv_heads, self.head_dim, format)
        self.address = ctypes.addressof(self.struct)


class QKParams:
    """One layer's norm weights and rotation tables (rq_qk_params); cos, sin:
    f32 [positions, rotary_dim / 2]."""

    def __init__(self, q_heads, kv_heads, head_dim, q_weight=None, k_weight=None, eps=1e-6,
                 cos=None, sin=None, rotary_dim=None, interleaved=False):
        if rotary_dim is None:
            rotary_dim = 0 if cos is None else head_dim
        for t in (q_weight, k_weight, cos, sin):
            if t is not None and not (t.is_contiguous() and _is_f32(t)):
                raise RqError(2, "QKParams: weights and tables are dense f32")
        for t in (q_weight, k_weight):
            if t is not None and t.numel() != head_dim:
                raise RqError(2, "QKParams: a weight per coordinate of a head")
        if cos is not None and (sin is None or cos.dim() != 2 or sin.shape != cos.shape or
                                cos.shape[1] * 2 != rotary_dim):
            raise RqError(2, "QKParams: tables are [positions, rotary_dim / 2]")
        self.tensors = (q_weight, k_weight, cos, sin)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.struct = _QKParamsStruct(_ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin),
                                      0 if cos is None else cos.shape[0], q_heads, kv_heads,
                                      head_dim, rotary_dim, int(bool(interleaved)), eps)
        self.address = ctypes.addressof(self.struct)


_DTYPES = {}


def _dtype(dtype, where, *tensors):
    """The one rq_dtype of a call's tensors; `dtype` where it is given (and
    vouched for by the caller: tensors may be addresses then)."""
    if dtype is not None:
        return dtype
    first = None
    for t in tensors:
        if t is None or isinstance(t, int):
            continue
        kind = t.dtype
        if kind is not first:
            if first is not None:
                raise RqError(3, where + ": tensors of different types")
            first = kind
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: RQ_F32, torch.float16: RQ_F16, torch.bfloat16: RQ_BF16})
    return _DTYPES.get(first, -1)


def _rows(t, where):
    """Address of an output's rows, which are dense."""
    try:
        if t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        return _ptr(t)
    raise RqError(2, where + " is not dense")


def _strided_rows(t, heads, head_dim, stride, where):
    """Address of an input's rows, and the elements between its tokens."""
    try:
        if stride is None:
            if t.is_contiguous():
                return t.data_ptr(), heads * head_dim
            return t.data_ptr(), _view_stride(t, heads, head_dim, where)
    except AttributeError:
        pass
    return _ptr(t), _row_stride(t, heads, head_dim, stride, where)


def _row_stride(t, heads, head_dim, stride, where):
    """Elements between a tensor's consecutive tokens: [tokens, heads,
    head_dim], [batch, tokens, heads, head_dim] or [tokens, heads * head_dim]
    with dense heads; `stride` where t is an address (None: dense)."""
    row = heads * head_dim
    if stride is not None:
        return stride
    if t is None or isinstance(t, int):
        return row
    return row if t.is_contiguous() else _view_stride(t, heads, head_dim, where)


def _view_stride(t, heads, head_dim, where):
    """The same of a tensor that is not dense."""
    row = heads * head_dim
    shape, st = t.shape, t.stride()
    lead = len(shape) - 1
    if shape[-1] != row:        # a token's heads are an axis of their own
        lead -= 1
        if (shape[-1] != head_dim or lead < 0 or shape[lead] != heads or
                st[lead] != head_dim):
            raise RqError(2, where)
    if st[-1] != 1:
        raise RqError(2, where)
    # what is left counts tokens: one distance throughout
    token, step = None, None
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if token is None:
            token, step = st[i], st[i] * shape[i]
        elif st[i] != step:
            raise RqError(2, where)
        else:
            step = st[i] * shape[i]
    return row if token is None else token


def rq_qk_norm_rope(params, q, k, position, q_out, k_out, tokens, dtype=None, q_stride=None,
                    k_stride=None, stream=None):
    """Per-head norm and position rotation: q -> q_out, k -> k_out (either
    pair may be None)."""
    d = params.head_dim
    qp, qs = _strided_rows(q, params.q_heads, d, q_stride, "rq_qk_norm_rope: q")
    kp, ks = _strided_rows(k, params.kv_heads, d, k_stride, "rq_qk_norm_rope: k")
    _check(_lib.rq_qk_norm_rope(params.address,
                                _dtype(dtype, "rq_qk_norm_rope", q, k, q_out, k_out), qp, qs,
                                kp, ks, _dense(position, "int32", "rq_qk_norm_rope: position"),
                                _rows(q_out, "rq_qk_norm_rope: q_out"),
                                _rows(k_out, "rq_qk_norm_rope: k_out"), tokens, _stream(stream)),
           "rq_qk_norm_rope")


def rq_qkv_to_cache(params, q, k, v, position, q_out, cache, slot, tokens, dtype=None,
                    q_stride=None, k_stride=None, v_stride=None, stream=None):
    """The same, with k and v quantized into the cache at slot (int64)."""
    d, hk = params.head_dim, params.kv_heads
    qp, qs = _strided_rows(q, params.q_heads, d, q_stride, "rq_qkv_to_cache: q")
    kp, ks = _strided_rows(k, hk, d, k_stride, "rq_qkv_to_cache: k")
    vp, vs = _strided_rows(v, hk, d, v_stride, "rq_qkv_to_cache: v")
    _check(_lib.rq_qkv_to_cache(params.address, _dtype(dtype, "rq_qkv_to_cache", q, k, v, q_out),
                                qp, qs, kp, ks, vp, vs,
                                _dense(position, "int32", "rq_qkv_to_cache: position"),
                                _rows(q_out, "rq_qkv_to_cache: q_out"), cache.address,
                                _dense(slot, "int64", "rq_qkv_to_cache: slot"), tokens,
                                _stream(stream)), "rq_qkv_to_cache")


def rq_kv_write(cache, k, v, slot, tokens, dtype=None, k_stride=None, v_stride=None,
                stream=None):
    """Quantize k and v rows into the cache at slot (int64)."""
    kp, ks = _strided_rows(k, cache.kv_heads, cache.head_dim, k_stride, "rq_kv_write: k")
    vp, vs = _strided_rows(v, cache.kv_heads, cache.head_dim, v_stride, "rq_kv_write: v")
    _check(_lib.rq_kv_write(cache.address, _dtype(dtype, "rq_kv_write", k, v), kp, ks, vp, vs,
                            _dense(slot, "int64", "rq_kv_write: slot"), tokens, _stream(stream)),
           "rq_kv_write")


def rq_kv_read(cache, slot, k_out, v_out, tokens, dtype=None, stream=None):
    """Read the cache back at slot (int64) into dense rows."""
    _check(_lib.rq_kv_read(cache.address, _dtype(dtype, "rq_kv_read", k_out, v_out),
                           _dense(slot, "int64", "rq_kv_read: slot"),
                           _rows(k_out, "rq_kv_read: k_out"), _rows(v_out, "rq_kv_read: v_out"),
                           tokens, _stream(stream)), "rq_kv_read")


def rq_verify_chain(token, p, q, u, accepted, next, batch, drafts, vocab, stream=None):
    """Keep or reject chains of drafts and draw the next token (q may be None)."""
    _check(_lib.rq_verify_chain(_dense(token, "int32", "rq_verify_chain: token"),
                                _dense(p, "float32", "rq_verify_chain: p"),
                                None if q is None else
                                _dense(q, "float32", "rq_verify_chain: q"),
                                _dense(u, "float32", "rq_verify_chain: u"),
                                _dense(accepted, "int32", "rq_verify_chain: accepted"),
                                _dense(next, "int32", "rq_verify_chain: next"), batch, drafts,
                                vocab, _stream(stream)), "rq_verify_chain")


def rq_verify_tree(token, parent, p, u, accepted, next, path, batch, drafts, vocab, stream=None):
    """Walk trees of drafts by draws from the target, and draw the next token."""
    _check(_lib.rq_verify_tree(_dense(token, "int32", "rq_verify_tree: token"),
                               _dense(parent, "int32", "rq_verify_tree: parent"),
                               _dense(p, "float32", "rq_verify_tree: p"),
                               _dense(u, "float32", "rq_verify_tree: u"),
                               _dense(accepted, "int32", "rq_verify_tree: accepted"),
                               _dense(next, "int32", "rq_verify_tree: next"),
                               _dense(path, "int32", "rq_verify_tree: path"), batch, drafts, vocab,
                               _stream(stream)), "rq_verify_tree")


class Context:
    """Owns an rq_ctx: FP8 weight cache, activation scratch, device scalars."""

    def __init__(self, gemm_threshold=None):
        h = _vp()
        _check(_lib.rq_ctx_create(ctypes.byref(h)), "rq_ctx_create")
        self._h = h
        if gemm_threshold is not None:
            self.set_gemm_threshold(gemm_threshold)

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            _lib.rq_ctx_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_gemm_threshold(self, m):
        _check(_lib.rq_ctx_set_gemm_threshold(self._h, m), "rq_ctx_set_gemm_threshold")

    @property
    def gemm_threshold(self):
        return _lib.rq_ctx_get_gemm_threshold(self._h)

    def stats(self):
        vals = [_i64() for _ in range(4)]
        _check(_lib.rq_ctx_get_stats(self._h, *[ctypes.byref(v) for v in vals]),
               "rq_ctx_get_stats")
        hits, misses, nw, nbytes = (v.value for v in vals)
        return {"act_hits": hits, "act_misses": misses, "weights": nw,
                "weight_bytes": nbytes}

    def rq_fp8_weight_cache(self, qtype, w, N, K, stream=None):
        """-> (device address of E4M3 [N x K], device address of the scale)."""
        wq = _vp()
        wd = _vp()
        _check(_lib.rq_fp8_weight_cache(self._h, qtype, _ptr(w), N, K, ctypes.byref(wq),
                                        ctypes.byref(wd), _stream(stream)),
               "rq_fp8_weight_cache")
        return wq.value, wd.value

    def rq_fp8_act_cache(self, x, M, K, stream=None):
        """-> (device address of E4M3 [M_pad x K], device address of the scale)."""
        xq = _vp()
        xd = _vp()
        _check(_lib.rq_fp8_act_cache(self._h, _ptr(x), M, K, ctypes.byref(xq),
                                     ctypes.byref(xd), _stream(stream)),
               "rq_fp8_act_cache")
        return xq.value, xd.value

    def rq_linear_group(self, qtypes, ws, x, ys, Ns, M, K, stream=None):
        """Linears sharing x: ys[i] = x . ws[i]^T, one call."""
        n = len(qtypes)
        qt = (_i32 * n)(*qtypes)
        wp = (_vp * n)(*[_ptr(w) for w in ws])
        yp = (_vp * n)(*[_ptr(y) for y in ys])
        nn = (_i32 * n)(*Ns)
        _check(_lib.rq_linear_group(self._h, n, qt, wp, _ptr(x), yp, nn, M, K,
                                    _stream(stream)), "rq_linear_group")

    def rq_linear(self, qtype, w, x, y, M, N, K, stream=None):
        _check(_lib.rq_linear(self._h, qtype, _ptr(w), _ptr(x), _ptr(y), M, N, K,
                              _stream(stream)), "rq_linear")

    def rq_cache_attention(self, cache, q, out, page_table, length, batch, new_tokens, q_heads,
                           scale, tree=None, max_pages=None, dtype=None, q_stride=None,
                           stream=None):
        """Attention of batch x new_tokens tokens over the cache; tree: 64-bit
        words [batch, new_tokens] of visible new tokens, None: causal.
        page_table [batch, max_pages] and length are dense int32 tensors (of a
        wider table, its part in use is taken as a dense copy, or the table
        whole)."""
        qp, qs = _strided_rows(q, q_heads, cache.head_dim, q_stride, "rq_cache_attention: q")
        if not isinstance(page_table, int):
            shape = page_table.shape
            if len(shape) != 2 or max_pages not in (None, shape[1]):
                raise RqError(2, "rq_cache_attention: page_table is [batch, max_pages]")
            max_pages = shape[1]
        _check(_lib.rq_cache_attention(self._h, cache.address,
                                       _dtype(dtype, "rq_cache_attention", q, out), qp, qs,
                                       _rows(out, "rq_cache_attention: out"), batch, new_tokens,
                                       q_heads,
                                       _dense(page_table, "int32", "rq_cache_attention: page_table"),
                                       max_pages,
                                       _dense(length, "int32", "rq_cache_attention: length"),
                                       None if tree is None else
                                       _dense(tree, "int64|uint64", "rq_cache_attention: tree"),
                                       scale, _stream(stream)), "rq_cache_attention")

    def attention_launches(self):
        """How many rq_cache_attention calls launched the kernel for few query
        rows, and the one for many."""
        few, many = _i64(), _i64()
        _check(_lib.rq_ctx_attention_launches(self._h, ctypes.byref(few), ctypes.byref(many)),
               "rq_ctx_attention_launches")
        return few.value, many.value

    TRACE_KINDS = ("gemv", "absmax", "quant", "gemm", "wcache")

    def rq_ctx_trace_begin(self, capacity):
        _check(_lib.rq_ctx_trace_begin(self._h, capacity), "rq_ctx_trace_begin")

    def rq_ctx_trace_kinds(self, kinds):
        """Trace only the named kinds (a subset of TRACE_KINDS)."""
        mask = 0
        for k in kinds:
            mask |= 1 << self.TRACE_KINDS.index(k)
        _check(_lib.rq_ctx_trace_kinds(self._h, mask), "rq_ctx_trace_kinds")

    def rq_ctx_trace_end(self):
        """-> {kind: (kernel count, summed device ms)}"""
        counts = (_i64 * 5)()
        ms = (ctypes.c_double * 5)()
        _check(_lib.rq_ctx_trace_end(self._h, counts, ms), "rq_ctx_trace_end")
        return {k: (counts[i], ms[i]) for i, k in enumerate(self.TRACE_KINDS)}

    def rq_act_cache_invalidate(self):
        _check(_lib.rq_act_cache_invalidate(self._h), "rq_act_cache_invalidate")
