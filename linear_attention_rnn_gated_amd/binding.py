"""ctypes binding of libgdn.so (include/gdn.h).

Argument marshalling only: torch provides device memory and the current HIP
stream; every step of the layer runs in the library's kernels.  If the library
is not built, lib() raises -- there is no fallback implementation.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_WORKSPACE = -3
GDN_ERR_HIP = -4
GDN_F32 = 0
GDN_BF16 = 1
OP_PREFILL, OP_DECODE, OP_FWD_BWD, OP_PREFILL_CHUNKED, OP_PREFILL_CONTINUE = 0, 1, 2, 3, 4

EXPORTS = ["gdn_workspace_bytes", "gdn_cache_init", "gdn_prefill", "gdn_decode_step",
           "gdn_fwd_bwd", "gdn_profile_enable", "gdn_profile_read", "gdn_contract_id",
           "gdn_contract_check", "gdn_error_string", "gdn_prefill_chunked",
           "gdn_prefill_continue", "gdn_fwd_bwd_ex", "gdn_decode_step_noalloc",
           "gdn_fwd_bwd_chunked", "gdn_decode_step_native", "gdn_profile_filter",
           "gdn_lru_cache_init", "gdn_lru_prefill", "gdn_lru_prefill_continue",
           "gdn_lru_decode_step", "gdn_lru_workspace_bytes", "gdn_lru_fwd_bwd",
           "gdn_qk_rotary", "gdn_qk_workspace_bytes", "gdn_qk_rotary_bwd", "gdn_rope_freqs"]

LRU_CHUNK = 32    # tokens per chunk of the gated linear recurrence
LRU_SMALL = 2048  # a prefill of at most so many tokens needs no workspace
LRU_GROUP = 256   # channels per position counter of its cache
LRU_GATES = {"none": 0, "complement": 1, "norm": 2}
QK_NORMS = {"none": 0, "l2": 1, "rms": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_DTYPE_CODES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_DTYPES = {GDN_F32: torch.float32, GDN_BF16: torch.bfloat16}


class Shape(ctypes.Structure):
    _fields_ = [("H_qk", ctypes.c_int32), ("H_v", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("C", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("qk_l2norm", ctypes.c_int32), ("scale", ctypes.c_float)]


class CacheStruct(ctypes.Structure):
    _fields_ = [("S_run", ctypes.c_void_p), ("S_chunk", ctypes.c_void_p),
                ("kbuf", ctypes.c_void_p), ("vbuf", ctypes.c_void_p),
                ("bbuf", ctypes.c_void_p), ("gbuf", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


class LruShape(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("g_dtype", ctypes.c_int32), ("gate", ctypes.c_int32)]


class LruCacheStruct(ctypes.Structure):
    _fields_ = [("S", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


class QkShape(ctypes.Structure):
    _fields_ = [("H_q", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d", ctypes.c_int32),
                ("r", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("rope_scale", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("attn", ctypes.c_double)]


_lib = None


def lib():
    """Loads libgdn.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run linear_attention_rnn_gated_amd/build.py "
                               "(the GPU path has no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sp = ctypes.POINTER(Shape)
        cp = ctypes.POINTER(CacheStruct)
        L.gdn_workspace_bytes.argtypes = [sp, i32, i64, i32]
        L.gdn_workspace_bytes.restype = sz
        L.gdn_cache_init.argtypes = [sp, i32, vp, cp, vp]
        L.gdn_cache_init.restype = ctypes.c_int
        L.gdn_prefill.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, cp, vp, sz, vp]
        L.gdn_prefill_chunked.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                          vp]
        L.gdn_prefill_chunked.restype = ctypes.c_int
        L.gdn_prefill_continue.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, cp, vp, vp,
                                           vp, sz, vp]
        L.gdn_prefill_continue.restype = ctypes.c_int
        L.gdn_prefill.restype = ctypes.c_int
        L.gdn_decode_step.argtypes = [sp, i32, vp, vp, vp, vp, vp, cp, vp, vp, vp, sz, vp]
        L.gdn_decode_step.restype = ctypes.c_int
        L.gdn_decode_step_noalloc.argtypes = [sp, i32, vp, vp, vp, vp, vp, cp, vp, vp, vp]
        L.gdn_decode_step_noalloc.restype = ctypes.c_int
        L.gdn_fwd_bwd.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  vp, vp, vp, vp, vp, vp, sz, vp]
        L.gdn_fwd_bwd.restype = ctypes.c_int
        L.gdn_fwd_bwd_ex.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                     vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.gdn_fwd_bwd_ex.restype = ctypes.c_int
        L.gdn_fwd_bwd_chunked.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.gdn_fwd_bwd_chunked.restype = ctypes.c_int
        L.gdn_decode_step_native.argtypes = [sp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.gdn_decode_step_native.restype = ctypes.c_int
        L.gdn_profile_enable.argtypes = [ctypes.c_int]
        L.gdn_profile_enable.restype = ctypes.c_int
        L.gdn_profile_filter.argtypes = [ctypes.c_char_p]
        L.gdn_profile_filter.restype = ctypes.c_int
        L.gdn_profile_read.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_int64)]
        L.gdn_profile_read.restype = ctypes.c_int
        L.gdn_contract_id.argtypes = []
        L.gdn_contract_id.restype = ctypes.c_char_p
        L.gdn_contract_check.argtypes = [ctypes.c_char_p]
        L.gdn_contract_check.restype = ctypes.c_int
        L.gdn_error_string.argtypes = [ctypes.c_int]
        L.gdn_error_string.restype = ctypes.c_char_p
        ls, lc, qs = (ctypes.POINTER(t) for t in (LruShape, LruCacheStruct, QkShape))
        L.gdn_lru_cache_init.argtypes = [ls, i32, vp, lc, vp]
        L.gdn_lru_prefill.argtypes = [ls, i32, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, lc, vp,
                                      sz, vp]
        L.gdn_lru_prefill_continue.argtypes = [ls, i32, vp, vp, vp, i64, vp, i64, lc, vp, i64, vp,
                                               vp, sz, vp]
        L.gdn_lru_decode_step.argtypes = [ls, i32, vp, i64, vp, i64, lc, vp, i64, vp]
        L.gdn_lru_workspace_bytes.argtypes = [ls, i32, i64, i32]
        L.gdn_lru_fwd_bwd.argtypes = [ls, i32, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, vp, i64,
                                      vp, vp, i64, vp, i64, vp, vp, sz, vp]
        L.gdn_qk_rotary.argtypes = [qs, i64, vp, i32, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp,
                                    i64, vp, i64, vp]
        L.gdn_qk_workspace_bytes.argtypes = [qs, i64]
        L.gdn_qk_rotary_bwd.argtypes = [qs, i64, vp, i32, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp,
                                        i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, sz, vp]
        L.gdn_rope_freqs.argtypes = [i32, ctypes.c_double, ctypes.POINTER(RopeScaling), vp, vp]
        for name in ("lru_cache_init", "lru_prefill", "lru_prefill_continue", "lru_decode_step",
                     "lru_fwd_bwd", "qk_rotary", "qk_rotary_bwd", "rope_freqs"):
            getattr(L, "gdn_" + name).restype = ctypes.c_int
        L.gdn_lru_workspace_bytes.restype = L.gdn_qk_workspace_bytes.restype = sz
        _lib = L
    return _lib


class GdnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().gdn_error_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _check(status, where):
    if status != GDN_OK:
        raise GdnError(status, where)


def make_shape(H_qk, H_v, d, C, in_dtype, qk_l2norm=True, scale=1.0, d_v=None):
    dt = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}[in_dtype] \
        if isinstance(in_dtype, torch.dtype) else int(in_dtype)
    return Shape(H_qk, H_v, d, d if d_v is None else d_v, C, dt, int(bool(qk_l2norm)),
                 float(scale))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def workspace_bytes(shape, n_seqs, total_tokens, op):
    return int(lib().gdn_workspace_bytes(ctypes.byref(shape), n_seqs, total_tokens, op))


def profile_enable(on=True):
    _check(lib().gdn_profile_enable(int(bool(on))), "gdn_profile_enable")


def profile_filter(kernel=""):
    """Only launches whose kernel name contains `kernel` are timed ("" = all)."""
    _check(lib().gdn_profile_filter(kernel.encode() if kernel else None), "gdn_profile_filter")


def profile_read(kernel=""):
    """(total ms, launches) of the timed launches whose name contains `kernel`;
    waits for them and forgets them."""
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    _check(lib().gdn_profile_read(kernel.encode() if kernel else None, ctypes.byref(ms),
                                  ctypes.byref(n)), "gdn_profile_read")
    return ms.value, n.value


def contract_id():
    return lib().gdn_contract_id().decode()


def contract_check(other_id):
    """GDN_OK (0) if another library's contract id equals this library's."""
    return lib().gdn_contract_check(other_id.encode())


def _workspace(shape, n, T, op, device, ws=None):
    need = workspace_bytes(shape, n, T, op)
    if need == 0:
        raise GdnError(GDN_ERR_UNSUPPORTED, "gdn_workspace_bytes")
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws


def _req(t, dtype, shape, name):
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")


class Cache:
    """Decode cache (gdn_cache_t) of n sequences, owned by torch tensors."""

    def __init__(self, shape, n, device, in_dtype):
        d, C, Hq, Hv = shape.d_k, shape.C, shape.H_qk, shape.H_v
        f32 = dict(dtype=torch.float32, device=device)
        self.S_run = torch.empty(n, Hv, d, d, **f32)
        self.S_chunk = torch.empty(n, Hv, d, d, **f32)
        self.kbuf = torch.empty(n, C, Hq, d, **f32)
        self.vbuf = torch.empty(n, C, Hv, d, dtype=in_dtype, device=device)
        self.bbuf = torch.empty(n, C, Hv, **f32)
        self.gbuf = torch.empty(n, C, Hv, **f32)
        self.pos = torch.zeros(n, Hv, dtype=torch.int32, device=device)
        self.n = n

    def struct(self):
        return CacheStruct(*[t.data_ptr() for t in self.tensors()])

    def tensors(self):
        return [self.S_run, self.S_chunk, self.kbuf, self.vbuf, self.bbuf, self.gbuf, self.pos]

    def clone(self):
        c = object.__new__(Cache)
        for name in ["S_run", "S_chunk", "kbuf", "vbuf", "bbuf", "gbuf", "pos"]:
            setattr(c, name, getattr(self, name).clone())
        c.n = self.n
        return c


def gdn_cache_init(shape, n, device, in_dtype, h0=None):
    c = Cache(shape, n, device, in_dtype)
    cs = c.struct()
    _check(lib().gdn_cache_init(ctypes.byref(shape), n, _ptr(h0), ctypes.byref(cs),
                                _stream(device)), "gdn_cache_init")
    return c


def _cu_pair(cu_seqlens, dev, cu_seqlens_host):
    """Device and host int32 copies of cu_seqlens.  A caller that keeps a host
    copy (cu_seqlens_host, CPU int32 [N+1], same values) saves the
    device-to-host copy, which waits for the stream, on every call.  With
    cu_seqlens_host=False the library gets NULL and makes that copy itself."""
    cu_dev = cu_seqlens.to(dev, torch.int32).contiguous()
    if cu_seqlens_host is False:
        return cu_dev, None
    if cu_seqlens_host is None:
        return cu_dev, cu_seqlens.to("cpu", torch.int32).contiguous()
    if (cu_seqlens_host.device.type != "cpu" or cu_seqlens_host.dtype != torch.int32
            or cu_seqlens_host.numel() != cu_seqlens.numel()):
        raise ValueError("cu_seqlens_host: expected a CPU int32 tensor shaped like cu_seqlens")
    return cu_dev, cu_seqlens_host.contiguous()


def gdn_prefill(shape, q, k, v, beta, g, cu_seqlens, h0=None, cache=None, want_hT=True,
                ws=None, out=None, cu_seqlens_host=None, hT_out=None):
    """Packed prefill.  cu_seqlens: int32 device tensor [N+1]; its host copy is
    taken here unless cu_seqlens_host is given.  out / hT_out: optional
    caller-owned o [T, H_v, d] and hT [N, H_v, d, d] fp32.  Returns (o, hT)."""
    dev = q.device
    T = q.shape[0]
    n = cu_seqlens.numel() - 1
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (T, Hq, d), "q")
    _req(k, idt, (T, Hq, d), "k")
    _req(v, idt, (T, Hv, d), "v")
    _req(beta, torch.float32, (T, Hv), "beta")
    _req(g, torch.float32, (T, Hv), "g")
    if h0 is not None:
        _req(h0, torch.float32, (n, Hv, d, d), "h0")
    cu_dev, cu_host = _cu_pair(cu_seqlens, dev, cu_seqlens_host)
    o = torch.empty(T, Hv, d, dtype=torch.float32, device=dev) if out is None else out
    _req(o, torch.float32, (T, Hv, d), "out")
    if hT_out is not None:
        _req(hT_out, torch.float32, (n, Hv, d, d), "hT_out")
        hT = hT_out
    else:
        hT = torch.empty(n, Hv, d, d, dtype=torch.float32, device=dev) if want_hT else None
    ws = _workspace(shape, n, T, OP_PREFILL, dev, ws)
    cs = cache.struct() if cache is not None else None
    st = lib().gdn_prefill(ctypes.byref(shape), n, _ptr(cu_dev),
                           _ptr(cu_host), _ptr(q), _ptr(k), _ptr(v),
                           _ptr(beta), _ptr(g), _ptr(h0), _ptr(o), _ptr(hT),
                           ctypes.byref(cs) if cs is not None else None, _ptr(ws),
                           ws.numel(), _stream(dev))
    _check(st, "gdn_prefill")
    return o, hT


def gdn_prefill_continue(shape, q, k, v, beta, g, cu_seqlens, cache, pos_host, want_hT=True,
                         ws=None, out=None, cu_seqlens_host=None):
    """Next tokens of sequences whose cache stands anywhere inside a chunk.
    pos_host: each sequence's position in its current chunk (host int32 [N],
    the value of cache.pos).  Returns (o, hT) of the new tokens."""
    dev = q.device
    T = q.shape[0]
    n = cu_seqlens.numel() - 1
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (T, Hq, d), "q")
    _req(k, idt, (T, Hq, d), "k")
    _req(v, idt, (T, Hv, d), "v")
    _req(beta, torch.float32, (T, Hv), "beta")
    _req(g, torch.float32, (T, Hv), "g")
    cu_dev, cu_host = _cu_pair(cu_seqlens, dev, cu_seqlens_host)
    pos = torch.as_tensor(pos_host, dtype=torch.int32).to("cpu").contiguous()
    if pos.numel() != n:
        raise ValueError(f"pos_host: expected {n} values, got {pos.numel()}")
    o = torch.empty(T, Hv, d, dtype=torch.float32, device=dev) if out is None else out
    hT = torch.empty(n, Hv, d, d, dtype=torch.float32, device=dev) if want_hT else None
    ws = _workspace(shape, n, T, OP_PREFILL_CONTINUE, dev, ws)
    cs = cache.struct()
    st = lib().gdn_prefill_continue(ctypes.byref(shape), n, _ptr(cu_dev),
                                    _ptr(cu_host),
                                    ctypes.c_void_p(pos.data_ptr()), _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(beta), _ptr(g), ctypes.byref(cs), _ptr(o), _ptr(hT),
                                    _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "gdn_prefill_continue")
    return o, hT


def gdn_prefill_chunked(shape, q, k, v, beta, g, cu_seqlens, h0=None, want_hT=True, ws=None,
                        out=None, cu_seqlens_host=None):
    """Native-mixed baseline prefill (chunk-form outputs; not bit-identical to
    gdn_prefill / decode).  Returns (o, hT)."""
    dev = q.device
    T = q.shape[0]
    n = cu_seqlens.numel() - 1
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (T, Hq, d), "q")
    _req(k, idt, (T, Hq, d), "k")
    _req(v, idt, (T, Hv, d), "v")
    _req(beta, torch.float32, (T, Hv), "beta")
    _req(g, torch.float32, (T, Hv), "g")
    if h0 is not None:
        _req(h0, torch.float32, (n, Hv, d, d), "h0")
    cu_dev, cu_host = _cu_pair(cu_seqlens, dev, cu_seqlens_host)
    o = torch.empty(T, Hv, d, dtype=torch.float32, device=dev) if out is None else out
    hT = torch.empty(n, Hv, d, d, dtype=torch.float32, device=dev) if want_hT else None
    ws = _workspace(shape, n, T, OP_PREFILL_CHUNKED, dev, ws)
    st = lib().gdn_prefill_chunked(ctypes.byref(shape), n, _ptr(cu_dev),
                                   _ptr(cu_host), _ptr(q), _ptr(k), _ptr(v),
                                   _ptr(beta), _ptr(g), _ptr(h0), _ptr(o), _ptr(hT), _ptr(ws),
                                   ws.numel(), _stream(dev))
    _check(st, "gdn_prefill_chunked")
    return o, hT


def gdn_decode_step(shape, q, k, v, beta, g, cache, pos_host=None, ws=None, out=None):
    """One token per sequence: q, k [N, H_qk, d], v [N, H_v, d], beta, g [N, H_v].
    pos_host: optional int32 CPU tensor [N, H_v] mirroring cache.pos.  Returns o."""
    dev = q.device
    n = q.shape[0]
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (n, Hq, d), "q")
    _req(k, idt, (n, Hq, d), "k")
    _req(v, idt, (n, Hv, d), "v")
    _req(beta, torch.float32, (n, Hv), "beta")
    _req(g, torch.float32, (n, Hv), "g")
    o = torch.empty(n, Hv, d, dtype=torch.float32, device=dev) if out is None else out
    ws = _workspace(shape, n, 0, OP_DECODE, dev, ws)
    cs = cache.struct()
    ph = None
    if pos_host is not None:
        ph = ctypes.c_void_p(pos_host.data_ptr())
    st = lib().gdn_decode_step(ctypes.byref(shape), n, _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                               _ptr(g), ctypes.byref(cs), ph, _ptr(o), _ptr(ws), ws.numel(),
                               _stream(dev))
    _check(st, "gdn_decode_step")
    return o


def gdn_decode_step_noalloc(shape, q, k, v, beta, g, cache, pos_host=None, out=None):
    """gdn_decode_step without a workspace: the library's fixed device scratch
    holds the resync's chunk factors (for callers that cannot allocate).  Pass
    `out` (fp32 [N, H_v, d]) to keep this call free of allocations too."""
    dev = q.device
    n = q.shape[0]
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (n, Hq, d), "q")
    _req(k, idt, (n, Hq, d), "k")
    _req(v, idt, (n, Hv, d), "v")
    _req(beta, torch.float32, (n, Hv), "beta")
    _req(g, torch.float32, (n, Hv), "g")
    o = torch.empty(n, Hv, d, dtype=torch.float32, device=dev) if out is None else out
    _req(o, torch.float32, (n, Hv, d), "out")
    cs = cache.struct()
    ph = None if pos_host is None else ctypes.c_void_p(pos_host.data_ptr())
    st = lib().gdn_decode_step_noalloc(ctypes.byref(shape), n, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(beta), _ptr(g), ctypes.byref(cs), ph, _ptr(o),
                                       _stream(dev))
    _check(st, "gdn_decode_step_noalloc")
    return o


def gdn_decode_step_native(shape, q, k, v, beta, g, S, out=None):
    """Native-mixed baseline decode: the plain token step on the state S
    (fp32 [N, H_v, d, d], updated in place); no chunk buffers, no resync.
    Returns o."""
    dev = q.device
    n = q.shape[0]
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (n, Hq, d), "q")
    _req(k, idt, (n, Hq, d), "k")
    _req(v, idt, (n, Hv, d), "v")
    _req(beta, torch.float32, (n, Hv), "beta")
    _req(g, torch.float32, (n, Hv), "g")
    _req(S, torch.float32, (n, Hv, d, d), "S")
    o = torch.empty(n, Hv, d, dtype=torch.float32, device=dev) if out is None else out
    _req(o, torch.float32, (n, Hv, d), "out")
    st = lib().gdn_decode_step_native(ctypes.byref(shape), n, _ptr(q), _ptr(k), _ptr(v),
                                      _ptr(beta), _ptr(g), _ptr(S), _ptr(o), _stream(dev))
    _check(st, "gdn_decode_step_native")
    return o


def gdn_fwd_bwd_chunked(shape, q, k, v, beta, g, cu_seqlens, dO, h0=None, dhT=None, ws=None,
                        cu_seqlens_host=None):
    """Native-mixed baseline trainer step: chunk-form forward outputs, the same
    backward (fp32 gradients).  Returns dict(o, hT, dq, dk, dv, dbeta, dg, dh0)."""
    return gdn_fwd_bwd(shape, q, k, v, beta, g, cu_seqlens, dO, h0=h0, dhT=dhT, ws=ws,
                       cu_seqlens_host=cu_seqlens_host, _native=True)


def gdn_fwd_bwd(shape, q, k, v, beta, g, cu_seqlens, dO, h0=None, dhT=None, ws=None,
                grad_dtype=torch.float32, cu_seqlens_host=None, out=None, _native=False):
    """Trainer forward + backward.  Returns dict(o, hT, dq, dk, dv, dbeta, dg, dh0);
    dq, dk, dv in grad_dtype (float32 or bfloat16), the rest float32.  out:
    optional dict of caller-owned tensors for some or all of those outputs."""
    dev = q.device
    T = q.shape[0]
    n = cu_seqlens.numel() - 1
    d, Hq, Hv = shape.d_k, shape.H_qk, shape.H_v
    idt = q.dtype
    _req(q, idt, (T, Hq, d), "q")
    _req(k, idt, (T, Hq, d), "k")
    _req(v, idt, (T, Hv, d), "v")
    _req(beta, torch.float32, (T, Hv), "beta")
    _req(g, torch.float32, (T, Hv), "g")
    _req(dO, torch.float32, (T, Hv, d), "dO")
    if h0 is not None:
        _req(h0, torch.float32, (n, Hv, d, d), "h0")
    if dhT is not None:
        _req(dhT, torch.float32, (n, Hv, d, d), "dhT")
    cu_dev, cu_host = _cu_pair(cu_seqlens, dev, cu_seqlens_host)
    f32 = dict(dtype=torch.float32, device=dev)
    gd = dict(dtype=grad_dtype, device=dev)
    code = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}[grad_dtype]
    r = dict(o=torch.empty(T, Hv, d, **f32), hT=torch.empty(n, Hv, d, d, **f32),
             dq=torch.empty(T, Hq, d, **gd), dk=torch.empty(T, Hq, d, **gd),
             dv=torch.empty(T, Hv, d, **gd), dbeta=torch.empty(T, Hv, **f32),
             dg=torch.empty(T, Hv, **f32), dh0=torch.empty(n, Hv, d, d, **f32))
    for key, t in (out or {}).items():
        _req(t, r[key].dtype, tuple(r[key].shape), f"out[{key!r}]")
        r[key] = t
    ws = _workspace(shape, n, T, OP_FWD_BWD, dev, ws)
    if _native:
        if grad_dtype != torch.float32:
            raise ValueError("gdn_fwd_bwd_chunked writes fp32 gradients")
        st = lib().gdn_fwd_bwd_chunked(
            ctypes.byref(shape), n, _ptr(cu_dev), _ptr(cu_host), _ptr(q), _ptr(k), _ptr(v),
            _ptr(beta), _ptr(g), _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(r["o"]), _ptr(r["hT"]),
            _ptr(r["dq"]), _ptr(r["dk"]), _ptr(r["dv"]), _ptr(r["dbeta"]), _ptr(r["dg"]),
            _ptr(r["dh0"]), _ptr(ws), ws.numel(), _stream(dev))
        _check(st, "gdn_fwd_bwd_chunked")
        return r
    st = lib().gdn_fwd_bwd_ex(ctypes.byref(shape), n, _ptr(cu_dev),
                              _ptr(cu_host), _ptr(q), _ptr(k), _ptr(v),
                              _ptr(beta), _ptr(g), _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(r["o"]),
                              _ptr(r["hT"]), code, _ptr(r["dq"]), _ptr(r["dk"]), _ptr(r["dv"]),
                              _ptr(r["dbeta"]), _ptr(r["dg"]), _ptr(r["dh0"]), _ptr(ws),
                              ws.numel(), _stream(dev))
    _check(st, "gdn_fwd_bwd_ex")
    return r


# ---- gated linear recurrence, and the norms and rotation of q and k -----------
# These calls take rows with any distance between tokens (slices of wider
# projections), check that every tensor lies on the first one's GPU, and run
# there on that GPU's current stream, whichever GPU is current.
# Rows behind the last sequence of cu_seqlens are not written: in an output that
# the call makes itself they hold no values.


def _gpu(t, name):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name}: expected a GPU tensor, got one on {dev}")
    return dev


def _rows(t, dtype, n, width, dev, name):
    """The distance between the rows of t [n, width], after checking it."""
    if t.dtype != dtype or t.shape != (n, width) or t.device != dev:
        raise ValueError(f"{name}: expected {dtype} ({n}, {width}) on {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    ld, unit = t.stride()
    if n <= 1:
        ld = width
    if (unit != 1 and width > 1) or ld < width:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap, got strides "
                         f"{t.stride()}")
    return ld


def _heads(t, dtype, T, H, d, dev, name):
    """The distance between the tokens' rows of t [T, H, d], after checking it."""
    if t.dtype != dtype or t.shape != (T, H, d) or t.device != dev:
        raise ValueError(f"{name}: expected {dtype} ({T}, {H}, {d}) on {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    ld, head, unit = t.stride()
    if T <= 1:
        ld = H * d
    if unit != 1 or (head != d and H > 1) or ld < H * d:
        raise ValueError(f"{name}: a token's heads must be contiguous and tokens must not "
                         f"overlap, got strides {t.stride()}")
    return ld


def _dense(t, dtype, shape, dev, name):
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device} "
                         f"contiguous={t.is_contiguous()}")
    return t.data_ptr()


def _optional(t, dtype, shape, dev, name):
    return None if t is None else _dense(t, dtype, shape, dev, name)


def _launch(name, dev, *args):
    """Calls library function `name` with the current stream of `dev` as last
    argument (its raw handle: a stream object would cost 2 us a call)."""
    fn = getattr(_lib or lib(), name)
    index = dev.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != GDN_OK:
        raise GdnError(status, name)


def _packed(cu_seqlens, cu_seqlens_host, dev, T):
    """(N, device copy, host copy) of cu_seqlens over T rows."""
    i32 = torch.int32
    if (cu_seqlens_host is not None and cu_seqlens_host is not False and cu_seqlens.device == dev
            and cu_seqlens.dtype == i32 and cu_seqlens_host.dtype == i32
            and cu_seqlens_host.device.type == "cpu" and cu_seqlens.shape == cu_seqlens_host.shape
            and cu_seqlens.is_contiguous() and cu_seqlens_host.is_contiguous()):
        cu_dev, cu_host = cu_seqlens, cu_seqlens_host
    else:
        cu_dev, cu_host = _cu_pair(cu_seqlens, dev, cu_seqlens_host)
        if cu_host is None:
            raise ValueError("cu_seqlens_host: expected a CPU int32 tensor or None")
    n = cu_host.numel() - 1
    if cu_host.dim() != 1 or n < 0:
        raise ValueError("cu_seqlens: expected one dimension of N + 1 values")
    end = ctypes.c_int32.from_address(cu_host.data_ptr() + 4 * n).value
    if end > T:
        raise ValueError(f"cu_seqlens: ends at {end}, past the {T} rows given")
    return n, cu_dev, cu_host


def _host_copy(cu_seqlens_host):
    """cu_seqlens_host as _packed takes it.  False, as gdn_prefill takes it, has the
    device copy read back: here by the binding, whose check of the rows needs it."""
    return None if cu_seqlens_host is False else cu_seqlens_host


def make_lru_shape(D, in_dtype, g_dtype=torch.float32, gate="none"):
    """Shape of a gated linear recurrence of D channels: x, o in in_dtype, the
    log decay g in g_dtype; gate "none", "complement" or "norm" gives the
    input's weight 1, 1 - alpha or sqrt(1 - alpha^2).  g <= 0 is meant; the sum
    of larger ones over 32 tokens has to stay below 88.7 (see include/gdn.h)."""
    return LruShape(D, _DTYPE_CODES[in_dtype], _DTYPE_CODES[g_dtype], LRU_GATES[gate])


def lru_workspace_bytes(shape, n_seqs, total_tokens, op=OP_FWD_BWD):
    return int(lib().gdn_lru_workspace_bytes(ctypes.byref(shape), n_seqs, total_tokens, op))


def _cache_tensor(name):
    """A tensor attribute of LruCache: assigning another one drops the struct of addresses."""
    held = "_" + name

    def get(self):
        return getattr(self, held)

    def put(self, t):
        setattr(self, held, t)
        self._struct = None
    return property(get, put)


class LruCache:
    """Decode cache (gdn_lru_cache_t) of n sequences of D channels, owned by
    torch tensors.  S, A, B and pos may be assigned (a reordered batch, say); the
    next call checks and takes the tensors that are there then."""

    def __init__(self, D, n, device):
        f32 = dict(dtype=torch.float32, device=device)
        self._hold(torch.empty(n, D, **f32), torch.empty(n, D, **f32), torch.empty(n, D, **f32),
                   torch.zeros(n, -(-D // LRU_GROUP), dtype=torch.int32, device=device))

    @classmethod
    def of(cls, S, A, B, pos):
        """A cache over existing tensors: S, A, B fp32 [n, D], pos int32
        [n, ceil(D / 256)]."""
        c = object.__new__(cls)
        _gpu(S, "S")
        c._hold(S, A, B, pos)
        c.struct()
        return c

    S, A, B, pos = (_cache_tensor(name) for name in ("S", "A", "B", "pos"))
    n = property(lambda self: self._S.shape[0])
    D = property(lambda self: self._S.shape[1])
    device = property(lambda self: self._S.device)

    def _hold(self, S, A, B, pos):
        self.S, self.A, self.B, self.pos = S, A, B, pos

    def struct(self):
        # an assignment drops the struct; a tensor given other memory in place moves its address
        at = (self._S.data_ptr(), self._A.data_ptr(), self._B.data_ptr(), self._pos.data_ptr())
        if self._struct is None or at != self._at:
            (n, D), dev = self._S.shape, self._S.device
            for t, name in ((self._S, "S"), (self._A, "A"), (self._B, "B")):
                _dense(t, torch.float32, (n, D), dev, name)
            _dense(self._pos, torch.int32, (n, -(-D // LRU_GROUP)), dev, "pos")
            self._at, self._fits, self._struct = at, (n, D, dev), LruCacheStruct(*at)
        return self._struct

    def __getstate__(self):
        return dict(self.__dict__, _struct=None)  # a copy or a restored cache has addresses of its own

    def tensors(self):
        return [self._S, self._A, self._B, self._pos]

    def state(self):
        """The states now, [n, D]: A S + B, rounded twice.  The calls' o and hT are
        one fma and may differ in the last place; hT of a continuation without
        tokens (a cu_seqlens of zeros) is that fma."""
        return self._A * self._S + self._B

    def clone(self):
        return LruCache.of(*[t.clone() for t in self.tensors()])

    def check(self, shape, n, dev):
        """The struct, after checking that it is one of n sequences on dev."""
        struct = self.struct()
        if self._fits != (n, shape.D, dev):
            raise ValueError(f"cache: expected {n} sequences of {shape.D} channels on {dev}, got "
                             f"{self.n} of {self.D} on {self.device}")
        return struct


def gdn_lru_cache_init(shape, n, device, h0=None):
    """Cache of n sequences with nothing decoded yet, from h0 (fp32 [n, D])."""
    c = LruCache(shape.D, n, device)
    dev = _gpu(c.S, "device")
    _launch("gdn_lru_cache_init", dev, ctypes.byref(shape), n,
            _optional(h0, torch.float32, (n, shape.D), dev, "h0"), ctypes.byref(c.struct()))
    return c


def _lru_prefill(name, shape, x, g, cu_seqlens, h0, cache, want_hT, ws, out, hT_out,
                 cu_seqlens_host):
    dev = _gpu(x, "x")
    T, D = x.shape[0], shape.D
    xt = _DTYPES.get(shape.in_dtype)
    ldx = _rows(x, xt, T, D, dev, "x")
    ldg = _rows(g, _DTYPES.get(shape.g_dtype), T, D, dev, "g")
    n, cu_dev, cu_host = _packed(cu_seqlens, _host_copy(cu_seqlens_host), dev, T)
    o = torch.empty(T, D, dtype=xt, device=dev) if out is None else out
    ldo = _rows(o, xt, T, D, dev, "out")
    hT = hT_out
    if hT is None and want_hT:
        hT = torch.empty(n, D, dtype=torch.float32, device=dev)
    p_hT = _optional(hT, torch.float32, (n, D), dev, "hT_out")
    cs = None if cache is None else ctypes.byref(cache.check(shape, n, dev))
    tail = (None, 0)
    if T > LRU_SMALL:
        ws = _scratch(ws, lru_workspace_bytes(shape, n, T, OP_PREFILL), dev,
                      "gdn_lru_workspace_bytes")
        tail = (ws.data_ptr(), ws.numel())
    head = (ctypes.byref(shape), n, cu_dev.data_ptr(), cu_host.data_ptr(), x.data_ptr(), ldx,
            g.data_ptr(), ldg)
    if name == "gdn_lru_prefill":
        p_h0 = _optional(h0, torch.float32, (n, D), dev, "h0")
        _launch(name, dev, *head, p_h0, o.data_ptr(), ldo, p_hT, cs, *tail)
    else:
        _launch(name, dev, *head, cs, o.data_ptr(), ldo, p_hT, *tail)
    return o, hT


def gdn_lru_prefill(shape, x, g, cu_seqlens, h0=None, cache=None, want_hT=True, ws=None,
                    out=None, hT_out=None, cu_seqlens_host=None):
    """Packed prefill of the gated linear recurrence: x, g [T, D] from h0 (fp32
    [N, D]); fills `cache` for decode if given.  Returns (o [T, D] in x's type,
    hT fp32 [N, D]).  out may be x."""
    return _lru_prefill("gdn_lru_prefill", shape, x, g, cu_seqlens, h0, cache, want_hT, ws,
                        out, hT_out, cu_seqlens_host)


def gdn_lru_prefill_continue(shape, x, g, cu_seqlens, cache, want_hT=True, ws=None, out=None,
                             hT_out=None, cu_seqlens_host=None):
    """The next tokens of the sequences of `cache`, which may stand anywhere in
    their chunks; the cache moves on.  Returns (o, hT) of the new tokens."""
    return _lru_prefill("gdn_lru_prefill_continue", shape, x, g, cu_seqlens, None, cache, want_hT,
                        ws, out, hT_out, cu_seqlens_host)


def gdn_lru_decode_step(shape, x, g, cache, out=None):
    """One token per sequence: x, g [N, D]; the cache moves on.  Returns o."""
    dev = _gpu(x, "x")
    n, D = x.shape[0], shape.D
    xt = _DTYPES.get(shape.in_dtype)
    ldx = _rows(x, xt, n, D, dev, "x")
    ldg = _rows(g, _DTYPES.get(shape.g_dtype), n, D, dev, "g")
    o = torch.empty(n, D, dtype=xt, device=dev) if out is None else out
    ldo = _rows(o, xt, n, D, dev, "out")
    cs = cache.check(shape, n, dev)
    _launch("gdn_lru_decode_step", dev, ctypes.byref(shape), n, x.data_ptr(), ldx, g.data_ptr(),
            ldg, ctypes.byref(cs), o.data_ptr(), ldo)
    return o


def gdn_lru_fwd_bwd(shape, x, g, cu_seqlens, dO, h0=None, dhT=None, ws=None, want_o=True,
                    out=None, cu_seqlens_host=None):
    """Trainer forward + backward of the gated linear recurrence, or with
    want_o=False the backward alone.  Returns dict(o, hT, dx, dg, dh0), without
    o and hT in the latter case; o, dx in x's type, dg in g's.  out: optional
    dict of caller-owned tensors for some of them."""
    dev = _gpu(x, "x")
    T, D = x.shape[0], shape.D
    xt, gt = _DTYPES.get(shape.in_dtype), _DTYPES.get(shape.g_dtype)
    ldx = _rows(x, xt, T, D, dev, "x")
    ldg = _rows(g, gt, T, D, dev, "g")
    lddo = _rows(dO, xt, T, D, dev, "dO")
    n, cu_dev, cu_host = _packed(cu_seqlens, _host_copy(cu_seqlens_host), dev, T)
    kinds = {"o": (xt, T), "hT": (torch.float32, n), "dx": (xt, T), "dg": (gt, T),
             "dh0": (torch.float32, n)}
    if not want_o:
        del kinds["o"], kinds["hT"]
    out = out or {}
    if not set(out) <= set(kinds):
        raise ValueError(f"out: expected some of {sorted(kinds)}, got {sorted(out)}")
    r = {key: out[key] if key in out else torch.empty(rows, D, dtype=dt, device=dev)
         for key, (dt, rows) in kinds.items()}
    ld = {key: _rows(r[key], kinds[key][0], T, D, dev, f"out[{key!r}]")
          for key in ("o", "dx", "dg") if key in r}
    for key in ("hT", "dh0"):
        if key in r:
            _dense(r[key], torch.float32, (n, D), dev, f"out[{key!r}]")
    ws = _scratch(ws, lru_workspace_bytes(shape, n, T), dev, "gdn_lru_workspace_bytes")
    ptr = {key: t.data_ptr() for key, t in r.items()}
    _launch("gdn_lru_fwd_bwd", dev, ctypes.byref(shape), n, cu_dev.data_ptr(), cu_host.data_ptr(),
            x.data_ptr(), ldx, g.data_ptr(), ldg,
            _optional(h0, torch.float32, (n, D), dev, "h0"), dO.data_ptr(), lddo,
            _optional(dhT, torch.float32, (n, D), dev, "dhT"), ptr.get("o"), ld.get("o", 0),
            ptr.get("hT"), ptr["dx"], ld["dx"], ptr["dg"], ld["dg"], ptr["dh0"], ws.data_ptr(),
            ws.numel())
    return r


def _scratch(ws, need, dev, where):
    if need == 0:
        raise GdnError(GDN_ERR_UNSUPPORTED, where)
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws: expected contiguous uint8 on {dev}")
    return ws


def rope_freqs(r, base=10000.0, kind="none", factor=1.0, orig_len=0.0, low=1.0, high=32.0,
               attn=0.0):
    """(inv_freq fp32 CPU [r / 2], rope_scale): the rotary frequencies of r
    elements, scaled for contexts `factor` times longer than orig_len (kind
    "none", "linear", "ntk", "yarn" or "bands"; see include/gdn.h)."""
    inv_freq = torch.empty(max(r, 0) // 2, dtype=torch.float32)
    scale = ctypes.c_float()
    s = RopeScaling(ROPE_SCALINGS[kind], factor, orig_len, low, high, attn)
    _check(lib().gdn_rope_freqs(r, base, ctypes.byref(s), inv_freq.data_ptr() or None,
                                ctypes.addressof(scale)), "gdn_rope_freqs")
    return inv_freq, scale.value


def make_qk_shape(H_q, H_k, d, r, in_dtype, out_dtype=None, norm="l2", layout="half", eps=1e-6,
                  scale=1.0, rope_scale=1.0, weight_offset=0.0):
    """Shape of gdn_qk_rotary: H_q and H_k heads of d elements, the first r of
    them rotated; norm "l2", "rms" or "none"; layout "half" or "interleaved";
    q is multiplied by scale; RMS weights act as weight_offset + w."""
    return QkShape(H_q, H_k, d, r, _DTYPE_CODES[in_dtype],
                   _DTYPE_CODES[in_dtype if out_dtype is None else out_dtype], QK_NORMS[norm],
                   ROPE_LAYOUTS[layout], eps, scale, rope_scale, weight_offset)


def qk_workspace_bytes(shape, total_tokens):
    return int(lib().gdn_qk_workspace_bytes(ctypes.byref(shape), total_tokens))


def _qk_args(shape, q, k, inv_freq, pos, cu_seqlens, start, w_q, w_k):
    """The device of q, the arguments that the two calls share, and the types."""
    dev = _gpu(q, "q")
    T, d = q.shape[0], shape.d
    it = _DTYPES.get(shape.in_dtype)
    ldq = _heads(q, it, T, shape.H_q, d, dev, "q")
    ldk, pk = 0, None
    if shape.H_k > 0:
        ldk, pk = _heads(k, it, T, shape.H_k, d, dev, "k"), k.data_ptr()
    if (pos is None) == (cu_seqlens is None):
        raise ValueError("expected either pos or cu_seqlens")
    n, i32 = 0, torch.int32
    if pos is None:
        n = cu_seqlens.numel() - 1
        if n < 0 or (n == 0 and T > 0):
            raise ValueError("cu_seqlens: expected N + 1 values")
        p_cu = _dense(cu_seqlens, i32, (n + 1,), dev, "cu_seqlens")
        where = (None, n, p_cu, _optional(start, i32, (n,), dev, "start"))
    else:
        if start is not None:
            raise ValueError("start: only with cu_seqlens")
        where = (_dense(pos, i32, (T,), dev, "pos"), 0, None, None)
    f32 = torch.float32
    freq = None
    if shape.r > 0:
        if inv_freq is None:
            raise ValueError("inv_freq: expected the frequencies of the rotation")
        freq = _dense(inv_freq, f32, (shape.r // 2,), dev, "inv_freq")
    weights = (_optional(w_q, f32, (d,), dev, "w_q"), _optional(w_k, f32, (d,), dev, "w_k"))
    return dev, (ctypes.byref(shape), T, *where, freq, *weights, q.data_ptr(), ldq, pk, ldk)


def gdn_qk_rotary(shape, q, k, inv_freq, pos=None, cu_seqlens=None, start=None, w_q=None,
                  w_k=None, q_out=None, k_out=None):
    """Norms of q [T, H_q, d] and k [T, H_k, d] per head and the rotation by
    each token's position, in one pass.  Positions: pos (int32 GPU tensor [T]),
    or, from cu_seqlens (int32 GPU tensor), the place in the sequence plus
    start[n].  Returns (q, k) in the shape's output type; q_out / k_out may be q
    and k themselves.  Prepares q and k for gdn_prefill and gdn_decode_step with
    qk_l2norm=False (and scale 1)."""
    dev, args = _qk_args(shape, q, k, inv_freq, pos, cu_seqlens, start, w_q, w_k)
    T, d, ot = q.shape[0], shape.d, _DTYPES.get(shape.out_dtype)
    qo = torch.empty(T, shape.H_q, d, dtype=ot, device=dev) if q_out is None else q_out
    ko = torch.empty(T, shape.H_k, d, dtype=ot, device=dev) if k_out is None else k_out
    ldq = _heads(qo, ot, T, shape.H_q, d, dev, "q_out")
    ldk = _heads(ko, ot, T, shape.H_k, d, dev, "k_out")
    _launch("gdn_qk_rotary", dev, *args, qo.data_ptr(), ldq, ko.data_ptr(), ldk)
    return qo, ko


def gdn_qk_rotary_bwd(shape, q, k, dq_out, dk_out, inv_freq, pos=None, cu_seqlens=None,
                      start=None, w_q=None, w_k=None, ws=None):
    """Gradient of gdn_qk_rotary: from the gradients of its outputs, dict(dq,
    dk) in q's type and, with norm "rms", dw_q and dw_k (fp32 [d]).  dq and dk are
    dense tensors of their own (the C entry takes rows of any distance)."""
    dev, args = _qk_args(shape, q, k, inv_freq, pos, cu_seqlens, start, w_q, w_k)
    T, d = q.shape[0], shape.d
    ot = _DTYPES.get(shape.out_dtype)
    lddq = _heads(dq_out, ot, T, shape.H_q, d, dev, "dq_out")
    lddk, pdk = 0, None
    if shape.H_k > 0:
        lddk, pdk = _heads(dk_out, ot, T, shape.H_k, d, dev, "dk_out"), dk_out.data_ptr()
    r = {"dq": torch.empty(T, shape.H_q, d, dtype=q.dtype, device=dev),
         "dk": torch.empty(T, shape.H_k, d, dtype=q.dtype, device=dev)}
    p_dw, p_ws, ws_bytes = (None, None), None, 0
    if shape.norm == QK_NORMS["rms"]:
        r["dw_q"] = torch.empty(d, dtype=torch.float32, device=dev)
        r["dw_k"] = torch.empty(d, dtype=torch.float32, device=dev)
        ws = _scratch(ws, qk_workspace_bytes(shape, T), dev, "gdn_qk_workspace_bytes")
        p_dw, p_ws, ws_bytes = (r["dw_q"].data_ptr(), r["dw_k"].data_ptr()), ws.data_ptr(), ws.numel()
    _launch("gdn_qk_rotary_bwd", dev, *args, dq_out.data_ptr(), lddq, pdk, lddk,
            r["dq"].data_ptr(), 0, r["dk"].data_ptr(), 0, *p_dw, p_ws, ws_bytes)
    return r
