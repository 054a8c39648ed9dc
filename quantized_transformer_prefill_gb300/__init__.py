"""Python binding of ``libminfer.so`` (the C ABI in ``include/minfer.h``).

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  The library must have been built (``build.build()``); there is
no fallback of any kind when it is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import build as _build

LIB_PATH = _build.LIB_PATH
_lock = threading.Lock()
_lib = None

MINFER_F32 = 0
MINFER_F16 = 1
MINFER_Q8_0 = 8
MINFER_BF16 = 30
ROPE_STYLES = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

ERR_NAMES = {0: "OK", -1: "ERR_ARG", -2: "ERR_POS_OOB", -3: "ERR_TOKEN_OOB",
             -4: "ERR_MISSING_TENSOR", -5: "ERR_SHAPE", -6: "ERR_CUDA", -7: "ERR_OOM",
             -8: "ERR_DEVICE", -9: "ERR_STATE", -10: "ERR_TOO_LARGE"}
# device status codes (minfer_device_status): the bounded wait that gave up
DEV_NAMES = {0: "DEV_OK", 1: "DEV_TIMEOUT_TMA_EMPTY", 2: "DEV_TIMEOUT_MMA_FULL",
             3: "DEV_TIMEOUT_MMA_SLOT", 4: "DEV_TIMEOUT_EPILOGUE", 5: "DEV_TIMEOUT_DRAIN",
             6: "DEV_TIMEOUT_ATTN"}

# every entry point declared in include/minfer.h: name -> (argtypes, restype)
_P, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class Hparams(ctypes.Structure):
    _fields_ = [("n_layer", ctypes.c_int), ("n_embd", ctypes.c_int), ("n_head", ctypes.c_int),
                ("n_head_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("n_ff", ctypes.c_int),
                ("n_vocab", ctypes.c_int), ("max_seq_len", ctypes.c_int),
                ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("tied_embeddings", ctypes.c_int), ("qk_norm", ctypes.c_int)]


class Tensor(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("type", ctypes.c_int), ("ne0", ctypes.c_int64),
                ("ne1", ctypes.c_int64), ("data", ctypes.c_void_p)]


class PagedCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_head_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int), ("style", ctypes.c_int),
                ("scaling", ctypes.c_int), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("n_ctx_orig", ctypes.c_int), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("attn_factor", ctypes.c_double)]


class RopeTableDesc(ctypes.Structure):
    _fields_ = [("turn", ctypes.c_uint64 * 64), ("mscale", ctypes.c_float),
                ("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int), ("style", ctypes.c_int)]


SIGNATURES = {
    "minfer_model_create": ([ctypes.POINTER(Hparams), ctypes.POINTER(_P)], _I),
    "minfer_model_set_tensor": ([_P, ctypes.POINTER(Tensor)], _I),
    "minfer_model_finalize": ([_P], _I),
    "minfer_load_weights": ([ctypes.POINTER(Hparams), ctypes.POINTER(Tensor), _I,
                             ctypes.POINTER(_P)], _I),
    "minfer_free": ([_P], None),
    "minfer_kv_create": ([_P, _I, ctypes.POINTER(_P)], _I),
    "minfer_kv_n_ctx": ([_P], _I),
    "minfer_kv_free": ([_P], None),
    "minfer_kv_read": ([_P, _I, _I, _I, _I, _P], _I),
    "minfer_kv_write": ([_P, _I, _I, _I, _I, _P], _I),
    "minfer_prefill": ([_P, _P, _P, _I, _P, _P], _I),
    "minfer_prefill_device": ([_P, _P, _P, _I, _P, _P, _P], _I),
    "minfer_prefill_n": ([_P, _P, _P, _I, _P, _I, _P], _I),
    "minfer_prefill_device_n": ([_P, _P, _P, _I, _P, _I, _P, _P], _I),
    "minfer_sync_status": ([_P, _P], _I),
    "minfer_set_dump": ([_P, _P, _I], _I),
    "minfer_debug_read": ([_P, ctypes.c_char_p, _P, _I64], _I),
    "minfer_debug_layer": ([_P, _I], _I),
    "minfer_profile_enable": ([_P, _I], _I),
    "minfer_profile_read": ([_P, _I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(_I64),
                             ctypes.POINTER(ctypes.c_double)], _I),
    "minfer_op_quantize": ([_P, _I64, _I64, _P, _P], _I),
    "minfer_op_rmsnorm_quantize": ([_P, _P, _I64, _I64, _F, _P, _P], _I),
    "minfer_op_gemm": ([_P, _P, _I64, _P, _P, _I64, _I64, _P, _P], _I),
    "minfer_op_gemm_noalloc": ([_P, _P, _I64, _P, _P, _I64, _I64, _P], _I),
    "minfer_op_gemm_swiglu": ([_P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P], _I),
    "minfer_op_attention": ([_P, _P, _I, _P, _P, _I, _I, _I, _I, _P], _I),
    "minfer_op_rope_store": ([_P, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P], _I),
    "minfer_op_qknorm_rope_store": ([_P, _P, _P, _P, _F, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P], _I),
    "minfer_rope_prepare": ([ctypes.POINTER(RopeSpec), ctypes.POINTER(RopeTableDesc)], _I),
    "minfer_op_page_tables": ([_P, _P, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _I, _P, _P], _I),
    "minfer_op_rope_paged_store": ([_P, _I, _I64, _P, _P, _P, _F, _P, _P, _P, _I, _I, _P, _P, _I64,
                                    _P, _P], _I),
    "minfer_op_paged_attention_workspace": ([_I, _I, _P, ctypes.POINTER(_I64)], _I),
    "minfer_op_paged_attention": ([_P, _I64, _P, _P, _I64, _I, _P, _I, _I, _F, _P, _I64, _P, _P,
                                   _I64, _P, _P], _I),
    "minfer_op_token_logprobs_workspace": ([_I64, _I64, _I, ctypes.POINTER(_I64)], _I),
    "minfer_op_token_logprobs": ([_P, _I, _I64, _I64, _I64, _P, _I, _P, _P, _P, _P, _P, _I64, _P,
                                  _P], _I),
    "minfer_strerror": ([_I], ctypes.c_char_p),
    "minfer_device_status": ([_P], _I),
    "minfer_debug_fault": ([_P, _I, _I64], _I),
}


class MinferError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = lib().minfer_strerror(code).decode()
        super().__init__(f"{what}: {ERR_NAMES.get(code, code)} ({msg})")


def lib():
    """The loaded library.  Raises when it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "quantized_transformer_prefill_gb300.build.build()")
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def check(rc: int, what: str = "minfer"):
    if rc != 0:
        raise MinferError(rc, what)


def hparams_of(cfg) -> Hparams:
    return Hparams(cfg.n_layer, cfg.n_embd, cfg.n_head, cfg.n_head_kv, cfg.head_dim, cfg.n_ff,
                   cfg.n_vocab, cfg.max_seq_len, cfg.rope_theta, cfg.rms_eps, int(cfg.tied),
                   int(getattr(cfg, "qk_norm", False)))


class Model:
    """A model on the current CUDA device."""

    def __init__(self, hp: Hparams):
        self._hp = hp
        ptr = ctypes.c_void_p()
        check(lib().minfer_model_create(ctypes.byref(hp), ctypes.byref(ptr)), "model_create")
        self.ptr = ptr.value
        self.n_vocab = hp.n_vocab
        self.n_embd = hp.n_embd
        self.n_layer = hp.n_layer
        self._dump = None

    def set_tensor(self, name: str, data: np.ndarray, ne0: int, ne1: int, ttype: int = MINFER_F32):
        data = np.ascontiguousarray(data)
        t = Tensor(name.encode(), ttype, ne0, ne1, data.ctypes.data)
        check(lib().minfer_model_set_tensor(self.ptr, ctypes.byref(t)), f"set_tensor {name}")

    def finalize(self):
        check(lib().minfer_model_finalize(self.ptr), "finalize")

    def kv(self, n_ctx: int) -> "KV":
        return KV(self, n_ctx)

    def prefill(self, kv: "KV", ids: np.ndarray, pos: np.ndarray, out: np.ndarray | None = None):
        """Host-buffer prefill: returns the last token's logits (float32 [V])."""
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        pos = np.ascontiguousarray(pos, dtype=np.int32)
        if out is None:
            out = np.empty(self.n_vocab, np.float32)
        rc = lib().minfer_prefill(self.ptr, ids.ctypes.data, pos.ctypes.data, ids.size, kv.ptr,
                                  out.ctypes.data)
        check(rc, "prefill")
        return out

    def prefill_n(self, kv: "KV", ids: np.ndarray, pos: np.ndarray, n_out: int,
                  out: np.ndarray | None = None):
        """Host-buffer prefill returning the logits of the last n_out tokens
        (float32 [n_out][V], token order)."""
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        pos = np.ascontiguousarray(pos, dtype=np.int32)
        if out is None:
            out = np.empty((n_out, self.n_vocab), np.float32)
        check(lib().minfer_prefill_n(self.ptr, ids.ctypes.data, pos.ctypes.data, ids.size, kv.ptr,
                                     n_out, out.ctypes.data), "prefill_n")
        return out

    def prefill_device_n(self, kv: "KV", d_ids: int, d_pos: int, nt: int, n_out: int,
                         d_logits: int, stream: int | None = None) -> int:
        return lib().minfer_prefill_device_n(self.ptr, d_ids, d_pos, nt, kv.ptr, n_out, d_logits,
                                             stream)

    def prefill_rc(self, kv: "KV", ids, pos, out=None) -> int:
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        pos = np.ascontiguousarray(pos, dtype=np.int32)
        if out is None:
            out = np.empty(self.n_vocab, np.float32)
        return lib().minfer_prefill(self.ptr, ids.ctypes.data, pos.ctypes.data, ids.size, kv.ptr,
                                    out.ctypes.data)

    def prefill_device(self, kv: "KV", d_ids: int, d_pos: int, nt: int, d_logits: int,
                       stream: int | None = None) -> int:
        """Device-buffer prefill enqueued on `stream` (raw cudaStream_t); no sync."""
        return lib().minfer_prefill_device(self.ptr, d_ids, d_pos, nt, kv.ptr, d_logits, stream)

    def sync_status(self, stream: int | None = None) -> int:
        return lib().minfer_sync_status(self.ptr, stream)

    def set_dump(self, buf: np.ndarray | None):
        """buf: float32 [n_layer + 1][max_tokens][n_embd] host array, or None."""
        if buf is None:
            check(lib().minfer_set_dump(self.ptr, None, 0), "set_dump")
            self._dump = None
            return
        assert buf.dtype == np.float32 and buf.flags.c_contiguous
        self._dump = buf
        check(lib().minfer_set_dump(self.ptr, buf.ctypes.data, buf.shape[1]), "set_dump")

    def debug_read(self, name: str, out: np.ndarray) -> np.ndarray:
        check(lib().minfer_debug_read(self.ptr, name.encode(), out.ctypes.data, out.nbytes),
              f"debug_read {name}")
        return out

    def debug_layer(self, layer: int):
        """Capture layer `layer`'s intermediates on the next prefill (-1: off)."""
        check(lib().minfer_debug_layer(self.ptr, layer), "debug_layer")

    def debug_fault(self, layer: int, wait_limit_ns: int = 0):
        """Test hook: layer >= 0 makes that layer's gate/up GEMM withhold one
        operand stage and every GEMM wait give up after wait_limit_ns;
        -1 turns it off."""
        check(lib().minfer_debug_fault(self.ptr, layer, wait_limit_ns), "debug_fault")

    def device_status(self) -> int:
        return lib().minfer_device_status(self.ptr)

    def profile_enable(self, on: bool = True):
        check(lib().minfer_profile_enable(self.ptr, int(on)), "profile_enable")

    def profile_read(self) -> dict:
        out = {}
        k = 0
        while True:
            name = ctypes.c_char_p()
            n = ctypes.c_int64()
            ms = ctypes.c_double()
            if lib().minfer_profile_read(self.ptr, k, ctypes.byref(name), ctypes.byref(n),
                                         ctypes.byref(ms)) != 0:
                break
            out[name.value.decode()] = (int(n.value), float(ms.value))
            k += 1
        return out

    def free(self):
        if getattr(self, "ptr", None):
            lib().minfer_free(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class KV:
    def __init__(self, model: Model, n_ctx: int):
        ptr = ctypes.c_void_p()
        check(lib().minfer_kv_create(model.ptr, n_ctx, ctypes.byref(ptr)), "kv_create")
        self.ptr = ptr.value
        self.model = model
        self.n_ctx = lib().minfer_kv_n_ctx(self.ptr)
        self.width = model._hp.n_head_kv * model._hp.head_dim

    def read(self, layer: int, which: int, row0: int = 0, nrows: int | None = None) -> np.ndarray:
        nrows = self.n_ctx - row0 if nrows is None else nrows
        out = np.empty((nrows, self.width), np.float32)
        check(lib().minfer_kv_read(self.ptr, layer, which, row0, nrows, out.ctypes.data), "kv_read")
        return out

    def write(self, layer: int, which: int, row0: int, data: np.ndarray):
        data = np.ascontiguousarray(data, dtype=np.float32)
        check(lib().minfer_kv_write(self.ptr, layer, which, row0, data.shape[0], data.ctypes.data),
              "kv_write")

    def free(self):
        if getattr(self, "ptr", None):
            lib().minfer_kv_free(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def load_model(cfg, tensors) -> Model:
    """Create a model from an iterable of (name, array, ne0, ne1, type)."""
    m = Model(hparams_of(cfg))
    for name, arr, ne0, ne1, ttype in tensors:
        m.set_tensor(name, arr, ne0, ne1, ttype)
    m.finalize()
    return m


# ------------------------------------------------------------------ single stages
# torch tensors (CUDA) in, torch tensors out; the library does the work.

def _ptr(t):
    return t.data_ptr() if t is not None else None


def op_quantize(x):
    import torch
    rows, n = x.shape
    nb = (n + 31) // 32
    q = torch.zeros((rows, nb * 32), dtype=torch.int8, device=x.device)
    d = torch.zeros((rows, nb), dtype=torch.int16, device=x.device)
    check(lib().minfer_op_quantize(_ptr(x.contiguous()), rows, n, _ptr(q), _ptr(d)), "op_quantize")
    return q, d


def op_rmsnorm_quantize(x, w, eps: float):
    import torch
    rows, n = x.shape
    nb = (n + 31) // 32
    q = torch.zeros((rows, nb * 32), dtype=torch.int8, device=x.device)
    d = torch.zeros((rows, nb), dtype=torch.int16, device=x.device)
    check(lib().minfer_op_rmsnorm_quantize(_ptr(x.contiguous()), _ptr(w.contiguous()), rows, n,
                                           eps, _ptr(q), _ptr(d)), "op_rmsnorm_quantize")
    return q, d


def op_gemm(xq, xd, wq, wd, K: int, dots: bool = False):
    import torch
    M, N = xq.shape[0], wq.shape[0]
    nb = (K + 31) // 32
    y = torch.zeros((M, N), dtype=torch.float32, device=xq.device)
    dd = torch.zeros((M, N, nb), dtype=torch.int32, device=xq.device) if dots else None
    check(lib().minfer_op_gemm(_ptr(xq), _ptr(xd), M, _ptr(wq), _ptr(wd), N, K, _ptr(y), _ptr(dd)),
          "op_gemm")
    return (y, dd) if dots else y


def op_gemm_noalloc(xq, xd, wq, wd, K: int):
    """minfer_op_gemm without device allocation (fixed 32 MiB scratch in the
    library).  The call runs on the library's own stream, so the operands
    must be complete when it starts: the current stream is synchronized
    first."""
    import torch
    M, N = xq.shape[0], wq.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=xq.device)
    torch.cuda.current_stream(xq.device).synchronize()
    check(lib().minfer_op_gemm_noalloc(_ptr(xq), _ptr(xd), M, _ptr(wq), _ptr(wd), N, K, _ptr(y)),
          "op_gemm_noalloc")
    return y


def op_gemm_swiglu(xq, xd, gq, gd, uq, ud, F: int, K: int):
    import torch
    M = xq.shape[0]
    nbF = (F + 31) // 32
    sq = torch.zeros((M, nbF * 32), dtype=torch.int8, device=xq.device)
    sd = torch.zeros((M, nbF), dtype=torch.int16, device=xq.device)
    check(lib().minfer_op_gemm_swiglu(_ptr(xq), _ptr(xd), M, _ptr(gq), _ptr(gd), _ptr(uq), _ptr(ud),
                                      F, K, _ptr(sq), _ptr(sd)), "op_gemm_swiglu")
    return sq, sd


def op_attention(q, pos, K, V, nh: int, nkv: int, hd: int):
    import torch
    o = torch.zeros_like(q)
    check(lib().minfer_op_attention(_ptr(q), _ptr(pos), q.shape[0], _ptr(K), _ptr(V), K.shape[0],
                                    nh, nkv, hd, _ptr(o)), "op_attention")
    return o


def op_qknorm_rope_store(qkv, bias, qnorm, knorm, eps: float, pos, nh: int, nkv: int, hd: int,
                         theta: float, K, V):
    """RoPE/store with the Qwen3 per-head Q/K RMSNorm first (bias may be None)."""
    import torch
    nt = qkv.shape[0]
    q_out = torch.zeros((nt, nh * hd), dtype=torch.float32, device=qkv.device)
    check(lib().minfer_op_qknorm_rope_store(_ptr(qkv), _ptr(bias), _ptr(qnorm), _ptr(knorm), eps,
                                            _ptr(pos), nt, nh, nkv, hd, theta, K.shape[0],
                                            _ptr(q_out), _ptr(K), _ptr(V)), "op_qknorm_rope_store")
    return q_out


def op_rope_store(qkv, bias, pos, nh: int, nkv: int, hd: int, theta: float, K, V):
    import torch
    nt = qkv.shape[0]
    q_out = torch.zeros((nt, nh * hd), dtype=torch.float32, device=qkv.device)
    check(lib().minfer_op_rope_store(_ptr(qkv), _ptr(bias), _ptr(pos), nt, nh, nkv, hd, theta,
                                     K.shape[0], _ptr(q_out), _ptr(K), _ptr(V)), "op_rope_store")
    return q_out


# ------------------------------------------------------------------ batch operators
# One step of a batch of requests over a paged K/V cache: torch tensors (CUDA)
# in and out.  The calls enqueue on the current stream of the tensors' device,
# wait for nothing, and can be captured into a CUDA graph.  `out`, `workspace`
# and the like may be given, so that a loop allocates nothing; `status` is an
# int32 tensor of one element in which the kernels leave the first error code
# they find (check_status reads it).

def _torch_types():
    import torch
    return {torch.float32: MINFER_F32, torch.float16: MINFER_F16, torch.bfloat16: MINFER_BF16}


def _type_of(t, what: str) -> int:
    code = _torch_types().get(t.dtype)
    if code is None:
        raise MinferError(-5, f"{what}: {t.dtype} (float32, float16 or bfloat16 wanted)")
    return code


def _need(ok: bool, what: str, code: int = -1):
    if not ok:
        raise MinferError(code, what)


def _vector(t, dtype, n: int, device, what: str):
    """A contiguous tensor of one dimension, n elements (None: any number)."""
    _need(t.dtype == dtype and t.dim() == 1 and t.device == device and t.is_contiguous()
          and (n is None or t.shape[0] == n), f"{what}: {list(t.shape)} {t.dtype} on {t.device}")


class _on:
    """The tensors' device current during a call; .stream its current stream."""

    def __init__(self, device):
        import torch
        _need(device.type == "cuda", f"tensors on {device} (a CUDA device wanted)")
        self.guard = None
        if device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)
        self.device = device

    def __enter__(self):
        import torch
        if self.guard is not None:
            self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


class PagedCache:
    """A pool of K/V pages: k and v [n_pages, page_size, n_head_kv, head_dim], of
    one type and with the same strides (a permuted view whose last dimension is
    contiguous will do, e.g. of [n_pages, n_head_kv, page_size, head_dim])."""

    def __init__(self, k, v):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.device == v.device
              and k.stride() == v.stride() and k.stride(3) == 1,
              "PagedCache: k and v differ, or are not [pages][rows][heads][dims] with contiguous dims")
        self.k, self.v = k, v
        self.device = k.device
        n, rows, heads, dims = k.shape
        self.n_pages, self.page_size, self.n_head_kv, self.head_dim = n, rows, heads, dims
        self.dtype = k.dtype
        self.desc = PagedCacheDesc(k.data_ptr(), v.data_ptr(), _type_of(k, "PagedCache"), n, rows,
                                   heads, dims, k.stride(0), k.stride(1), k.stride(2))
        self.ptr = ctypes.addressof(self.desc)


class RopeTable:
    """Rotary positions of one head layout (host memory): rot_dim leading dims
    of a head (None: all), style "half" or "interleaved", scaling "none",
    "linear", "ntk" or "yarn"."""

    def __init__(self, head_dim: int, rot_dim: int | None = None, theta: float = 1.0e6,
                 style: str = "half", scaling: str = "none", factor: float = 1.0,
                 n_ctx_orig: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 attn_factor: float = 0.0):
        _need(style in ROPE_STYLES and scaling in ROPE_SCALINGS,
              f"RopeTable: style {style!r}, scaling {scaling!r}")
        spec = RopeSpec(head_dim, head_dim if rot_dim is None else rot_dim, ROPE_STYLES[style],
                        ROPE_SCALINGS[scaling], theta, factor, n_ctx_orig, beta_fast, beta_slow,
                        attn_factor)
        self.desc = RopeTableDesc()
        check(lib().minfer_rope_prepare(ctypes.byref(spec), ctypes.byref(self.desc)), "RopeTable")
        self.head_dim = head_dim
        self.ptr = ctypes.addressof(self.desc)


def check_status(status):
    """Raise the error that a batch operator left in `status`, if any (waits for
    the device)."""
    check(int(status.item()), "batch operator")


def op_page_tables(length, target, page_size: int, table, free, n_free, n_pages: int,
                   max_tokens: int, out=None, status=None):
    """Block tables and slot maps of a step (minfer_op_page_tables): requests
    holding `length` rows are to hold `target`.  int32 tensors; `table`
    [n_req][max_pages] and the stack `free` [n_pages] are updated in place.
    Returns (start [n_req + 1], pos [max_tokens], slot [max_tokens], n_free
    [1]), or fills `out`, four such tensors; the last may be n_free itself."""
    import torch
    i32, dev = torch.int32, length.device
    n = length.shape[0]
    _vector(length, i32, n, dev, "length")
    _vector(target, i32, n, dev, "target")
    _vector(free, i32, n_pages, dev, "free")
    _vector(n_free, i32, 1, dev, "n_free")
    _need(table.dtype == i32 and table.dim() == 2 and table.shape[0] == n and table.is_contiguous()
          and table.device == dev, "table: int32 [n_req][max_pages] wanted")
    with _on(dev) as stream:
        if out is None:
            out = (torch.empty(n + 1, dtype=i32, device=dev), torch.empty(max_tokens, dtype=i32, device=dev),
                   torch.empty(max_tokens, dtype=i32, device=dev), torch.empty(1, dtype=i32, device=dev))
        else:
            for t, m, what in zip(out, (n + 1, max_tokens, max_tokens, 1), ("start", "pos", "slot", "n_free")):
                _vector(t, i32, m, dev, what)
        if status is not None:
            _vector(status, i32, 1, dev, "status")
        start, pos, slot, left = out
        check(lib().minfer_op_page_tables(_ptr(length), _ptr(target), n, page_size, n_pages, _ptr(table),
                                          table.shape[1], _ptr(free), _ptr(n_free), _ptr(left), _ptr(start),
                                          _ptr(pos), _ptr(slot), max_tokens, _ptr(status), stream),
              "op_page_tables")
    return out


def op_rope_paged_store(qkv, rope: RopeTable, pos, slot, cache: PagedCache, n_head: int, bias=None,
                        q_norm=None, k_norm=None, eps: float = 1e-6, out=None, status=None):
    """Bias, QK-norm and RoPE of fused Q|K|V rows [n][(n_head + 2 n_head_kv) *
    head_dim] (float32 or the cache's type), K and V stored at `slot`
    (minfer_op_rope_paged_store).  Returns the rotated Q [n][n_head*head_dim]
    in the cache's type; rows with a negative slot are skipped (without `out`
    they are zero)."""
    import torch
    dev, f32 = qkv.device, torch.float32
    n, hd = qkv.shape[0], cache.head_dim
    width = (n_head + 2 * cache.n_head_kv) * hd
    _need(qkv.dim() == 2 and qkv.shape[1] == width and qkv.stride(1) == 1 and cache.device == dev,
          f"qkv: {list(qkv.shape)} on {dev} (rows of {width} on {cache.device} wanted)")
    _vector(pos, torch.int32, n, dev, "pos")
    _vector(slot, torch.int32, n, dev, "slot")
    for t, m, what in ((bias, width, "bias"), (q_norm, hd, "q_norm"), (k_norm, hd, "k_norm")):
        if t is not None:
            _vector(t, f32, m, dev, what)
    if status is not None:
        _vector(status, torch.int32, 1, dev, "status")
    with _on(dev) as stream:
        if out is None:
            out = torch.zeros((n, n_head * hd), dtype=cache.dtype, device=dev)
        else:
            _need(out.dim() == 2 and out.shape[0] == n and out.shape[1] == n_head * hd and out.stride(1) == 1
                  and out.dtype == cache.dtype and out.device == dev, "out: the cache's type, [n][n_head*head_dim]")
        check(lib().minfer_op_rope_paged_store(_ptr(qkv), _type_of(qkv, "qkv"), qkv.stride(0), _ptr(bias),
                                               _ptr(q_norm), _ptr(k_norm), eps, rope.ptr, _ptr(pos), _ptr(slot),
                                               n, n_head, cache.ptr, _ptr(out), out.stride(0), _ptr(status),
                                               stream), "op_rope_paged_store")
    return out


def op_paged_attention_workspace(cache: PagedCache, n_req: int, n_head: int):
    """A workspace for op_paged_attention calls of up to n_req requests, one call
    at a time."""
    import torch
    n = ctypes.c_int64()
    with _on(cache.device):
        check(lib().minfer_op_paged_attention_workspace(n_req, n_head, cache.ptr, ctypes.byref(n)),
              "op_paged_attention_workspace")
        return torch.empty(n.value, dtype=torch.uint8, device=cache.device)


def op_paged_attention(q, cache: PagedCache, table, length, n_head: int, scale: float | None = None,
                       out=None, lse=None, workspace=None, status=None):
    """Attention of one new token per request over its pages
    (minfer_op_paged_attention): q [n_req][n_head*head_dim] in the cache's type,
    table int32 [n_req][max_pages], length int32 [n_req] rows to attend to, the
    new one included.  Returns o like q; `lse` (float32 [n_req][n_head]), when
    given, gets ln sum exp(scale q.k)."""
    import torch
    dev, n, width = q.device, q.shape[0], n_head * cache.head_dim
    _need(q.dim() == 2 and q.shape[1] == width and q.stride(1) == 1 and q.dtype == cache.dtype
          and cache.device == dev, f"q: {list(q.shape)} {q.dtype} on {dev} (rows of {width} {cache.dtype} on {cache.device} wanted)")
    _need(table.dtype == torch.int32 and table.dim() == 2 and table.shape[0] == n and table.stride(1) == 1
          and table.device == dev, "table: int32 [n_req][max_pages] wanted")
    _vector(length, torch.int32, n, dev, "length")
    if lse is not None:
        _need(lse.dtype == torch.float32 and lse.dim() == 2 and lse.shape[0] == n and lse.shape[1] == n_head
              and lse.is_contiguous() and lse.device == dev, "lse: float32 [n_req][n_head] wanted")
    if status is not None:
        _vector(status, torch.int32, 1, dev, "status")
    with _on(dev) as stream:
        if out is None:
            out = torch.empty((n, width), dtype=q.dtype, device=dev)
        else:
            _need(out.dim() == 2 and out.shape == q.shape and out.stride(1) == 1 and out.dtype == q.dtype
                  and out.device == dev, "out: like q")
        if workspace is None:
            workspace = op_paged_attention_workspace(cache, n, n_head)
        else:
            _vector(workspace, torch.uint8, None, dev, "workspace")
        check(lib().minfer_op_paged_attention(_ptr(q), q.stride(0), cache.ptr, _ptr(table), table.stride(0),
                                              table.shape[1], _ptr(length), n, n_head, scale or 0.0, _ptr(out),
                                              out.stride(0), _ptr(lse), _ptr(workspace), workspace.shape[0],
                                              _ptr(status), stream), "op_paged_attention")
    return out


def op_token_logprobs_workspace(logits, k: int):
    """A workspace for op_token_logprobs calls on logits of this shape, one call
    at a time."""
    import torch
    n = ctypes.c_int64()
    with _on(logits.device):
        check(lib().minfer_op_token_logprobs_workspace(logits.shape[0], logits.shape[1], k, ctypes.byref(n)),
              "op_token_logprobs_workspace")
        return torch.empty(n.value, dtype=torch.uint8, device=logits.device)


def op_token_logprobs(logits, ids=None, k: int = 0, out=None, workspace=None, status=None):
    """Log probabilities of the tokens `ids` (int32 [rows], negative: skip the
    row; or None) under logits [rows][vocab] (float32, float16 or bfloat16, any
    row stride), the rows' entropy and k largest with their log probabilities
    (minfer_op_token_logprobs).  Returns (logprob, entropy, top_ids,
    top_logprobs), or fills `out`, four such tensors; logprob is None without
    ids."""
    import torch
    dev, f32 = logits.device, torch.float32
    _need(logits.dim() == 2 and (logits.stride(1) == 1 or logits.shape[1] == 1), "logits: [rows][vocab] wanted")
    rows, vocab = logits.shape
    if ids is not None:
        _vector(ids, torch.int32, rows, dev, "ids")
    if status is not None:
        _vector(status, torch.int32, 1, dev, "status")
    with _on(dev) as stream:
        if out is None:
            out = (None if ids is None else torch.empty(rows, dtype=f32, device=dev),
                   torch.empty(rows, dtype=f32, device=dev),
                   torch.empty((rows, k), dtype=torch.int32, device=dev), torch.empty((rows, k), dtype=f32, device=dev))
        else:
            for t, dtype, what in ((out[0], f32, "logprob"), (out[1], f32, "entropy")):
                if t is not None:
                    _vector(t, dtype, rows, dev, what)
            for t, dtype, what in ((out[2], torch.int32, "top_ids"), (out[3], f32, "top_logprobs")):
                _need(k == 0 or (t.dtype == dtype and t.dim() == 2 and t.shape[0] == rows and t.shape[1] == k
                                 and t.is_contiguous() and t.device == dev), f"{what}: [rows][k] wanted")
        if workspace is None:
            workspace = op_token_logprobs_workspace(logits, k)
        else:
            _vector(workspace, torch.uint8, None, dev, "workspace")
        check(lib().minfer_op_token_logprobs(_ptr(logits), _type_of(logits, "logits"), rows, vocab,
                                             logits.stride(0), _ptr(ids), k, _ptr(out[0]), _ptr(out[1]),
                                             _ptr(out[2]), _ptr(out[3]), _ptr(workspace), workspace.shape[0],
                                             _ptr(status), stream), "op_token_logprobs")
    return out
