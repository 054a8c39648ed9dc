"""The batch operators of the library for torch tensors: one step of a batch of
requests over a paged K/V cache.

The calls enqueue on the current stream of the tensors' device, wait for
nothing, and can be captured into a CUDA graph.  `out`, `lse`, `workspace` and
the like may be given, so that a loop allocates nothing; `status` is an int32
tensor of one element in which the kernels leave the first error code they find
(check_status reads it).  A step without rows (no requests, no tokens) is done
without a kernel.

A small call takes less time on the GPU than its arguments take to be checked
in Python, so the checks are written out, with the attributes that are cheapest
to read (a vector is any contiguous tensor of so many elements), and an error
message is put together only when one fails (measured on the host of a GB300: a
helper per tensor with its message 1.2 us, written out 0.3 us).
"""
from __future__ import annotations

import ctypes

import torch

from . import (MINFER_BF16, MINFER_F16, MINFER_F32, ROPE_SCALINGS, ROPE_STYLES, MinferError,
               PagedCacheDesc, RopeSpec, RopeTableDesc, check, lib)

_TYPES = {torch.float32: MINFER_F32, torch.float16: MINFER_F16, torch.bfloat16: MINFER_BF16}
_I32, _F32 = torch.int32, torch.float32
_ERR_ARG, _ERR_SHAPE, _ERR_TOO_LARGE = -1, -5, -10
_INT_MAX = 2 ** 31 - 1

_L = lib()
_page_tables = _L.minfer_op_page_tables
_rope_paged_store = _L.minfer_op_rope_paged_store
_paged_attention = _L.minfer_op_paged_attention
_token_logprobs = _L.minfer_op_token_logprobs

# The raw handle of a device's current stream and the current device's index:
# torch's own accessors take 2 us for the first and 0.3 us for the second.
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(what: str, *tensors, code: int = _ERR_ARG):
    seen = ", ".join("none" if t is None else f"{list(t.shape)} {t.dtype} on {t.device}" for t in tensors)
    raise MinferError(code, f"{what}{': got ' + seen if seen else ''}")


def _type_of(t, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        _refuse(f"{what}: float32, float16 or bfloat16 wanted", t, code=_ERR_SHAPE)
    return code


class PagedCache:
    """A pool of K/V pages: k and v [n_pages, page_size, n_head_kv, head_dim], of
    one type and with the same strides (a permuted view whose last dimension is
    contiguous will do, e.g. of [n_pages, n_head_kv, page_size, head_dim]; the
    stride of a dimension of one does not matter)."""

    def __init__(self, k, v):
        if not (k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.device == v.device
                and all(a == b for a, b, n in zip(k.stride(), v.stride(), k.shape) if n > 1) and k.stride(3) == 1):
            _refuse("PagedCache: k and v differ, or are not [pages][rows][heads][dims] with contiguous dims", k, v)
        if max(k.shape) > _INT_MAX:
            _refuse("PagedCache: sizes below 2^31 wanted", k, code=_ERR_TOO_LARGE)
        self.k, self.v = k, v
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        self.n_pages, self.page_size, self.n_head_kv, self.head_dim = k.shape
        self.desc = PagedCacheDesc(k.data_ptr(), v.data_ptr(), _type_of(k, "PagedCache"), *k.shape,
                                   *k.stride()[:3])
        self.ptr = ctypes.addressof(self.desc)


class RopeTable:
    """Rotary positions of one head layout (host memory): rot_dim leading dims
    of a head (None: all), style "half" or "interleaved", scaling "none",
    "linear", "ntk" or "yarn"."""

    def __init__(self, head_dim: int, rot_dim: int | None = None, theta: float = 1.0e6,
                 style: str = "half", scaling: str = "none", factor: float = 1.0,
                 n_ctx_orig: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 attn_factor: float = 0.0):
        if style not in ROPE_STYLES or scaling not in ROPE_SCALINGS:
            _refuse(f"RopeTable: style {style!r}, scaling {scaling!r}")
        spec = RopeSpec(head_dim, head_dim if rot_dim is None else rot_dim, ROPE_STYLES[style],
                        ROPE_SCALINGS[scaling], theta, factor, n_ctx_orig, beta_fast, beta_slow,
                        attn_factor)
        self.desc = RopeTableDesc()
        check(_L.minfer_rope_prepare(ctypes.byref(spec), ctypes.byref(self.desc)), "RopeTable")
        self.head_dim = head_dim
        self.ptr = ctypes.addressof(self.desc)


class Workspace:
    """Device memory of one operator's calls, zero-filled once; one call at a
    time may use it (calls on one stream follow one another).  It belongs to the
    operator that uses it first (`op`): another one would find its counters
    overwritten."""

    def __init__(self, nbytes: int, device, op: str | None = None):
        self.buffer = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.nbytes, self.index, self.ptr, self.op = nbytes, self.buffer.get_device(), self.buffer.data_ptr(), op

    def claim(self, op: str):
        if self.op is not None:
            _refuse(f"workspace: one of {op} wanted, got one of {self.op}")
        self.op = op


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
    [1]), or fills `out`, four such tensors; the last may be n_free itself.
    After a refused step the returned n_free is the old one, and that of `out`
    is as it was."""
    dev = length.get_device()
    n = length.numel()
    if not (length.dtype is _I32 and length.is_contiguous()):
        _refuse("length: int32 [n_req] wanted", length)
    if not (target.dtype is _I32 and target.numel() == n and target.is_contiguous() and target.get_device() == dev):
        _refuse("target: int32 [n_req] wanted", target)
    shape = table.shape
    if not (table.dtype is _I32 and len(shape) == 2 and shape[0] == n and table.is_contiguous()
            and table.get_device() == dev):
        _refuse("table: int32 [n_req][max_pages] wanted", table)
    if not (free.dtype is _I32 and free.numel() == n_pages and free.is_contiguous() and free.get_device() == dev):
        _refuse("free: int32 [n_pages] wanted", free)
    if not (n_free.dtype is _I32 and n_free.numel() == 1 and n_free.get_device() == dev):
        _refuse("n_free: int32 [1] wanted", n_free)
    if page_size > _INT_MAX or max_tokens > _INT_MAX:
        _refuse(f"page_size {page_size}, max_tokens {max_tokens}", code=_ERR_TOO_LARGE)
    if status is not None and not (status.dtype is _I32 and status.numel() == 1 and status.get_device() == dev):
        _refuse("status: int32 [1] wanted", status)
    if dev < 0:
        _refuse("a CUDA device wanted", length)
    if dev != _current():
        with torch.cuda.device(dev):
            return op_page_tables(length, target, page_size, table, free, n_free, n_pages, max_tokens, out, status)
    if out is None:
        start, pos, slot = (torch.empty(m, dtype=_I32, device=length.device) for m in (n + 1, max_tokens, max_tokens))
        left = n_free.reshape(1).clone()  # what a refused step leaves
        out = start, pos, slot, left
    else:
        start, pos, slot, left = out
        if not (start.dtype is _I32 and start.numel() == n + 1 and start.is_contiguous() and start.get_device() == dev):
            _refuse("start: int32 [n_req + 1] wanted", start)
        if not (pos.dtype is _I32 and pos.numel() == max_tokens and pos.is_contiguous() and pos.get_device() == dev):
            _refuse("pos: int32 [max_tokens] wanted", pos)
        if not (slot.dtype is _I32 and slot.numel() == max_tokens and slot.is_contiguous() and slot.get_device() == dev):
            _refuse("slot: int32 [max_tokens] wanted", slot)
        if not (left.dtype is _I32 and left.numel() == 1 and left.get_device() == dev):
            _refuse("n_free of out: int32 [1] wanted", left)
    if n == 0:
        start.zero_(), pos.fill_(-1), slot.fill_(-1), left.reshape(1).copy_(n_free.reshape(1))
        return out
    rc = _page_tables(length.data_ptr(), target.data_ptr(), n, page_size, n_pages, table.data_ptr(), shape[1],
                      free.data_ptr(), n_free.data_ptr(), left.data_ptr(), start.data_ptr(), pos.data_ptr(),
                      slot.data_ptr(), max_tokens, None if status is None else status.data_ptr(), _stream_of(dev))
    if rc:
        raise MinferError(rc, "op_page_tables")
    return out


def op_rope_paged_store(qkv, rope: RopeTable, pos, slot, cache: PagedCache, n_head: int, bias=None,
                        q_norm=None, k_norm=None, eps: float = 1e-6, out=None, status=None):
    """Bias, QK-norm and RoPE of fused Q|K|V rows [n][(n_head + 2 n_head_kv) *
    head_dim] (float32 or the cache's type), K and V stored at `slot`
    (minfer_op_rope_paged_store).  Returns the rotated Q [n][n_head*head_dim]
    in the cache's type; rows with a negative slot are skipped (without `out`
    they are zero)."""
    dev, hd = qkv.get_device(), cache.head_dim
    width = (n_head + 2 * cache.n_head_kv) * hd
    shape = qkv.shape
    if not (len(shape) == 2 and shape[1] == width and dev == cache.index):
        _refuse(f"qkv: rows of {width} on the cache's device wanted", qkv)
    n = shape[0]
    row_stride, one = qkv.stride()
    if one != 1:
        _refuse("qkv: contiguous rows wanted", qkv)
    if not (pos.dtype is _I32 and pos.numel() == n and pos.is_contiguous() and pos.get_device() == dev):
        _refuse("pos: int32 [n] wanted", pos)
    if not (slot.dtype is _I32 and slot.numel() == n and slot.is_contiguous() and slot.get_device() == dev):
        _refuse("slot: int32 [n] wanted", slot)
    if bias is not None and not (bias.dtype is _F32 and bias.numel() == width and bias.is_contiguous()
                                 and bias.get_device() == dev):
        _refuse(f"bias: float32 [{width}] wanted", bias)
    for w in (q_norm, k_norm):
        if w is not None and not (w.dtype is _F32 and w.numel() == hd and w.is_contiguous() and w.get_device() == dev):
            _refuse(f"q_norm, k_norm: float32 [{hd}] wanted", w)
    if status is not None and not (status.dtype is _I32 and status.numel() == 1 and status.get_device() == dev):
        _refuse("status: int32 [1] wanted", status)
    if dev < 0:
        _refuse("a CUDA device wanted", qkv)
    if dev != _current():
        with torch.cuda.device(dev):
            return op_rope_paged_store(qkv, rope, pos, slot, cache, n_head, bias, q_norm, k_norm, eps, out, status)
    if out is None:
        out = torch.zeros((n, n_head * hd), dtype=cache.dtype, device=qkv.device)
        q_stride = n_head * hd
    else:
        if not (out.dtype is cache.dtype and out.shape == (n, n_head * hd) and out.get_device() == dev):
            _refuse("out: [n][n_head*head_dim] of the cache's type wanted", out)
        q_stride, one = out.stride()
        if one != 1:
            _refuse("out: contiguous rows wanted", out)
    if n == 0:
        return out
    rc = _rope_paged_store(qkv.data_ptr(), _type_of(qkv, "qkv"), row_stride, None if bias is None else bias.data_ptr(),
                           None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                           eps, rope.ptr, pos.data_ptr(), slot.data_ptr(), n, n_head, cache.ptr, out.data_ptr(), q_stride,
                           None if status is None else status.data_ptr(), _stream_of(dev))
    if rc:
        raise MinferError(rc, "op_rope_paged_store")
    return out


def op_paged_attention_workspace(cache: PagedCache, n_req: int, n_head: int) -> Workspace:
    """A workspace for op_paged_attention calls of up to n_req requests, one call
    at a time."""
    n = ctypes.c_int64()
    with torch.cuda.device(cache.device):
        check(_L.minfer_op_paged_attention_workspace(n_req, n_head, cache.ptr, ctypes.byref(n)),
              "op_paged_attention_workspace")
        return Workspace(n.value, cache.device, "op_paged_attention")


def op_paged_attention(q, cache: PagedCache, table, length, n_head: int, scale: float | None = None,
                       out=None, lse=None, workspace: Workspace | None = None, status=None):
    """Attention of one new token per request over its pages
    (minfer_op_paged_attention): q [n_req][n_head*head_dim] in the cache's type,
    table int32 [n_req][max_pages], length int32 [n_req] rows to attend to, the
    new one included, scale None or 0 for 1 / sqrt(head_dim).  Returns o like q; `lse` (float32 [n_req][n_head]), when
    given, gets ln sum exp(scale q.k).  Rows of refused requests are not written
    (without `out` they are zero)."""
    dev, width = q.get_device(), n_head * cache.head_dim
    shape = q.shape
    if not (q.dtype is cache.dtype and len(shape) == 2 and shape[1] == width and dev == cache.index):
        _refuse(f"q: rows of {width} {cache.dtype} on {cache.device} wanted", q)
    n = shape[0]
    q_stride, one = q.stride()
    if one != 1:
        _refuse("q: contiguous rows wanted", q)
    pages = table.shape
    if not (table.dtype is _I32 and len(pages) == 2 and pages[0] == n and table.get_device() == dev):
        _refuse("table: int32 [n_req][max_pages] wanted", table)
    table_stride, one = table.stride()
    max_pages = pages[1]
    if one != 1 and max_pages > 1:
        _refuse("table: contiguous rows wanted", table)
    if not (length.dtype is _I32 and length.numel() == n and length.is_contiguous() and length.get_device() == dev):
        _refuse("length: int32 [n_req] wanted", length)
    if lse is not None and not (lse.dtype is _F32 and lse.shape == (n, n_head) and lse.is_contiguous()
                                and lse.get_device() == dev):
        _refuse("lse: float32 [n_req][n_head] wanted", lse)
    if status is not None and not (status.dtype is _I32 and status.numel() == 1 and status.get_device() == dev):
        _refuse("status: int32 [1] wanted", status)
    if dev < 0:
        _refuse("a CUDA device wanted", q)
    if dev != _current():
        with torch.cuda.device(dev):
            return op_paged_attention(q, cache, table, length, n_head, scale, out, lse, workspace, status)
    if out is None:
        out = torch.zeros((n, width), dtype=q.dtype, device=q.device)
        o_stride = width
    else:
        if not (out.dtype is cache.dtype and out.shape == shape and out.get_device() == dev):
            _refuse("out: like q wanted", out)
        o_stride, one = out.stride()
        if one != 1:
            _refuse("out: contiguous rows wanted", out)
    if n == 0:
        return out
    if workspace is None:
        workspace = op_paged_attention_workspace(cache, n, n_head)
    elif workspace.index != dev:
        _refuse("workspace: on the tensors' device wanted", workspace.buffer)
    elif workspace.op != "op_paged_attention":
        workspace.claim("op_paged_attention")
    rc = _paged_attention(q.data_ptr(), q_stride, cache.ptr, table.data_ptr(), table_stride, max_pages,
                          length.data_ptr(), n, n_head, scale or 0.0, out.data_ptr(), o_stride,
                          None if lse is None else lse.data_ptr(), workspace.ptr, workspace.nbytes,
                          None if status is None else status.data_ptr(), _stream_of(dev))
    if rc:
        raise MinferError(rc, "op_paged_attention")
    return out


def op_token_logprobs_workspace(logits, k: int) -> Workspace:
    """A workspace for op_token_logprobs calls on logits of this shape, one call
    at a time."""
    n = ctypes.c_int64()
    with torch.cuda.device(logits.device):
        check(_L.minfer_op_token_logprobs_workspace(logits.shape[0], logits.shape[1], k, ctypes.byref(n)),
              "op_token_logprobs_workspace")
        return Workspace(n.value, logits.device, "op_token_logprobs")


def op_token_logprobs(logits, ids=None, k: int = 0, out=None, workspace: Workspace | None = None, status=None):
    """Log probabilities of the tokens `ids` (int32 [rows], negative: skip the
    row; or None) under logits [rows][vocab] (float32, float16 or bfloat16, rows
    of any distance that do not overlap), the rows' entropy and k largest with their log probabilities
    (minfer_op_token_logprobs).  Returns (logprob, entropy, top_ids,
    top_logprobs), or fills `out`, four such tensors (logprob without ids,
    entropy, and the last two with k = 0 may be None); logprob is None without
    ids.  Skipped and refused rows are not written (without `out` they are zero,
    with top_ids of -1)."""
    dev, shape = logits.get_device(), logits.shape
    if len(shape) != 2:
        _refuse("logits: [rows][vocab] wanted", logits)
    rows, vocab = shape
    row_stride, one = logits.stride()
    if one != 1 and vocab > 1:
        _refuse("logits: contiguous rows wanted", logits)
    if ids is not None and not (ids.dtype is _I32 and ids.numel() == rows and ids.is_contiguous()
                                and ids.get_device() == dev):
        _refuse("ids: int32 [rows] wanted", ids)
    if status is not None and not (status.dtype is _I32 and status.numel() == 1 and status.get_device() == dev):
        _refuse("status: int32 [1] wanted", status)
    if k < 0 or k > 32:
        _refuse(f"k: {k}")
    if dev < 0:
        _refuse("a CUDA device wanted", logits)
    if dev != _current():
        with torch.cuda.device(dev):
            return op_token_logprobs(logits, ids, k, out, workspace, status)
    if out is None:
        if ids is None:  # every row is written
            logprob, new = None, torch.empty(rows * (1 + k), dtype=_F32, device=logits.device)
            top_ids = torch.empty((rows, k), dtype=_I32, device=logits.device)
        else:
            new = torch.zeros(rows * (2 + k), dtype=_F32, device=logits.device)
            top_ids = torch.full((rows, k), -1, dtype=_I32, device=logits.device)
            logprob, new = new[:rows], new[rows:]
        entropy, top_logprobs = new[:rows], new[rows:].view(rows, k)
        out = logprob, entropy, top_ids, top_logprobs
    else:
        logprob, entropy, top_ids, top_logprobs = out
        if logprob is not None and not (logprob.dtype is _F32 and logprob.numel() == rows and logprob.is_contiguous()
                                        and logprob.get_device() == dev):
            _refuse("logprob: float32 [rows] wanted", logprob)
        if entropy is not None and not (entropy.dtype is _F32 and entropy.numel() == rows and entropy.is_contiguous()
                                        and entropy.get_device() == dev):
            _refuse("entropy: float32 [rows] wanted", entropy)
        if k > 0:
            if top_ids is None or not (top_ids.dtype is _I32 and top_ids.shape == (rows, k) and top_ids.is_contiguous()
                                       and top_ids.get_device() == dev):
                _refuse("top_ids: int32 [rows][k] wanted", top_ids)
            if top_logprobs is None or not (top_logprobs.dtype is _F32 and top_logprobs.shape == (rows, k)
                                            and top_logprobs.is_contiguous() and top_logprobs.get_device() == dev):
                _refuse("top_logprobs: float32 [rows][k] wanted", top_logprobs)
    if rows == 0:
        return out
    if workspace is None:
        workspace = op_token_logprobs_workspace(logits, k)
    elif workspace.index != dev:
        _refuse("workspace: on the tensors' device wanted", workspace.buffer)
    elif workspace.op != "op_token_logprobs":
        workspace.claim("op_token_logprobs")
    rc = _token_logprobs(logits.data_ptr(), _type_of(logits, "logits"), rows, vocab, row_stride,
                         None if ids is None else ids.data_ptr(), k, None if logprob is None else logprob.data_ptr(),
                         None if entropy is None else entropy.data_ptr(), top_ids.data_ptr() if k else None,
                         top_logprobs.data_ptr() if k else None, workspace.ptr, workspace.nbytes,
                         None if status is None else status.data_ptr(), _stream_of(dev))
    if rc:
        raise MinferError(rc, "op_token_logprobs")
    return out
