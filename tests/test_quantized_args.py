"""The operators of a quantized paged cache and sampling without a GPU: every refusal that needs no device, and the binding's own checks.

The pointers given here are never dereferenced: the library checks its host arguments before it enqueues anything, and
without a device a call that passes the checks returns MINFER_ERR_CUDA."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

ARG, SHAPE, CUDA, TOO_LARGE = -1, -5, -6, -10
PTR = 0x10000  # 16-byte aligned, never read
F32, F16, BF16 = 0, 1, 30
I32 = torch.int32


@pytest.fixture(scope="module")
def qp():
    from quantized_transformer_prefill_gb300 import build
    build.build()
    import quantized_transformer_prefill_gb300 as qp
    qp.lib()
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: a call that passes the checks would run")
    return qp


def _call(fn, args, **change):
    assert not set(change) - set(args), change
    return fn(*{**args, **change}.values())


def _cache(qp, **change):
    a = dict(k=PTR, v=PTR, k_scale=PTR, v_scale=PTR, n_pages=8, page_size=16, n_head_kv=2, head_dim=64, page_stride=2048, row_stride=128,
             head_stride=64, scale_page_stride=64, scale_row_stride=4, scale_head_stride=2)
    assert not set(change) - set(a)
    return qp.PagedCacheQ8Desc(*{**a, **change}.values())


def _rope(qp, head_dim=64):
    spec, out = qp.RopeSpec(head_dim, head_dim, 0, 0, 1e6, 1.0, 0, 0.0, 0.0, 0.0), qp.RopeTableDesc()
    assert qp.lib().minfer_rope_prepare(ctypes.byref(spec), ctypes.byref(out)) == 0
    return out


def _store(qp, cache=None, rope=None):
    cache, rope = cache or _cache(qp), rope or _rope(qp)
    return (cache, rope), dict(qkv=PTR, type=BF16, row_stride=512, bias=None, qnorm=None, knorm=None, eps=1e-6, rope=ctypes.addressof(rope),
                               pos=PTR, slot=PTR, n_tokens=3, n_head=4, cache=ctypes.addressof(cache), q_out=PTR, q_type=BF16, q_stride=256,
                               status=None, stream=None)


def _read(qp, cache=None):
    cache = cache or _cache(qp)
    return cache, dict(cache=ctypes.addressof(cache), slot=PTR, n_rows=3, type=F32, k=PTR, v=PTR, out_stride=128, status=None, stream=None)


def _attention(qp, cache=None):
    cache = cache or _cache(qp)
    return cache, dict(q=PTR, type=BF16, q_stride=256, cache=ctypes.addressof(cache), table=PTR, table_stride=8, max_pages=8, len=PTR, n_req=3,
                       n_head=4, scale=0.0, o=PTR, o_stride=256, lse=None, ws=PTR, ws_bytes=2 ** 40, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(type=F32), CUDA), (dict(type=F32, q_type=F32), CUDA), (dict(type=F16, q_type=F16), CUDA),
    (dict(type=F32, q_type=F16), CUDA), (dict(bias=PTR, qnorm=PTR, knorm=PTR), CUDA), (dict(row_stride=520), CUDA),
    (dict(n_tokens=1, row_stride=3, q_stride=-1), CUDA),
    (dict(qkv=None), ARG), (dict(rope=None), ARG), (dict(pos=None), ARG), (dict(slot=None), ARG), (dict(cache=None), ARG),
    (dict(q_out=None), ARG), (dict(n_tokens=0), ARG), (dict(n_head=0), ARG), (dict(n_head=3), ARG), (dict(qnorm=PTR), ARG),
    (dict(knorm=PTR), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(type=F16), SHAPE), (dict(type=8), SHAPE),
    (dict(q_type=8), SHAPE), (dict(q_type=F32), SHAPE), (dict(qkv=PTR + 2), ARG), (dict(q_out=PTR + 4), ARG), (dict(bias=PTR + 4), ARG),
    (dict(row_stride=516), ARG), (dict(row_stride=504), ARG), (dict(q_stride=248), ARG), (dict(q_stride=260), ARG),
    (dict(n_head=65536, row_stride=2 ** 23, q_stride=2 ** 23), TOO_LARGE)])
def test_store_arguments(qp, change, code):
    keep, args = _store(qp)
    assert _call(qp.lib().minfer_op_rope_paged_store_q8, args, **change) == code


def test_store_refuses_other_rope_tables(qp):
    for rope in (_rope(qp, 128), _rope(qp)):
        if rope.head_dim == 64:
            rope.style = 2
        keep, args = _store(qp, rope=rope)
        assert _call(qp.lib().minfer_op_rope_paged_store_q8, args) == SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(k=None), CUDA), (dict(v=None), CUDA), (dict(type=F16), CUDA), (dict(type=BF16, out_stride=136), CUDA),
    (dict(n_rows=1, out_stride=0), CUDA),
    (dict(cache=None), ARG), (dict(slot=None), ARG), (dict(k=None, v=None), ARG), (dict(n_rows=0), ARG), (dict(n_rows=-4), ARG),
    (dict(type=8), SHAPE), (dict(k=PTR + 4), ARG), (dict(v=PTR + 8), ARG), (dict(out_stride=130), ARG), (dict(out_stride=124), ARG),
    (dict(type=F16, out_stride=132), ARG)])
def test_read_arguments(qp, change, code):
    keep, args = _read(qp)
    assert _call(qp.lib().minfer_op_paged_read_q8, args, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(type=F32), CUDA), (dict(type=F16, scale=0.5, lse=PTR), CUDA), (dict(n_req=1, q_stride=0, o_stride=0, table_stride=0), CUDA),
    (dict(q=None), ARG), (dict(cache=None), ARG), (dict(table=None), ARG), (dict(len=None), ARG), (dict(o=None), ARG), (dict(ws=None), ARG),
    (dict(n_req=0), ARG), (dict(n_head=0), ARG), (dict(n_head=5), ARG), (dict(max_pages=0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG), (dict(q=PTR + 2), ARG), (dict(o=PTR + 8), ARG), (dict(ws=PTR + 8), ARG),
    (dict(q_stride=252), ARG), (dict(type=F32, q_stride=258), ARG), (dict(q_stride=248), ARG), (dict(o_stride=248), ARG),
    (dict(table_stride=7), ARG), (dict(type=8), SHAPE), (dict(max_pages=2 ** 28, table_stride=2 ** 28), TOO_LARGE),
    (dict(n_head=131072, q_stride=2 ** 23, o_stride=2 ** 23), TOO_LARGE)])
def test_attention_arguments(qp, change, code):
    keep, args = _attention(qp)
    assert _call(qp.lib().minfer_op_paged_attention_q8, args, **change) == code


BAD_CACHES = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG), (dict(n_pages=0), ARG),
    (dict(page_size=0), ARG), (dict(n_head_kv=0), ARG), (dict(head_dim=96), SHAPE), (dict(head_dim=32), SHAPE), (dict(k=PTR + 8), ARG),
    (dict(v=PTR + 1), ARG), (dict(k_scale=PTR + 2), ARG), (dict(v_scale=PTR + 2), ARG), (dict(page_stride=2040), ARG), (dict(row_stride=120), ARG),
    (dict(head_stride=72), ARG), (dict(page_stride=-2048), ARG), (dict(scale_page_stride=65), ARG), (dict(scale_row_stride=5), ARG),
    (dict(scale_head_stride=3), ARG), (dict(scale_head_stride=-2), ARG), (dict(head_dim=128, scale_head_stride=2), ARG),
    (dict(head_dim=128, k_scale=PTR + 4, scale_head_stride=4), ARG), (dict(n_pages=2 ** 28), TOO_LARGE)]
FINE_CACHES = [dict(n_pages=1, page_stride=3, scale_page_stride=1), dict(page_size=1, row_stride=-5, scale_row_stride=7),
               dict(n_head_kv=1, head_stride=1, scale_head_stride=-1), dict(k_scale=PTR + 4, v_scale=PTR + 4)]


@pytest.mark.parametrize("change,code", BAD_CACHES + [(c, CUDA) for c in FINE_CACHES])
def test_caches_are_checked(qp, change, code):
    """Strides that nothing steps over are not."""
    cache, L, n = _cache(qp, **change), qp.lib(), ctypes.c_int64()
    assert _call(L.minfer_op_paged_read_q8, _read(qp, cache)[1], out_stride=256) == code
    assert L.minfer_op_paged_attention_q8_workspace(3, 4, ctypes.addressof(cache), ctypes.byref(n)) == code
    assert _call(L.minfer_op_paged_attention_q8, _attention(qp, cache)[1], q_stride=512, o_stride=512) == code
    rope = _rope(qp, 128 if change.get("head_dim") == 128 else 64)
    keep, args = _store(qp, cache, rope)
    assert _call(L.minfer_op_rope_paged_store_q8, args, row_stride=1024, q_stride=512) == code


def test_the_binding_refuses(qp):
    codes, scales = torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.zeros(4, 16, 2, 2, dtype=torch.float16)
    cache = qp.PagedCacheQ8(codes, codes.clone(), scales, scales.clone())
    n, table = torch.zeros(2, dtype=I32), torch.zeros(2, 3, dtype=I32)
    refused = lambda match: pytest.raises(qp.MinferError, match=match)  # noqa: E731
    with refused("CUDA device wanted"):
        qp.op_paged_attention_q8(torch.zeros(2, 256), cache, table, n, 4)
    with refused("CUDA device wanted"):
        qp.op_rope_paged_store_q8(torch.zeros(2, 512), qp.RopeTable(64), n, n, cache, 4)
    with refused("CUDA device wanted"):
        qp.op_paged_read_q8(cache, n)
    with refused("rows of 256"):
        qp.op_paged_attention_q8(torch.zeros(2, 320), cache, table, n, 4)
    with refused("length"):
        qp.op_paged_attention_q8(torch.zeros(2, 256), cache, table, n.long(), 4)
    with refused("table"):
        qp.op_paged_attention_q8(torch.zeros(2, 256), cache, torch.zeros(3, 3, dtype=I32), n, 4)
    with refused("slot"):
        qp.op_paged_read_q8(cache, n.long())
    with refused("int8"):
        qp.PagedCacheQ8(codes.half(), codes.half(), scales, scales)
    with refused("float16"):
        qp.PagedCacheQ8(codes, codes, scales.float(), scales.float())
    with refused("contiguous dims"):
        qp.PagedCacheQ8(codes.transpose(2, 3), codes.transpose(2, 3), scales, scales)
    with refused("same strides"):
        qp.PagedCacheQ8(codes, torch.zeros(4, 2, 16, 64, dtype=torch.int8).transpose(1, 2), scales, scales)
    with refused("same strides"):
        qp.PagedCacheQ8(codes, codes, scales, scales[:3])
    with refused("scale per 32"):
        qp.PagedCacheQ8(codes, codes, scales[..., :1], scales[..., :1])
    with refused("scale per 32"):
        qp.PagedCacheQ8(codes[..., :48], codes[..., :48], scales[..., :1], scales[..., :1])
    one = torch.zeros(1, 1, 1, 64, dtype=torch.int8)
    two = torch.zeros(1, 1, 1, 2, dtype=torch.float16)
    with refused("TOO_LARGE"):
        qp.PagedCacheQ8(one.expand(2 ** 32 + 1, 1, 1, 64), one.expand(2 ** 32 + 1, 1, 1, 64), two.expand(2 ** 32 + 1, 1, 1, 2), two.expand(2 ** 32 + 1, 1, 1, 2))


def test_caches_of_the_other_kind_are_refused(qp):
    """Their descriptions have other layouts: a call that read one as the other would take scales' addresses for sizes."""
    codes, scales = torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.zeros(4, 16, 2, 2, dtype=torch.float16)
    q8, plain = qp.PagedCacheQ8(codes, codes, scales, scales), qp.PagedCache(codes.half(), codes.half())
    n, table = torch.zeros(2, dtype=I32), torch.zeros(2, 3, dtype=I32)
    for call in (lambda: qp.op_rope_paged_store_q8(torch.zeros(2, 512), qp.RopeTable(64), n, n, plain, 4), lambda: qp.op_paged_read_q8(plain, n),
                 lambda: qp.op_paged_attention_q8(torch.zeros(2, 256), plain, table, n, 4), lambda: qp.op_paged_attention_q8_workspace(plain, 2, 4)):
        with pytest.raises(qp.MinferError, match="PagedCacheQ8 wanted"):
            call()
    for call in (lambda: qp.op_rope_paged_store(torch.zeros(2, 512), qp.RopeTable(64), n, n, q8, 4), lambda: qp.op_paged_attention(torch.zeros(2, 256), q8, table, n, 4),
                 lambda: qp.op_paged_attention_workspace(q8, 2, 4)):
        with pytest.raises((qp.MinferError, AttributeError)):
            call()


def test_operators_over_float_pages_refuse_a_quantized_cache_by_its_class(qp):
    """Not by what it happens to lack: one with a `dtype`, which the other checks would let through, is refused as well."""
    codes, scales = torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.zeros(4, 16, 2, 2, dtype=torch.float16)
    n, table = torch.zeros(2, dtype=I32), torch.zeros(2, 3, dtype=I32)

    class Named(qp.PagedCacheQ8):
        dtype = torch.float16

    for q8 in (qp.PagedCacheQ8(codes, codes, scales, scales), Named(codes, codes, scales, scales)):
        for call in (lambda: qp.op_rope_paged_store(torch.zeros(2, 512, dtype=torch.float16), qp.RopeTable(64), n, n, q8, 4),  # noqa: B023
                     lambda: qp.op_paged_attention(torch.zeros(2, 256, dtype=torch.float16), q8, table, n, 4),  # noqa: B023
                     lambda: qp.op_paged_attention_workspace(q8, 2, 4)):  # noqa: B023
            with pytest.raises(qp.MinferError, match="cache: a PagedCache wanted"):
                call()
        # (what is made for it takes a class derived from it)
        with pytest.raises(qp.MinferError, match="CUDA device wanted"):
            qp.op_paged_attention_q8(torch.zeros(2, 256), q8, table, n, 4)
        with pytest.raises(qp.MinferError, match="CUDA device wanted"):
            qp.op_paged_read_q8(q8, n)


SAMPLE = dict(logits=PTR, type=F32, rows=3, vocab=100, row_stride=101, u=PTR, temperature=PTR, top_k=PTR, top_p=PTR, min_p=PTR, first=0,
              token=PTR, logprob=PTR, ws=PTR, ws_bytes=2 ** 40, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(logits=PTR + 4), CUDA), (dict(type=BF16, logits=PTR + 2), CUDA), (dict(temperature=None, top_k=None, top_p=None, min_p=None), CUDA),
    (dict(logprob=None), CUDA), (dict(rows=1, row_stride=0), CUDA), (dict(first=1), CUDA),
    (dict(logits=None), ARG), (dict(u=None), ARG), (dict(token=None), ARG), (dict(rows=0), ARG), (dict(rows=-1), ARG), (dict(vocab=0), ARG),
    (dict(row_stride=99), ARG), (dict(rows=1, row_stride=-1), ARG), (dict(logits=PTR + 2), ARG), (dict(type=F16, logits=PTR + 1), ARG),
    (dict(ws=PTR + 8), ARG), (dict(ws=None), CUDA),
    (dict(type=8), SHAPE), (dict(vocab=2 ** 31, row_stride=2 ** 31), TOO_LARGE), (dict(rows=2 ** 31), TOO_LARGE)])
def test_sample_arguments(qp, change, code):
    assert _call(qp.lib().minfer_op_sample, SAMPLE, **change) == code


def test_the_binding_refuses_samples(qp):
    x, u, i32 = torch.zeros(2, 50), torch.zeros(2), torch.zeros(2, dtype=I32)
    refused = lambda match: pytest.raises(qp.MinferError, match=match)  # noqa: E731
    with refused("CUDA device wanted"):
        qp.op_sample(x, u, u, i32, u, u)
    for args, match in (((x[0], u), "rows"), ((x.t(), u), "contiguous rows"), ((x, u[:1]), "u:"), ((x, u.double()), "u:"), ((x, u, i32), "temperature"),
                        ((x, u, u, u), "top_k"), ((x, u, u, i32.long()), "top_k"), ((x, u, u, i32, i32), "top_p"), ((x, u, u, i32, u, u[:1]), "min_p")):
        with refused(match):
            qp.op_sample(*args)
    with refused("status"):
        qp.op_sample(x, u, status=u)
