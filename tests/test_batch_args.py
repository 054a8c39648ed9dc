"""The batch operators without a GPU: every refusal that needs no device, the
binding's own checks, and the rotary turns against their formulas.

The pointers given here are never dereferenced: the library checks its host
arguments before it enqueues anything, and without a device a call that passes
the checks returns MINFER_ERR_CUDA."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

ARG, SHAPE, CUDA, TOO_LARGE = -1, -5, -6, -10
PTR = 0x10000  # 16-byte aligned, never read
F32, F16, BF16 = 0, 1, 30


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


TABLES = dict(len=PTR, target=PTR, n_req=4, page_size=16, n_pages=64, table=PTR, max_pages=8, free=PTR,
              n_free=PTR, n_free_out=PTR, start=PTR, pos=PTR, slot=PTR, max_tokens=32, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(max_tokens=0, pos=None, slot=None), CUDA), (dict(n_req=16384), CUDA),
    (dict(len=None), ARG), (dict(target=None), ARG), (dict(table=None), ARG), (dict(free=None), ARG),
    (dict(n_free=None), ARG), (dict(n_free_out=None), ARG), (dict(start=None), ARG), (dict(pos=None), ARG),
    (dict(slot=None), ARG), (dict(n_req=0), ARG), (dict(n_req=-1), ARG), (dict(page_size=0), ARG),
    (dict(n_pages=0), ARG), (dict(max_pages=0), ARG), (dict(max_tokens=-1), ARG),
    (dict(n_req=16385), TOO_LARGE), (dict(max_pages=2 ** 20, n_req=2048), TOO_LARGE),
    (dict(max_pages=2 ** 20, page_size=2048, n_req=1), TOO_LARGE), (dict(n_pages=2 ** 27, page_size=16), TOO_LARGE),
    (dict(max_tokens=2 ** 30), TOO_LARGE)])
def test_page_tables_arguments(qp, change, code):
    assert _call(qp.lib().minfer_op_page_tables, TABLES, **change) == code


def _cache(qp, **change):
    a = dict(k=PTR, v=PTR, type=BF16, n_pages=8, page_size=16, n_head_kv=2, head_dim=64, page_stride=2048,
             row_stride=128, head_stride=64)
    assert not set(change) - set(a)
    return qp.PagedCacheDesc(*{**a, **change}.values())


BAD_CACHES = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(n_pages=0), ARG), (dict(page_size=0), ARG), (dict(n_head_kv=0), ARG),
    (dict(type=8), SHAPE), (dict(type=2), SHAPE), (dict(head_dim=96), SHAPE), (dict(head_dim=32), SHAPE),
    (dict(k=PTR + 2), ARG), (dict(v=PTR + 8), ARG), (dict(page_stride=2044), ARG), (dict(row_stride=132), ARG),
    (dict(head_stride=68), ARG), (dict(page_stride=-2048), ARG), (dict(type=F32, head_stride=66), ARG),
    (dict(n_pages=2 ** 28), TOO_LARGE)]


def _rope(qp, head_dim=64, **change):
    a = dict(head_dim=head_dim, rot_dim=head_dim, style=0, scaling=0, theta=1e6, factor=1.0, n_ctx_orig=0, beta_fast=0.0,
             beta_slow=0.0, attn_factor=0.0)
    assert not set(change) - set(a)
    spec, out = qp.RopeSpec(*{**a, **change}.values()), qp.RopeTableDesc()
    return qp.lib().minfer_rope_prepare(ctypes.byref(spec), ctypes.byref(out)), out


def _store_args(qp, cache=None, rope=None):
    cache = cache if cache is not None else _cache(qp)
    rope = rope if rope is not None else _rope(qp)[1]
    keep = (cache, rope)
    return keep, dict(qkv=PTR, type=BF16, row_stride=512, bias=None, qnorm=None, knorm=None, eps=1e-6, rope=ctypes.addressof(rope), pos=PTR,
                      slot=PTR, n_tokens=3, n_head=4, cache=ctypes.addressof(cache), q_out=PTR, q_stride=256, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(type=F32), CUDA), (dict(bias=PTR, qnorm=PTR, knorm=PTR), CUDA), (dict(row_stride=520), CUDA),
    (dict(qkv=None), ARG), (dict(rope=None), ARG), (dict(pos=None), ARG), (dict(slot=None), ARG), (dict(cache=None), ARG),
    (dict(q_out=None), ARG), (dict(n_tokens=0), ARG), (dict(n_head=0), ARG), (dict(n_head=3), ARG), (dict(qnorm=PTR), ARG),
    (dict(knorm=PTR), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(type=F16), SHAPE), (dict(type=8), SHAPE),
    (dict(qkv=PTR + 2), ARG), (dict(q_out=PTR + 4), ARG), (dict(bias=PTR + 4), ARG), (dict(row_stride=516), ARG),
    (dict(row_stride=504), ARG), (dict(q_stride=248), ARG), (dict(q_stride=260), ARG),
    (dict(n_head=65536, row_stride=2 ** 23, q_stride=2 ** 23), TOO_LARGE)])
def test_rope_store_arguments(qp, change, code):
    keep, args = _store_args(qp)
    assert _call(qp.lib().minfer_op_rope_paged_store, args, **change) == code


def test_rope_store_refuses_another_head_dim(qp):
    keep, args = _store_args(qp, rope=_rope(qp, head_dim=128)[1])
    assert _call(qp.lib().minfer_op_rope_paged_store, args) == SHAPE


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_caches_are_checked(qp, change, code):
    cache = _cache(qp, **change)
    keep, args = _store_args(qp, cache=cache)
    assert _call(qp.lib().minfer_op_rope_paged_store, args) == code
    n = ctypes.c_int64()
    assert qp.lib().minfer_op_paged_attention_workspace(3, 4, ctypes.addressof(cache), ctypes.byref(n)) == code
    assert _call(qp.lib().minfer_op_paged_attention, _attention_args(qp, cache)[1]) == code


def _attention_args(qp, cache=None):
    cache = cache if cache is not None else _cache(qp)
    return cache, dict(q=PTR, q_stride=256, cache=ctypes.addressof(cache), table=PTR, table_stride=8, max_pages=8, len=PTR, n_req=3,
                       n_head=4, scale=0.0, o=PTR, o_stride=256, lse=None, ws=PTR, ws_bytes=2 ** 40, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(scale=0.5, lse=PTR), CUDA), (dict(n_req=1, q_stride=0, o_stride=0, table_stride=0), CUDA),
    (dict(q=None), ARG), (dict(cache=None), ARG), (dict(table=None), ARG), (dict(len=None), ARG), (dict(o=None), ARG), (dict(ws=None), ARG),
    (dict(n_req=0), ARG), (dict(n_head=0), ARG), (dict(n_head=5), ARG), (dict(max_pages=0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=math.inf), ARG), (dict(scale=math.nan), ARG), (dict(q=PTR + 2), ARG), (dict(o=PTR + 8), ARG), (dict(ws=PTR + 8), ARG),
    (dict(q_stride=252), ARG), (dict(q_stride=248), ARG), (dict(o_stride=248), ARG), (dict(table_stride=7), ARG),
    (dict(max_pages=2 ** 28, table_stride=2 ** 28), TOO_LARGE), (dict(n_head=65536 * 2), TOO_LARGE)])
def test_attention_arguments(qp, change, code):
    keep, args = _attention_args(qp)
    if "n_head" in change and change["n_head"] > 5:
        change = {**change, "q_stride": change["n_head"] * 64, "o_stride": change["n_head"] * 64}
    assert _call(qp.lib().minfer_op_paged_attention, args, **change) == code


LOGPROBS = dict(logits=PTR, type=F32, rows=3, vocab=100, row_stride=101, ids=PTR, k=5, logprob=PTR, entropy=PTR, top_ids=PTR,
                top_logprobs=PTR, ws=PTR, ws_bytes=2 ** 40, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(), CUDA), (dict(logits=PTR + 4), CUDA), (dict(ids=None, logprob=None), CUDA), (dict(k=0, top_ids=None, top_logprobs=None), CUDA),
    (dict(entropy=None), CUDA), (dict(rows=1, row_stride=0), CUDA),
    (dict(logits=None), ARG), (dict(rows=0), ARG), (dict(vocab=0), ARG), (dict(k=-1), ARG), (dict(k=33), ARG), (dict(vocab=4), ARG),
    (dict(row_stride=99), ARG), (dict(rows=1, row_stride=-1), ARG), (dict(logprob=None), ARG), (dict(top_ids=None), ARG), (dict(top_logprobs=None), ARG), (dict(ws=None), ARG),
    (dict(ws=PTR + 4), ARG), (dict(logits=PTR + 2), ARG), (dict(type=F16, logits=PTR + 1), ARG), (dict(type=8), SHAPE),
    (dict(vocab=2 ** 31, row_stride=2 ** 31), TOO_LARGE), (dict(rows=2 ** 31), TOO_LARGE)])
def test_logprobs_arguments(qp, change, code):
    assert _call(qp.lib().minfer_op_token_logprobs, LOGPROBS, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=7), SHAPE), (dict(rot_dim=66), SHAPE), (dict(head_dim=96, rot_dim=64), SHAPE),
    (dict(style=2), ARG), (dict(style=-1), ARG), (dict(scaling=4), ARG), (dict(theta=1.0), ARG), (dict(theta=math.nan), ARG),
    (dict(theta=math.inf), ARG), (dict(factor=0.0), ARG), (dict(factor=math.inf), ARG), (dict(scaling=3, factor=4.0), ARG),
    (dict(attn_factor=math.nan), ARG), (dict(beta_fast=-1.0), ARG), (dict(beta_slow=math.inf), ARG)])
def test_rope_specs_are_checked(qp, change, code):
    assert _rope(qp, **change)[0] == code


@pytest.mark.parametrize("rot", [2, 24, 64])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rope_turns(qp, rot, scaling):
    """Each turn is f_i / 2 pi of the scaling's formula to 53 bits."""
    theta, s, ctx = 1e4, 3.5, 4096
    t = qp.RopeTable(64, rot, theta, "half", scaling, s, ctx)
    want_scale = 1.0
    if scaling == "ntk" and rot > 2:
        theta *= s ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= s
        if scaling == "yarn":
            d = [rot * math.log(ctx / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32, 1)]
            low, high = max(math.floor(d[0]), 0), min(math.ceil(d[1]), rot - 1)
            g = min(max((i - low) / max(high - low, 1e-3), 0), 1)
            f = f / s * g + f * (1 - g)
            want_scale = 0.1 * math.log(s) + 1
        got = t.desc.turn[i] / 2.0 ** 64
        assert abs(got - f / (2 * math.pi)) <= 8 * 2.0 ** -53 * f, (i, got)
    assert all(t.desc.turn[i] == 0 for i in range(rot // 2, 64))
    assert t.desc.mscale == np.float32(want_scale)
    assert qp.RopeTable(64, rot, theta, "half", scaling, s, ctx, attn_factor=1.25).desc.mscale == 1.25


def test_binding_refuses_host_tensors_and_wrong_shapes(qp):
    k = torch.zeros(4, 16, 2, 64)
    cache = qp.PagedCache(k, k.clone())
    i32 = torch.int32
    n = torch.zeros(2, dtype=i32)
    with pytest.raises(qp.MinferError, match="CUDA device wanted"):
        qp.op_paged_attention(torch.zeros(2, 256), cache, torch.zeros(2, 3, dtype=i32), n, 4)
    with pytest.raises(qp.MinferError, match="CUDA device wanted"):
        qp.op_token_logprobs(torch.zeros(2, 50), n, 3)
    with pytest.raises(qp.MinferError, match="CUDA device wanted"):
        qp.op_rope_paged_store(torch.zeros(2, 512), qp.RopeTable(64), n, n, cache, 4)
    with pytest.raises(qp.MinferError, match="CUDA device wanted"):
        qp.op_page_tables(n, n, 16, torch.zeros(2, 3, dtype=i32), torch.zeros(4, dtype=i32), torch.zeros(1, dtype=i32), 4, 8)
    with pytest.raises(qp.MinferError, match="rows of 256"):
        qp.op_paged_attention(torch.zeros(2, 320), cache, torch.zeros(2, 3, dtype=i32), n, 4)
    with pytest.raises(qp.MinferError, match="length"):
        qp.op_paged_attention(torch.zeros(2, 256), cache, torch.zeros(2, 3, dtype=i32), n.long(), 4)
    with pytest.raises(qp.MinferError, match="table"):
        qp.op_paged_attention(torch.zeros(2, 256), cache, torch.zeros(3, 3, dtype=i32), n, 4)
    with pytest.raises(qp.MinferError, match="contiguous dims"):
        qp.PagedCache(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(qp.MinferError, match="differ"):
        qp.PagedCache(k, k.half())
    with pytest.raises(qp.MinferError, match="float64"):
        qp.PagedCache(k.double(), k.double())
    with pytest.raises(qp.MinferError, match="scaling"):
        qp.RopeTable(64, scaling="cubic")
    with pytest.raises(qp.MinferError, match="ERR_SHAPE"):
        qp.RopeTable(64, 65)


# strides between things of which there is one: never used, whatever they are
@pytest.mark.parametrize("change", [dict(n_pages=1, page_stride=2044), dict(n_pages=1, page_stride=-3), dict(page_size=1, row_stride=132),
                                    dict(n_head_kv=1, head_stride=68), dict(n_head_kv=1, head_stride=-1),
                                    dict(n_pages=1, page_size=1, n_head_kv=1, page_stride=1, row_stride=3, head_stride=5)])
def test_unused_cache_strides(qp, change):
    cache = _cache(qp, **change)
    keep, args = _store_args(qp, cache=cache)
    assert _call(qp.lib().minfer_op_rope_paged_store, args) == CUDA
    assert _call(qp.lib().minfer_op_paged_attention, _attention_args(qp, cache)[1]) == CUDA


@pytest.mark.parametrize("change", [dict(row_stride=515), dict(q_stride=3), dict(row_stride=1, q_stride=-7)])
def test_unused_row_strides(qp, change):
    keep, args = _store_args(qp)
    assert _call(qp.lib().minfer_op_rope_paged_store, args, n_tokens=1, **change) == CUDA
    assert _call(qp.lib().minfer_op_rope_paged_store, args, n_tokens=2, **change) == ARG
    change = {{"row_stride": "o_stride"}.get(name, name): x for name, x in change.items()}
    keep, args = _attention_args(qp)
    assert _call(qp.lib().minfer_op_paged_attention, args, n_req=1, **change) == CUDA
    assert _call(qp.lib().minfer_op_paged_attention, args, n_req=2, **change) == ARG


def test_the_binding_compares_used_strides_only(qp):
    a = torch.zeros(1, 16, 1, 64)
    b = torch.zeros(3, 16, 1, 64)[1:2].as_strided((1, 16, 1, 64), (7, 64, 9, 1))
    assert qp.PagedCache(a, b).desc.n_pages == 1
    with pytest.raises(qp.MinferError, match="differ"):
        qp.PagedCache(torch.zeros(2, 16, 2, 64), torch.zeros(2, 2, 16, 64).transpose(1, 2))


def test_a_workspace_is_claimed_once(qp):
    w = qp.Workspace(64, "cpu")
    assert w.op is None
    w.claim("op_paged_attention")
    with pytest.raises(qp.MinferError, match="got one of op_paged_attention"):
        w.claim("op_token_logprobs")


@pytest.mark.parametrize("change", [dict(scaling=1, factor=1e-320), dict(scaling=2, factor=1e-200, rot_dim=4),
                                    dict(scaling=3, factor=1e-320, n_ctx_orig=4096), dict(scaling=1, factor=5e-324)])
def test_rope_frequencies_past_the_range_of_a_double(qp, change):
    """An infinite number of turns per position has no fraction: refused, and the table is left as it was."""
    assert _rope(qp, **change)[0] == ARG
    assert not any(bytes(_rope(qp, **change)[1]))


def test_sizes_past_31_bits_are_refused(qp):
    """The library's ints would drop their upper bits: 2^32 + 1 pages are not one page."""
    one = torch.zeros(1, 1, 1, 64)
    for shape in ((2 ** 32 + 1, 1, 1, 64), (1, 2 ** 32 + 16, 1, 64), (1, 1, 2 ** 31, 64)):
        with pytest.raises(qp.MinferError, match="TOO_LARGE"):
            qp.PagedCache(one.expand(shape), one.expand(shape))
    n = torch.zeros(2, dtype=torch.int32)
    for page_size, max_tokens in ((2 ** 32 + 16, 8), (16, 2 ** 32 + 8)):
        with pytest.raises(qp.MinferError, match="TOO_LARGE"):
            qp.op_page_tables(n, n, page_size, torch.zeros(2, 3, dtype=torch.int32), n.new_zeros(4), n[:1], 4, max_tokens)
    with pytest.raises(qp.MinferError, match="k: 4294967301"):
        qp.op_token_logprobs(torch.zeros(2, 50), n, 2 ** 32 + 5)


@pytest.mark.parametrize("style", [2, 7, -1])
@pytest.mark.parametrize("rot", [24, 64])
def test_rope_store_refuses_a_table_of_an_unknown_style(qp, style, rot):
    """A table that minfer_rope_prepare did not fill: its style decides what shared memory the launch asks for."""
    table = _rope(qp, rot_dim=rot)[1]
    table.style = style
    keep, args = _store_args(qp, rope=table)
    assert _call(qp.lib().minfer_op_rope_paged_store, args) == SHAPE
