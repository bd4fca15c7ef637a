"""The cache, attention and verification entry points refuse bad arguments on
the host, before anything is launched (CPU only)."""
import ctypes

import pytest

A = 0x10000          # aligned fake address: never dereferenced
NULL = None


@pytest.fixture(scope="module")
def rq():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_linear_layers_gb300 as rq
    return rq


def cache(rq, **over):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, pages=4, page_size=64, kv_heads=4, head_dim=128,
             format=0)
    f.update(over)
    return ctypes.byref(rq._KVCacheStruct(**f))


def params(rq, **over):
    f = dict(q_weight=A, k_weight=A, cos_table=A, sin_table=A, positions=16, q_heads=28,
             kv_heads=4, head_dim=128, rotary_dim=128, interleaved=0, eps=1e-6)
    f.update(over)
    return ctypes.byref(rq._QKParamsStruct(**f))


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
             (dict(v_scale=None), 1), (dict(format=2), 3), (dict(format=-1), 3),
             (dict(page_size=0), 2), (dict(page_size=48), 2), (dict(page_size=8), 2),
             (dict(page_size=512), 2), (dict(head_dim=96), 2), (dict(head_dim=0), 2),
             (dict(kv_heads=0), 2), (dict(pages=0), 2), (dict(pages=1 << 30), 2),
             (dict(k=A + 8), 2), (dict(v=A + 1), 2), (dict(k_scale=A + 4), 2),
             (dict(v_scale=A + 8), 2)]


@pytest.mark.parametrize("over,status", BAD_CACHE)
def test_bad_caches(rq, over, status):
    lib, c = rq.lib(), cache(rq, **over)
    assert lib.rq_kv_write(c, 0, A, 512, A, 512, A, 1, NULL) == status
    assert lib.rq_kv_read(c, 0, A, A, A, 1, NULL) == status
    assert lib.rq_qkv_to_cache(params(rq), 0, A, 3584, A, 512, A, 512, A, A, c, A, 1,
                               NULL) == status
    assert lib.rq_cache_attention(ctypes.c_void_p(A), c, 0, A, 3584, A, 1, 1, 28, A, 4, A, NULL,
                                  0.1, NULL) == status


def test_null_cache_and_params(rq):
    lib = rq.lib()
    assert lib.rq_kv_write(NULL, 0, A, 512, A, 512, A, 1, NULL) == 1
    assert lib.rq_kv_read(NULL, 0, A, A, A, 1, NULL) == 1
    assert lib.rq_qkv_to_cache(NULL, 0, A, 3584, A, 512, A, 512, A, A, cache(rq), A, 1, NULL) == 1
    assert lib.rq_qk_norm_rope(NULL, 0, A, 3584, A, 512, A, A, A, 1, NULL) == 1
    assert lib.rq_cache_attention(NULL, cache(rq), 0, A, 3584, A, 1, 1, 28, A, 4, A, NULL, 0.1,
                                  NULL) == 1


@pytest.mark.parametrize("over,status", [
    (dict(head_dim=80), 2), (dict(rotary_dim=136), 2), (dict(rotary_dim=24), 2),
    (dict(rotary_dim=-16), 2), (dict(cos_table=None), 1), (dict(sin_table=None), 1),
    (dict(positions=0), 2), (dict(cos_table=A + 4), 2), (dict(q_weight=A + 4), 2),
    (dict(k_weight=A + 8), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(q_heads=0), 2), (dict(kv_heads=0), 2)])
def test_bad_params(rq, over, status):
    lib, p = rq.lib(), params(rq, **over)
    assert lib.rq_qk_norm_rope(p, 0, A, 1 << 16, A, 1 << 16, A, A, A, 1, NULL) == status
    assert lib.rq_qkv_to_cache(p, 0, A, 1 << 16, A, 1 << 16, A, 1 << 16, A, A, cache(rq), A, 1,
                               NULL) == status


def test_bad_rows(rq):
    lib, p, c = rq.lib(), params(rq), cache(rq)
    nr = lib.rq_qk_norm_rope
    assert nr(p, 0, A, 3584, A, 512, NULL, A, A, 1, NULL) == 1        # positions wanted
    assert nr(p, 0, A, 3584, A, 512, A, NULL, A, 1, NULL) == 1        # q without its output
    assert nr(p, 0, NULL, 0, A, 512, A, A, A, 1, NULL) == 1
    assert nr(p, 0, NULL, 0, NULL, 0, A, NULL, NULL, 1, NULL) == 1    # nothing to do
    assert nr(p, 3, A, 3584, A, 512, A, A, A, 1, NULL) == 3           # dtype
    assert nr(p, 0, A + 4, 3584, A, 512, A, A, A, 1, NULL) == 2
    assert nr(p, 0, A, 3583, A, 512, A, A, A, 1, NULL) == 2           # heads overlap
    assert nr(p, 0, A, 3586, A, 512, A, A, A, 1, NULL) == 2           # stride not 16 bytes
    assert nr(p, 1, A, 3588, A, 512, A, A, A, 1, NULL) == 2
    assert nr(p, 0, A, 3584, A, 511, A, A, A, 1, NULL) == 2
    assert nr(p, 0, A, 3584, A, 512, A + 2, A, A, 1, NULL) == 2
    assert nr(p, 0, A, 3584, A, 512, A, A + 8, A, 1, NULL) == 2
    assert nr(p, 0, A, 3584, A, 512, A, A, A, -1, NULL) == 2
    assert nr(p, 0, A, 3584, A, 512, A, A, A, 0, NULL) == 0           # nothing to do
    tc = lib.rq_qkv_to_cache
    assert tc(p, 0, A, 3584, A, 512, NULL, 512, A, A, c, A, 1, NULL) == 1
    assert tc(p, 0, A, 3584, A, 512, A, 512, A, A, c, NULL, 1, NULL) == 1
    assert tc(p, 0, A, 3584, A, 512, A, 512, A, NULL, c, A, 1, NULL) == 1
    assert tc(p, 0, A, 3584, A, 512, A, 512, A, A, c, A + 4, 1, NULL) == 2
    assert tc(p, 0, A, 3584, A, 512, A, 512, A, A, cache(rq, kv_heads=2), A, 1, NULL) == 2
    assert tc(p, 0, A, 3584, A, 512, A, 512, A, A, cache(rq, head_dim=64), A, 1, NULL) == 2
    assert tc(p, 0, A, 3584, A, 512, A, 512, A, A, c, A, 0, NULL) == 0
    kw = lib.rq_kv_write
    assert kw(c, 7, A, 512, A, 512, A, 1, NULL) == 3
    assert kw(c, 0, NULL, 512, A, 512, A, 1, NULL) == 1
    assert kw(c, 0, A, 512, A, 508, A, 1, NULL) == 2
    assert kw(c, 0, A, 512, A + 4, 512, A, 1, NULL) == 2
    assert kw(c, 0, A, 512, A, 512, A, 0, NULL) == 0
    kr = lib.rq_kv_read
    assert kr(c, 0, NULL, A, A, 1, NULL) == 1
    assert kr(c, 0, A, NULL, A, 1, NULL) == 1
    assert kr(c, 5, A, A, A, 1, NULL) == 3
    assert kr(c, 0, A, A + 8, A, 1, NULL) == 2
    assert kr(c, 0, A, A, A, 0, NULL) == 0


def test_bad_attention(rq):
    lib, c = rq.lib(), cache(rq)
    ctx = ctypes.c_void_p(A)        # not dereferenced: the checks come first

    def call(dtype=0, q=A, stride=3584, out=A, batch=1, new=1, heads=28, table=A, pages=4,
             length=A, tree=NULL, scale=0.1):
        return lib.rq_cache_attention(ctx, c, dtype, q, stride, out, batch, new, heads, table,
                                      pages, length, tree, scale, NULL)

    for name in ("q", "out", "table", "length"):
        assert call(**{name: NULL}) == 1
    assert call(dtype=3) == 3
    for over in (dict(batch=-1), dict(new=0), dict(heads=0), dict(heads=30, stride=3840),
                 dict(pages=0), dict(tree=A, new=65), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=float("nan")), dict(scale=float("inf")), dict(q=A + 4),
                 dict(stride=3580), dict(stride=3586), dict(out=A + 8), dict(table=A + 2),
                 dict(length=A + 1), dict(tree=A + 4)):
        assert call(**over) == 2, over
    assert call(batch=0) == 0


def test_bad_verification(rq):
    lib = rq.lib()
    chain, tree = lib.rq_verify_chain, lib.rq_verify_tree
    assert chain(NULL, A, A, A, A, A, 1, 1, 10, NULL) == 1
    assert chain(A, NULL, A, A, A, A, 1, 1, 10, NULL) == 1
    assert chain(A, A, A, NULL, A, A, 1, 1, 10, NULL) == 1
    assert chain(A, A, A, A, NULL, A, 1, 1, 10, NULL) == 1
    assert chain(A, A, A, A, A, NULL, 1, 1, 10, NULL) == 1
    for b, n, v in ((-1, 1, 10), (1, -1, 10), (1, 1, 0), (1, 1, (1 << 20) + 1)):
        assert chain(A, A, A, A, A, A, b, n, v, NULL) == 2
        assert tree(A, A, A, A, A, A, A, b, n, v, NULL) == 2
    assert chain(A, A + 2, A, A, A, A, 1, 1, 10, NULL) == 2
    assert chain(A, A, A + 1, A, A, A, 1, 1, 10, NULL) == 2
    assert chain(A, A, A, A, A, A, 0, 1, 10, NULL) == 0
    assert tree(A, NULL, A, A, A, A, A, 1, 1, 10, NULL) == 1
    assert tree(A, A, A, A, A, A, NULL, 1, 1, 10, NULL) == 1
    assert tree(A, A, A, A, A, A, A, 1, 1025, 10, NULL) == 2
    assert tree(A, A + 2, A, A, A, A, A, 1, 1, 10, NULL) == 2
    assert tree(A, A, A, A, A, A, A, 0, 1, 10, NULL) == 0


def test_binding_refuses_tensors_that_are_not_rows(rq):
    import torch
    x = torch.zeros(6, 8, 64)
    assert rq._row_stride(x, 8, 64, None, "x") == 512
    assert rq._row_stride(x[::2], 8, 64, None, "x") == 1024
    assert rq._row_stride(x[:, 2:4], 2, 64, None, "x") == 512
    assert rq._row_stride(x[:1], 8, 64, None, "x") == 512
    assert rq._row_stride(x.view(6, 512), 8, 64, None, "x") == 512
    assert rq._row_stride(x.view(2, 3, 8, 64)[:, :, :2], 2, 64, None, "x") == 512
    for bad in (x.transpose(0, 1), x[..., ::2], x.view(2, 3, 8, 64)[:, :2], x[:, ::2]):
        with pytest.raises(rq.RqError):
            rq._row_stride(bad, bad.shape[-2], 64, None, "x")
    k = torch.zeros(2, 4, 16, 64, dtype=torch.int8)
    s = torch.zeros(2, 4, 16)
    rq.KVCache.from_tensors(k, k, s, s, format=rq.RQ_KV_I8)
    for args in ((k.transpose(1, 2), k, s, s), (k, k[:1], s, s), (k, k, s[..., :8], s),
                 (k, k, s, s.half()), (k.float(), k, s, s)):
        with pytest.raises(rq.RqError):
            rq.KVCache.from_tensors(*args, format=rq.RQ_KV_I8)
    with pytest.raises(rq.RqError):
        rq.QKParams(2, 1, 64, q_weight=torch.ones(32))
    with pytest.raises(rq.RqError):
        rq.QKParams(2, 1, 64, cos=torch.ones(8, 32), sin=torch.ones(8, 16))


def test_attention_counters_want_a_context(rq):
    assert rq.lib().rq_ctx_attention_launches(NULL, NULL, NULL) == 1


def test_binding_tells_tokens_from_a_single_head(rq):
    """[batch, tokens, head_dim] of one head: the second axis is tokens, not
    heads, and heads that are not as many as the call's are refused."""
    import torch
    x = torch.zeros(3, 5, 64)
    with pytest.raises(rq.RqError):      # batches lie further apart than tokens
        rq._row_stride(x[:, :4], 1, 64, None, "x")
    assert rq._row_stride(x[:, ::5], 1, 64, None, "x") == 320
    assert rq._row_stride(torch.zeros(3, 4, 96)[..., :64], 1, 64, None, "x") == 96
    assert rq._row_stride(torch.zeros(3, 4, 1, 96)[..., :64], 1, 64, None, "x") == 96
    assert rq._row_stride(torch.zeros(7, 96)[:, :64], 1, 64, None, "x") == 96
    y = torch.zeros(6, 8, 64)
    for bad, heads in ((y[::2], 4), (y[:, 1:4], 2), (torch.zeros(2, 512)[:, :64], 2)):
        with pytest.raises(rq.RqError):
            rq._row_stride(bad, heads, 64, None, "x")


def refused(rq, status, call, *args, **kw):
    with pytest.raises(rq.RqError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value


def small_cache(rq, **over):
    import torch
    k = torch.zeros(8, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(8, 2, 16)
    return rq.KVCache.from_tensors(k, k.clone(), s, s.clone(), **dict(dict(format=rq.RQ_KV_I8), **over))


class NoContext:
    """Stands for a Context where the binding refuses before the library."""
    _h = None


def test_binding_refuses_index_arrays_that_are_not_what_the_kernels_read(rq):
    import torch
    c, st = small_cache(rq), dict(stream=0)
    p = rq.QKParams(4, 2, 64, cos=torch.zeros(8, 32), sin=torch.zeros(8, 32))
    q, k, v = torch.zeros(4, 4, 64), torch.zeros(4, 2, 64), torch.zeros(4, 2, 64)
    pos, slot = torch.arange(4, dtype=torch.int32), torch.arange(4)
    for bad, status in ((pos.long(), 3), (torch.arange(8, dtype=torch.int32)[::2], 2)):
        refused(rq, status, rq.rq_qk_norm_rope, p, q, k, bad, q.clone(), k.clone(), 4, **st)
        refused(rq, status, rq.rq_qkv_to_cache, p, q, k, v, bad, q.clone(), c, slot, 4, **st)
    for bad, status in ((slot.int(), 3), (torch.arange(8)[::2], 2)):
        refused(rq, status, rq.rq_qkv_to_cache, p, q, k, v, pos, q.clone(), c, bad, 4, **st)
        refused(rq, status, rq.rq_kv_write, c, k, v, bad, 4, **st)
        refused(rq, status, rq.rq_kv_read, c, bad, k.clone(), v.clone(), 4, **st)

    attend = rq.Context.rq_cache_attention
    q4 = torch.zeros(2, 3, 4, 64)
    table = torch.zeros(2, 6, dtype=torch.int32)
    length = torch.zeros(2, dtype=torch.int32)
    tree = torch.zeros(2, 3, dtype=torch.int64)

    def call(table=table, length=length, tree=tree, **kw):
        attend(NoContext, c, q4, q4.clone(), table, length, 2, 3, 4, 0.1, tree=tree, stream=0, **kw)

    refused(rq, 1, call, tree=tree.view(torch.uint64))
    refused(rq, 1, call)                            # what is right reaches the library: no context
    refused(rq, 2, call, table=table[:, :4])        # the pages in use of a wider table
    refused(rq, 2, call, table=table.t())
    refused(rq, 2, call, table=table.view(-1))
    refused(rq, 2, call, max_pages=4)
    refused(rq, 3, call, table=table.long())
    refused(rq, 3, call, length=length.long())
    refused(rq, 2, call, length=torch.zeros(4, dtype=torch.int32)[::2])
    refused(rq, 3, call, tree=tree.int())
    refused(rq, 2, call, tree=torch.zeros(2, 6, dtype=torch.int64)[:, :3])

    token = torch.zeros(2, 3, dtype=torch.int32)
    prob, draft, u = torch.zeros(2, 4, 10), torch.zeros(2, 3, 10), torch.zeros(2, 4)
    out, path = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    good = dict(token=token, p=prob, q=draft, u=u, accepted=out, next=out.clone())
    tree_good = dict(token=token, parent=token.clone(), p=prob, u=u, accepted=out,
                     next=out.clone(), path=path)
    for call, args in ((rq.rq_verify_chain, good), (rq.rq_verify_tree, tree_good)):
        for name, t in args.items():
            other = t.long() if t.dtype == torch.int32 else t.double()
            apart = torch.stack([t, t], -1)[..., 0]
            refused(rq, 3, call, batch=2, drafts=3, vocab=10, stream=0, **dict(args, **{name: other}))
            refused(rq, 2, call, batch=2, drafts=3, vocab=10, stream=0, **dict(args, **{name: apart}))


def test_binding_refuses_rows_of_different_types_and_outputs_that_are_not_dense(rq):
    import torch
    c, st = small_cache(rq), dict(stream=0)
    p = rq.QKParams(4, 2, 64, cos=torch.zeros(8, 32), sin=torch.zeros(8, 32))
    q, k, v = torch.zeros(4, 4, 64), torch.zeros(4, 2, 64), torch.zeros(4, 2, 64)
    pos, slot = torch.arange(4, dtype=torch.int32), torch.arange(4)
    apart = torch.zeros(4, 8, 64)
    for q1, k1, v1, o1, status in (
            (q.bfloat16(), k, v, q.clone(), 3), (q, k.half(), v, q.clone(), 3),
            (q, k, v.half(), q.clone(), 3), (q, k, v, q.bfloat16(), 3),
            (q, k, v, apart[:, :4], 2), (q.double(), k.double(), v.double(), q.double(), 3)):
        refused(rq, status, rq.rq_qkv_to_cache, p, q1, k1, v1, pos, o1, c, slot, 4, **st)
    for q1, k1, qo, ko, status in (
            (q, k.half(), q.clone(), k.half(), 3), (q, k, q.half(), k.clone(), 3),
            (q, k, q.clone(), k.bfloat16(), 3), (q, k, apart[:, 4:], k.clone(), 2),
            (q, k, q.clone(), apart[:, ::4], 2), (None, k, None, k.half(), 3)):
        refused(rq, status, rq.rq_qk_norm_rope, p, q1, k1, pos, qo, ko, 4, **st)
    refused(rq, 3, rq.rq_kv_write, c, k, v.half(), slot, 4, **st)
    refused(rq, 3, rq.rq_kv_write, c, k.double(), v.double(), slot, 4, **st)
    refused(rq, 3, rq.rq_kv_read, c, slot, k.half(), v.clone(), 4, **st)
    refused(rq, 2, rq.rq_kv_read, c, slot, apart[:, :2], v.clone(), 4, **st)
    refused(rq, 2, rq.rq_kv_read, c, slot, k.clone(), apart[:, 1:3], 4, **st)

    q4 = torch.zeros(2, 3, 4, 64)
    table, length = torch.zeros(2, 6, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for out, status in ((q4.half(), 3), (torch.zeros(2, 3, 8, 64)[:, :, :4], 2), (q4.clone(), 1)):
        refused(rq, status, rq.Context.rq_cache_attention, NoContext, c, q4, out, table, length, 2,
                3, 4, 0.1, stream=0)
    with pytest.raises(rq.RqError):
        rq.QKParams(4, 2, 64, q_weight=torch.ones(64, dtype=torch.int32))
    with pytest.raises(rq.RqError):
        rq.KVCache.from_tensors(c.k, c.v, c.k_scale.int(), c.v_scale, format=rq.RQ_KV_I8)


def test_the_format_of_a_cache_is_its_codes_type(rq):
    import torch
    k, s = torch.zeros(8, 2, 16, 64, dtype=torch.int8), torch.zeros(8, 2, 16)
    e4m3, raw = k.view(torch.float8_e4m3fn), k.view(torch.uint8)
    make = rq.KVCache.from_tensors
    assert make(k, k, s, s).struct.format == rq.RQ_KV_I8
    assert make(k, k, s, s, format=rq.RQ_KV_I8).struct.format == rq.RQ_KV_I8
    assert make(e4m3, e4m3, s, s).struct.format == rq.RQ_KV_E4M3
    assert make(raw, raw, s, s).struct.format == rq.RQ_KV_E4M3
    assert make(raw, raw, s, s, format=rq.RQ_KV_I8).struct.format == rq.RQ_KV_I8
    refused(rq, 3, make, k, k, s, s, format=rq.RQ_KV_E4M3)
    refused(rq, 3, make, e4m3, e4m3, s, s, format=rq.RQ_KV_I8)
    refused(rq, 3, make, k, e4m3, s, s)


def test_more_drafts_than_rows_are_counted_in(rq):
    lib = rq.lib()
    for n in ((1 << 30) + 1, 0x7FFFFFFF - 511, 0x7FFFFFFF):
        assert lib.rq_verify_chain(A, A, NULL, A, A, A, 1, n, 1, NULL) == 2
        assert lib.rq_verify_tree(A, A, A, A, A, A, A, 1, n, 1, NULL) == 2
