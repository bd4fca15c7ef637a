"""The plan, norm, epilogue and sampling entry points refuse bad arguments on
the host, before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

A = 0x10000          # aligned fake addresses: never dereferenced
B = 0x20000
NULL = None


@pytest.fixture(scope="module")
def rq():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_linear_layers_gb300 as rq
    return rq


def epilogue(rq, **over):
    f = dict(bias=A, act=1, mul=A, residual=A, mul_stride=64, residual_stride=64)
    f.update(over)
    return rq._EPILOGUE.pack(*f.values())


def norm(rq, **over):
    f = dict(post_weight=A, pre_weight=A, width=64, norms=3, eps=1e-6, scale=1.0)
    f.update(over)
    return ctypes.byref(rq._NormStruct(**f))


def filters(rq, **over):
    f = dict(temperature=A, top_k=A, top_p=A, min_p=A)
    f.update(over)
    return rq._SAMPLING.pack(*f.values())


@pytest.mark.parametrize("over,status", [
    (dict(act=-1), 3), (dict(act=5), 3), (dict(bias=A + 2), 2), (dict(mul=A + 2), 2),
    (dict(residual=A + 1), 2), (dict(mul_stride=63), 2), (dict(residual_stride=0), 2),
    (dict(mul_stride=-64), 2), (dict(residual_stride=1 << 41), 2),
    (dict(mul=B, mul_stride=65), 2), (dict(residual=B, residual_stride=70), 2)])
def test_bad_epilogues(rq, over, status):
    lib, e = rq.lib(), epilogue(rq, **over)
    ctx = ctypes.c_void_p(A)        # not dereferenced: the checks come first
    assert lib.rq_fp8_gemm_epilogue(A, A, A, A, e, 0, B, 64, 16, 64, 128, NULL) == status
    assert lib.rq_linear_epilogue(ctx, 12, A, A, e, 0, B, 64, 16, 64, 256, NULL) == status


def test_bad_products(rq):
    lib, e = rq.lib(), epilogue(rq)
    f = lib.rq_fp8_gemm_epilogue
    for i in range(4):
        args = [A, A, A, A]
        args[i] = NULL
        assert f(*args, e, 0, B, 64, 16, 64, 128, NULL) == 1
    assert f(A, A, A, A, e, 0, NULL, 64, 16, 64, 128, NULL) == 1
    assert f(A, A, A, A, e, 3, B, 64, 16, 64, 128, NULL) == 3
    assert f(A, A, A, A, e, 0, B, 63, 16, 64, 128, NULL) == 2      # rows overlap
    assert f(A, A, A, A, e, 0, B + 2, 64, 16, 64, 128, NULL) == 2
    assert f(A + 8, A, A, A, e, 0, B, 64, 16, 64, 128, NULL) == 2
    assert f(A, A, A + 4, A, e, 0, B, 64, 16, 64, 128, NULL) == 2
    for M, N, K in ((0, 64, 128), (-1, 64, 128), (1, 0, 128), (1, 64, 0), (1, 64, 130)):
        assert f(A, A, A, A, NULL, 0, B, 64, M, N, K, NULL) == 2
    g, ctx = lib.rq_linear_epilogue, ctypes.c_void_p(A)
    assert g(NULL, 12, A, A, e, 0, B, 64, 16, 64, 256, NULL) == 1
    assert g(ctx, 12, NULL, A, e, 0, B, 64, 16, 64, 256, NULL) == 1
    assert g(ctx, 12, A, NULL, e, 0, B, 64, 16, 64, 256, NULL) == 1
    assert g(ctx, 12, A, A, e, 0, NULL, 64, 16, 64, 256, NULL) == 1
    assert g(ctx, 7, A, A, e, 0, B, 64, 16, 64, 256, NULL) == 3
    assert g(ctx, 12, A, A, e, 4, B, 64, 16, 64, 256, NULL) == 3
    assert g(ctx, 12, A, A, e, 0, B, 64, 16, 64, 128, NULL) == 2
    assert g(ctx, 12, A, A, e, 0, B, 64, 0, 64, 256, NULL) == 2
    assert g(ctx, 12, A + 4, A, e, 0, B, 64, 16, 64, 256, NULL) == 2
    assert g(ctx, 14, A + 4, A + 4, e, 0, B, 64, 16, 64, 256, NULL) == 2


@pytest.mark.parametrize("over", [
    dict(width=0), dict(width=16385), dict(norms=4), dict(norms=-1), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(post_weight=A + 2), dict(pre_weight=A + 1)])
def test_bad_norms(rq, over):
    assert rq.lib().rq_residual_norm(norm(rq, **over), 0, A, 16384, NULL, 0, 0, B, 16384, NULL,
                                     0x30000, NULL, 1, NULL) == 2


def test_bad_norm_rows(rq):
    lib, n = rq.lib(), norm(rq)
    C, D = 0x30000, 0x40000

    def call(p=n, dtype=0, y=A, ys=64, gate=NULL, gs=0, hd=0, h=B, hs=64, ho=C, x=D, top=NULL,
             tokens=1):
        return lib.rq_residual_norm(p, dtype, y, ys, gate, gs, hd, h, hs, ho, x, top, tokens, NULL)

    assert call(p=NULL) == 1
    assert call(h=NULL) == 1
    assert call(ho=NULL, x=NULL) == 1
    assert call(y=NULL) == 1                       # a sum without a block
    assert call(y=NULL, ho=NULL, gate=A) == 1
    assert call(x=NULL, top=A) == 1
    assert call(dtype=3) == 3
    assert call(hd=1) == 3 and call(dtype=1, hd=2) == 3 and call(hd=7) == 3
    assert call(dtype=2, hd=2, top=A) == 3         # the quantization reads f32
    assert call(tokens=-1) == 2
    assert call(ys=63) == 2 and call(hs=63) == 2 and call(gate=A, gs=1) == 2
    assert call(y=A + 2) == 2 and call(h=B + 1) == 2 and call(ho=C + 2) == 2
    assert call(x=D + 3) == 2 and call(gate=A + 2) == 2 and call(top=A + 2) == 2
    assert call(ho=B, hs=128) == 2                 # in place needs dense rows
    assert call(x=A, ys=128) == 2
    assert call(x=C) == 2 and call(x=B) == 2 and call(ho=A) == 2
    assert call(gate=D) == 2 and call(gate=C) == 2
    assert call(tokens=0) == 0


def test_bad_plans(rq):
    lib = rq.lib()

    def call(length=A, count=A, batch=2, new=3, page=16, table=A, pages=4, free=A, capacity=8,
             available=A, left=B, slot=A, position=A, sequence=A, rows=6, start=B, following=B):
        return lib.rq_batch_plan(length, count, batch, new, page, table, pages, free, capacity,
                                 available, left, slot, position, sequence, rows, start, following,
                                 NULL)

    for name in ("length", "table", "free", "available", "left", "slot", "position"):
        assert call(**{name: NULL}) == 1
    assert call(count=NULL, new=0) == 1
    for page in (0, 8, 24, 512, -16):
        assert call(page=page) == 2
    assert call(batch=-1, rows=0) == 2 and call(batch=65537, new=0) == 2
    assert call(new=-1) == 2 and call(rows=5) == 2 and call(rows=-1, new=0) == 2
    assert call(pages=0) == 2 and call(capacity=-1) == 2
    assert call(batch=65536, new=65536, rows=0) == 2   # a product past 32 bits
    for name in ("length", "count", "table", "free", "available", "left", "position", "sequence",
                 "start", "following"):
        assert call(**{name: A + 2}) == 2
    assert call(slot=A + 4) == 2
    # inputs that other blocks still read
    assert call(left=A) == 2 and call(following=A) == 2 and call(start=A) == 2
    assert call(length=0x30000, following=A) == 2 and call(length=0x30000, start=A) == 2


def test_bad_sampling(rq):
    lib, f = rq.lib(), filters(rq)
    for draw in (True, False):
        def call(p=f, dtype=0, logits=A, stride=100, u=A, out=B, rows=1, vocab=100):
            if draw:
                return lib.rq_sample(p, dtype, logits, stride, u, out, rows, vocab, NULL)
            return lib.rq_token_probs(p, dtype, logits, stride, out, rows, vocab, NULL)

        assert call(p=NULL) == 1 and call(logits=NULL) == 1 and call(out=NULL) == 1
        assert call(dtype=3) == 3 and call(dtype=-1) == 3
        assert call(stride=99) == 2 and call(vocab=0) == 2
        assert call(vocab=(1 << 20) + 1, stride=1 << 21) == 2
        assert call(rows=-1) == 2 and call(rows=(1 << 27) + 1) == 2
        assert call(logits=A + 2) == 2 and call(dtype=1, logits=A + 1) == 2
        assert call(out=B + 2) == 2
        for name in ("temperature", "top_k", "top_p", "min_p"):
            assert call(p=filters(rq, **{name: A + 2})) == 2
        assert call(rows=0) == 0
    assert lib.rq_sample(f, 0, A, 100, NULL, B, 1, 100, NULL) == 1
    assert lib.rq_sample(f, 0, A, 100, A + 2, B, 1, 100, NULL) == 2
    assert lib.rq_token_probs(f, 0, A, 100, A, 1, 100, NULL) == 2      # onto the logits


def refused(rq, status, f, *args, **more):
    with pytest.raises(rq.RqError) as e:
        f(*args, **more)
    assert e.value.status == status


def test_the_binding_refuses_what_the_library_cannot_see(rq):
    x, i = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    # tensors that are not on the GPU
    refused(rq, 2, rq.rq_sample, x, x[:, 0], i, 4, 64)
    refused(rq, 2, rq.rq_token_probs, x, x, 4, 64)
    refused(rq, 2, rq.rq_residual_norm, rq.NormParams(64), x, x, x, x, 4)
    refused(rq, 2, rq.NormParams, 64, post_weight=x[0])
    refused(rq, 2, rq.rq_fp8_gemm_epilogue, x, x, x, x, x, 4, 64, 128)
    refused(rq, 2, rq.rq_batch_plan, i, i[:, None], i, i, i, i.long(), i, 16, new_tokens=1)
    # types and lengths, whatever the device
    refused(rq, 3, rq.rq_sample, x, x.double()[:, 0], i, 4, 64, dtype=0, top_k=i.long())
    refused(rq, 3, rq.NormParams, 64, pre_weight=x[0].double())
    refused(rq, 2, rq.NormParams, 65, pre_weight=x[0])
    refused(rq, 3, rq.rq_batch_plan, i.long(), i[:, None], i, i, i, i.long(), i, 16, new_tokens=1)
    refused(rq, 2, rq.rq_batch_plan, i, i, i, i, i, i.long(), i, 16, new_tokens=1)
    refused(rq, 2, rq.rq_token_probs, x, x, 5, 64)
    refused(rq, 2, rq.rq_token_probs, x, x, 4, 63)
    refused(rq, 3, rq.rq_fp8_gemm_epilogue, x, x, x, x, x, 4, 64, 128, act="swish")
    refused(rq, 3, rq.rq_fp8_gemm_epilogue, x, x, x, x, x, 4, 64, 128, mul=x.half())
    refused(rq, 2, rq.rq_fp8_gemm_epilogue, x, x, x, x, x, 4, 64, 128, mul=x[:3])
    refused(rq, 3, rq.rq_residual_norm, rq.NormParams(64), x, x, x, x.half(), 4)


def test_rows_and_their_distance(rq):
    where = "test"
    t = torch.zeros(6, 96)

    def at(x, rows, cols, **more):
        saved, rq._on_device = rq._on_device, lambda t, dev, where, name: t.data_ptr()
        try:
            return rq._matrix(x, rows, cols, 0, where, "t", **more)
        finally:
            rq._on_device = saved

    assert at(t, 6, 96) == (t.data_ptr(), 96)
    assert at(t[:, 32:], 6, 64) == (t.data_ptr() + 128, 96)
    assert at(t[::2], 3, 96) == (t.data_ptr(), 192)
    assert at(t[0], 1, 96) == (t.data_ptr(), 96)
    assert at(t.view(2, 3, 96)[:, :, :10], 6, 10) == (t.data_ptr(), 96)
    assert at(t[:, :10].unsqueeze(1), 6, 10)[1] == 96
    assert at(t[0].expand(6, 96), 6, 96)[1] == 0    # the library refuses rows in one place
    for x, rows, cols in ((t, 7, 96), (t, 6, 95), (t.T, 96, 6), (t[:, ::2], 6, 48),
                          (t.view(2, 3, 96)[:, :2, :10], 4, 10)):
        refused(rq, 2, at, x, rows, cols)
    refused(rq, 2, at, t[:, 32:], 6, 64, dense=True)
