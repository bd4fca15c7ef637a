"""GPU: per-head norm and rotation, and the quantized cache's write and read
back, against 64-bit definitions (norm, rotation) and a CPU restatement in
correctly rounded f32 operations (codes and scales, bit for bit)."""
import pytest
import torch

from serving_util import ROUND, TOP, TORCH, U, encode, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def tables(r, most=500):
    f = 10000.0 ** (-torch.arange(r // 2, dtype=torch.float64) * 2 / r)
    a = torch.arange(most, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def turned(x, weight, eps, cos, sin, rotary, interleaved):
    """The definition in 64 bits and its f32 error bound per value."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    z, size = y.clone(), y.abs()
    if rotary:
        c, s = cos.double()[:, None], sin.double()[:, None]
        if interleaved:
            ia, ib = torch.arange(0, rotary, 2), torch.arange(1, rotary, 2)
        else:
            ia, ib = torch.arange(rotary // 2), torch.arange(rotary // 2, rotary)
        a, b = y[..., ia], y[..., ib]
        z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
        size = size.clone()
        size[..., ia] = (a * c).abs() + (b * s).abs()
        size[..., ib] = (b * c).abs() + (a * s).abs()
    # the norm: sum of D squares in lanes of D/32 and 5 shuffles, division,
    # root, two products; the turn: two products and a sum
    return z, 24 * U * size


CASES = [
    # tokens, hq, hk, d, rotary, interleaved, packed, dtype, norm
    (1, 28, 4, 128, 128, False, False, "f32", True),
    (3, 28, 4, 128, 64, True, True, "bf16", True),
    (70, 7, 1, 64, 64, False, True, "f16", True),
    (129, 5, 5, 64, 16, True, False, "f32", False),
    (33, 8, 2, 256, 256, False, False, "bf16", True),
    (257, 2, 1, 256, 48, True, True, "f32", True),
    (90, 3, 3, 128, 0, False, False, "f16", True),
    (2, 1, 1, 64, 32, False, False, "f32", True),
]


def inputs(seed, t, hq, hk, d, packed, dtype):
    g = gen(seed)
    x = torch.randn((t, hq + 2 * hk, d), generator=g)
    x = torch.where(torch.rand(x.shape, generator=g) < 1e-2, 30 * x, x).to(TORCH[dtype])
    parts = (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:])
    on = x.cuda()
    dev = (on[:, :hq], on[:, hq:hq + hk], on[:, hq + hk:])
    return parts, dev if packed else tuple(p.contiguous() for p in dev)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_and_rotation(rq, case):
    t, hq, hk, d, r, inter, packed, dtype, norm = case
    (q, k, _), (qd, kd, _) = inputs(11 + t, t, hq, hk, d, packed, dtype)
    g = gen(5)
    qw, kw = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    cos, sin = tables(r) if r else (None, None)
    pos = torch.randint(0, 500, (t,), generator=g)
    layer = rq.QKParams(hq, hk, d, qw.cuda() if norm else None, kw.cuda() if norm else None, 1e-5,
                        cos.cuda() if r else None, sin.cuda() if r else None, r, inter)
    qo = torch.empty((t, hq, d), dtype=TORCH[dtype], device="cuda")
    ko = torch.empty((t, hk, d), dtype=TORCH[dtype], device="cuda")
    pd = pos.int().cuda() if r else None
    rq.rq_qk_norm_rope(layer, qd, kd, pd, qo, ko, t)
    assert rq.rq_get_device_status() == 0
    cs = (cos[pos], sin[pos]) if r else (None, None)
    for x, w, got in ((q, qw, qo), (k, kw, ko)):
        ref, tol = turned(x, w if norm else None, 1e-5, *cs, r, inter)
        tol = tol + ROUND[dtype] * ref.abs() * 1.01 + (2.0 ** -25 if dtype == "f16" else 0)
        err = (got.cpu().double() - ref).abs()
        assert bool((err <= tol).all()), float((err / tol.clamp_min(1e-300)).max())
    # one side alone, and in place
    q2 = qd.clone()
    rq.rq_qk_norm_rope(layer, q2, None, pd, q2, None, t)
    assert torch.equal(q2.view(t, hq, d), qo)
    k2 = torch.empty_like(ko)
    rq.rq_qk_norm_rope(layer, None, kd, pd, None, k2, t)
    assert torch.equal(k2, ko)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_fused_write(rq, case, page, fmt):
    t, hq, hk, d, r, inter, packed, dtype, norm = case
    (q, k, v), (qd, kd, vd) = inputs(31 + t, t, hq, hk, d, packed, dtype)
    g = gen(6)
    qw, kw = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    cos, sin = tables(r) if r else (None, None)
    pos = torch.randint(0, 500, (t,), generator=g)
    layer = rq.QKParams(hq, hk, d, qw.cuda() if norm else None, kw.cuda() if norm else None, 1e-5,
                        cos.cuda() if r else None, sin.cuda() if r else None, r, inter)
    pages = -(-t // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:t]
    if t > 2:
        slots[1] = -1                       # not written
    cache = rq.KVCache(pages, page, hk, d, fmt)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).fill_(0x55)
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(-7.0)
    qo = torch.empty((t, hq, d), dtype=TORCH[dtype], device="cuda")
    pd = pos.int().cuda() if r else None
    rq.rq_qkv_to_cache(layer, qd, kd, vd, pd, qo, cache, slots.cuda(), t)
    assert rq.rq_get_device_status() == 0
    ko = torch.empty((t, hk, d), dtype=TORCH[dtype], device="cuda")
    q2 = torch.empty_like(qo)
    rq.rq_qk_norm_rope(layer, qd, kd, pd, q2, ko, t)
    assert torch.equal(q2, qo)

    codes, scales = cache.k.cpu(), cache.k_scale.cpu()
    vcodes, vscales = cache.v.cpu(), cache.v_scale.cpu()
    written = torch.zeros(pages * page, dtype=torch.bool)
    written[slots[slots >= 0]] = True
    untouched = ~written.view(pages, page)
    for c, s in ((codes, scales), (vcodes, vscales)):
        assert bool((c.view(torch.uint8).transpose(1, 2)[untouched] == 0x55).all())
        assert bool((s.transpose(1, 2)[untouched] == -7.0).all())
    live = slots >= 0
    pg, off = slots[live] // page, slots[live] % page
    # v as it came: bit for bit
    want, wscale = encode(v[live].float(), fmt)
    assert torch.equal(vcodes.view(torch.uint8)[pg, :, off], want.view(torch.uint8))
    assert torch.equal(vscales[pg, :, off], wscale)
    # k after norm and rotation: half a step of the format, and f32's errors
    cs = (cos[pos], sin[pos]) if r else (None, None)
    ref, tol = turned(k, kw if norm else None, 1e-5, *cs, r, inter)
    ref, tol = ref[live], tol[live]
    s = scales[pg, :, off].double()[..., None]
    amax = ref.abs().amax(-1, keepdim=True)
    assert bool(((s * TOP[fmt] - amax).abs() <= tol.amax(-1, keepdim=True) + 4 * U * amax).all())
    got = codes.view(torch.uint8)[pg, :, off].view(codes.dtype).float().double() * s
    half = torch.maximum(ref.abs() * 2.0 ** -4, s * 2.0 ** -10) if fmt == 0 else s * 0.5
    tol = half + 2 * tol + 8 * U * amax
    err = (got - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("t,hk,d,page", [(1, 1, 64, 16), (37, 4, 128, 32), (300, 3, 256, 128),
                                         (1000, 2, 64, 64)])
def test_write_and_read_back(rq, t, hk, d, page, fmt, dtype):
    g = gen(t + d)
    k = torch.randn((t, hk, d), generator=g) * torch.exp(6 * torch.randn((t, hk, 1), generator=g))
    v = torch.randn((t, hk, d), generator=g)
    v[0] = 0                                                  # a row of zeros
    if t > 30:
        if dtype != "f16":                                    # beyond f32's scale limit
            k[3] = 1e-35 * v[3]
        k[5, 0, 3], k[5, 0, 7], v[6, 0, 1] = float("inf"), -float("inf"), float("nan")
        v[7, 0] = float("inf")                                # nothing finite
        v[8, 0, :] = 2.0 ** -9 * torch.arange(d)
    k, v = k.to(TORCH[dtype]), v.to(TORCH[dtype])
    pages = -(-t // page) + 1
    slots = torch.randperm(pages * page, generator=g)[:t]
    cache = rq.KVCache(pages, page, hk, d, fmt)
    sd = slots.cuda()
    rq.rq_kv_write(cache, k.cuda(), v.cuda(), sd, t)
    pg, off = slots // page, slots % page
    for x, c, s in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        codes, scale = encode(x.float(), fmt)
        assert torch.equal(c.cpu().view(torch.uint8)[pg, :, off], codes.view(torch.uint8))
        assert torch.equal(s.cpu()[pg, :, off], scale)
    ko = torch.full((t, hk, d), 9.0, dtype=TORCH[dtype], device="cuda")
    vo = torch.full_like(ko, 9.0)
    read = slots.clone()
    if t > 3:
        read[2] = -5
    rq.rq_kv_read(cache, read.cuda(), ko, vo, t)
    assert rq.rq_get_device_status() == 0
    for x, got in ((k, ko), (v, vo)):
        codes, scale = encode(x.float(), fmt)
        want = (codes.float() * scale[..., None]).to(TORCH[dtype])
        if t > 3:
            want[2] = 0
        assert torch.equal(got.cpu(), want)


def test_rows_without_weight_keep_values(rq):
    """No norm, no rotation: q and k pass through unchanged."""
    x = torch.randn((9, 2, 64), device="cuda")
    out, ko = torch.empty_like(x), torch.empty_like(x)
    rq.rq_qk_norm_rope(rq.QKParams(2, 2, 64), x, x, None, out, ko, 9)
    assert torch.equal(out, x) and torch.equal(ko, x)


def test_indexes_outside_are_left_out_and_reported(rq):
    t, hk, d, page = 6, 2, 64, 16
    cache = rq.KVCache(2, page, hk, d)
    x = torch.randn((t, hk, d), device="cuda")
    assert rq.rq_get_device_status() == 0
    slots = torch.tensor([0, 32, 5, 1 << 40, -1, 31], device="cuda")
    rq.rq_kv_write(cache, x, x, slots, t)
    assert rq.rq_get_device_status() == 9
    assert rq.rq_get_device_status() == 0
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    rq.rq_kv_read(cache, slots, ko, vo, t)
    assert rq.rq_get_device_status() == 9
    assert not ko[[1, 3, 4]].any() and bool(ko[[0, 2, 5]].any())
    assert int((cache.k_scale != 0).sum()) == 3 * hk
    cos, sin = tables(64)
    layer = rq.QKParams(hk, hk, d, cos=cos.cuda(), sin=sin.cuda())
    pos = torch.tensor([0, 500, -1, 499, 7, 1], dtype=torch.int32, device="cuda")
    rq.rq_qk_norm_rope(layer, x, None, pos, ko, None, t)
    assert rq.rq_get_device_status() == 9
    assert torch.equal(ko[1], x[1]) and torch.equal(ko[2], x[2]) and not torch.equal(ko[3], x[3])


def test_cache_past_32_bit_offsets(rq):
    """A slot whose codes lie past 2^32 bytes."""
    hk, d, page = 8, 256, 256
    pages = (1 << 32) // (hk * d * page) + 3
    cache = rq.KVCache(pages, page, hk, d, rq.RQ_KV_I8)
    g = gen(3)
    x = torch.randn((2, hk, d), generator=g)
    slots = torch.tensor([pages * page - 1, (pages - 1) * page + 17])
    xd, sd = x.cuda(), slots.cuda()
    rq.rq_kv_write(cache, xd, xd, sd, 2)
    ko, vo = torch.empty_like(xd), torch.empty_like(xd)
    rq.rq_kv_read(cache, sd, ko, vo, 2)
    codes, scale = encode(x, 1)
    want = codes.float() * scale[..., None]
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)
    assert torch.equal(cache.k[pages - 1, :, [255, 17]].cpu().transpose(0, 1), codes)
    assert rq.rq_get_device_status() == 0
    del cache
    torch.cuda.empty_cache()


def test_other_stream_and_graph(rq):
    """The calls run on the given stream, and replay from a CUDA graph."""
    t, hk, d, page = 50, 2, 128, 32
    x, y = torch.randn((2, t, hk, d), device="cuda")
    cache = rq.KVCache(3, page, hk, d)
    slots = torch.arange(t, device="cuda")
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            rq.rq_kv_write(cache, x, y, slots, t)
            rq.rq_kv_read(cache, slots, ko, vo, t)
    for _ in range(2):
        x.normal_()
        y.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((x, ko), (y, vo)):
            c, s = encode(a.cpu(), 0)
            assert torch.equal(b.cpu(), c.float() * s[..., None])
