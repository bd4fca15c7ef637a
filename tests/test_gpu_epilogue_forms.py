"""GPU: what the epilogue's callers may rely on besides its sums: rows that are
rewritten in place are read anew, weights are waited for, and activations keep
their digits."""
import pytest
import torch

import pass_util as ref
import synthetic

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def packed(rq, seed, n, k):
    w = synthetic.weight_matrix(seed, rq.RQ_Q4K, n, k)
    return torch.from_numpy(w.view("uint8").reshape(-1).copy()).cuda()


def rows(seed, m, k):
    return torch.from_numpy(synthetic.activation(seed, m, k)).cuda()


@pytest.mark.parametrize("M", [1, 3])
def test_rows_rewritten_in_place_below_the_threshold(rq, M):
    # where rq_linear reads x itself, nothing has to be invalidated
    N, K = 512, 1024
    ctx, w = rq.Context(), packed(rq, 5, N, K)
    x, y = torch.empty(M, K, device="cuda"), torch.empty(M, N, device="cuda")
    for seed in (41, 42, 43):
        x.copy_(rows(seed, M, K))
        ctx.rq_linear_epilogue(rq.RQ_Q4K, w, x, y, M, N, K, act="silu")
        fresh, want = rq.Context(), torch.empty_like(y)
        fresh.rq_linear_epilogue(rq.RQ_Q4K, w, rows(seed, M, K), want, M, N, K, act="silu")
        torch.cuda.synchronize()
        fresh.close()
        assert torch.equal(y, want)
    ctx.close()


def test_nothing_is_left_in_the_cache_below_the_threshold(rq):
    # a call that asks for no invalidation is not what a later one finds
    M, N, K = 2, 512, 1024
    ctx, w = rq.Context(), packed(rq, 5, N, K)
    x, y, want = rows(44, M, K), *(torch.empty(M, N, device="cuda") for _ in range(2))
    ctx.rq_linear_epilogue(rq.RQ_Q4K, w, x, y, M, N, K)
    x.copy_(rows(45, M, K))
    ctx.set_gemm_threshold(1)
    ctx.rq_linear(rq.RQ_Q4K, w, x, y, M, N, K)
    fresh = rq.Context(gemm_threshold=1)
    fresh.rq_linear(rq.RQ_Q4K, w, rows(45, M, K), want, M, N, K)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert ctx.stats()["act_hits"] == 0
    fresh.close()
    ctx.close()


@pytest.mark.parametrize("M", [1, 3, 40])
def test_a_norm_and_a_gated_product_layer_after_layer(rq, M):
    # x is written in place by each layer's norm
    N, K = 512, 1024
    ctx = rq.Context()
    layers = [packed(rq, s, N, K) for s in (7, 8, 9)]
    norm, up = rq.NormParams(K), rows(50, M, N)
    h, x, y = rows(51, M, K), torch.empty(M, K, device="cuda"), torch.empty(M, N, device="cuda")
    for i, w in enumerate(layers):
        block = rows(52 + i, M, K)
        rq.rq_residual_norm(norm, block, h, h, x, M)
        ctx.rq_act_cache_invalidate()
        ctx.rq_linear_epilogue(rq.RQ_Q4K, w, x, y, M, N, K, act="silu", mul=up)
        fresh, want = rq.Context(), torch.empty_like(y)
        fresh.rq_linear_epilogue(rq.RQ_Q4K, w, x.clone(), want, M, N, K, act="silu", mul=up)
        torch.cuda.synchronize()
        fresh.close()
        assert torch.equal(y, want)
    ctx.close()


@pytest.mark.parametrize("M,N,K", [(8, 18944, 3584), (300, 18944, 3584), (2000, 9472, 3584)])
def test_a_weight_cached_right_before_a_product_of_a_cached_activation(rq, M, N, K):
    # nothing is launched between the weight's encoding and the product
    ctx = rq.Context()
    small, x = packed(rq, 11, 256, K), rows(12, M, K)
    w = [packed(rq, 13, N, K) for _ in range(3)]
    y, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    aside = torch.empty(M, 256, device="cuda")
    for i, linear in ((0, True), (1, False), (2, True)):
        ctx.rq_linear(rq.RQ_Q4K, small, x, aside, M, 256, K)        # x is cached
        hits = ctx.stats()["act_hits"]
        ctx.rq_fp8_weight_cache(rq.RQ_Q4K, w[i], N, K)
        if linear:
            ctx.rq_linear(rq.RQ_Q4K, w[i], x, y, M, N, K)
        else:
            ctx.rq_linear_epilogue(rq.RQ_Q4K, w[i], x, y, M, N, K)
        assert ctx.stats()["act_hits"] == hits + 1
        torch.cuda.synchronize()
        ctx.rq_linear(rq.RQ_Q4K, w[i], x, want, M, N, K)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    ctx.close()


def activated(rq, z, act, dtype, tiles):
    """act(z) by way of the bias.  tiles: enough tokens for the tile kernels (no
    split of K), each of which then has the same row."""
    N, K, M = len(z), 128, 300 if tiles else 1
    x, w = torch.zeros((M + 15) // 16 * 16, K), torch.zeros(N, K)
    args = (x.to(torch.float8_e4m3fn).cuda(), torch.ones(1).cuda(),
            w.to(torch.float8_e4m3fn).cuda(), torch.ones(1).cuda())
    y = torch.empty(M, N, dtype=ref.DTYPES[dtype], device="cuda")
    rq.rq_fp8_gemm_epilogue(*args, y, M, N, K, act=act, bias=z.cuda())
    assert rq.rq_get_device_status() == 0
    assert bool((y == y[0]).all())
    return y[0].double().cpu()


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gelu_keeps_its_digits(rq, dtype, tiles):
    """z from -13 to 13, small and large: within 2^-20 of the result itself, then
    rounded.  2^-20 = 16 u is the power's 2^-22 (4 u) and the reciprocal's 2^-23
    (2 u), the fit's 4.4e-8 (1 u), the sum of nine terms whose magnitudes add up
    to four times their sum (3 u), and the roundings of the root's argument, the
    halves and three products (6 u).  16-bit results leave the rounding of the
    power's argument, z^2 / 2 log2(e) 2^-24 ln 2, of log2(e) in it, a quarter of
    that, and of z^2 / 2 itself: 1.25 z^2 u."""
    g = ref.gen(60)
    z = torch.cat([-13 + 26 * torch.rand(4000, generator=g),
                   torch.randn(2000, generator=g),
                   10.0 ** (-6 * torch.rand(1000, generator=g)),
                   -(10.0 ** (-6 * torch.rand(1000, generator=g))),
                   torch.tensor([0.0, -0.0, 0.75, -0.75, 0.55, -0.55, 40.0, -40.0, 1e30, -1e30])])
    got = activated(rq, z, "gelu", dtype, tiles)
    want = ref.act(z.double(), "gelu")
    # (past where a 16-bit or a normal f32 result is one)
    e = 2.0 ** -20 * want.abs()
    if dtype != "f32":
        e = e + 1.25 * ref.U * z.double().square() * want.abs()
    tol = e + ref.ROUND[ref.DTYPES[dtype]] * (want.abs() + e) + \
        (2.0 ** -126 if dtype != "f16" else ref.TINY[torch.float16])
    off = (got - want).abs()
    # (what its type cannot hold is infinite)
    off = torch.where(want.abs() > torch.finfo(ref.DTYPES[dtype]).max,
                      torch.where(got == float("inf"), 0.0, off), off)
    worst = (off / tol).argmax()
    assert bool((off <= tol).all()), (float(z[worst]), float(got[worst]), float(want[worst]))


def test_gelu_of_normal_sums_is_as_near_as_the_plain_form(rq):
    """f32: u of the result, as a norm: the last rounding is below that for each,
    and the tail's 16 u are of values that are a tenth of the others."""
    g = ref.gen(61)
    for sigma in (0.05, 0.3, 1.0, 3.0):
        z = sigma * torch.randn(20000, generator=g)
        want = ref.act(z.double(), "gelu")
        off = activated(rq, z, "gelu", "f32", False) - want
        assert float(off.norm() / want.norm()) <= ref.U, sigma
