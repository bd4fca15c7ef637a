"""GPU: the FP8 product with bias, activation, multiplication and residual in
its epilogue, against 64 bits on the same codes."""
import pytest
import torch

import pass_util as ref

pytestmark = pytest.mark.gpu
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def codes(g, rows, K, pad=0):
    x = torch.randn(rows, K, generator=g)
    q = torch.zeros(rows + pad, K)
    q[:rows] = x * (448.0 / x.abs().max())
    if pad:
        q[rows:] = 448.0  # rows behind the last token must not matter
    return q.to(torch.float8_e4m3fn), torch.tensor([x.abs().max() / 448.0])


def operands(g, M, N, dtype, bias, mul, residual, stride):
    def rows():
        x = torch.randn(M, stride or N, generator=g).to(ref.DTYPES[dtype]).cuda()
        return x[:, :N]
    return (0.5 * torch.randn(N, generator=g).cuda() if bias else None, rows() if mul else None,
            rows() if residual else None)


def check(rq, M, N, K, dtype, act="none", bias=False, mul=False, residual=False, stride=None,
          y_stride=None, seed=0):
    g = ref.gen(seed + M + 3 * N + K)
    x, xs = codes(g, M, K, -M % 16)
    w, ws = codes(g, N, K)
    ws = ws * K ** -0.5
    b, m, r = operands(g, M, N, dtype, bias, mul, residual, stride)
    room = torch.full((M, y_stride or N), 7.0, dtype=ref.DTYPES[dtype], device="cuda")
    y = room[:, :N]
    rq.rq_fp8_gemm_epilogue(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y, M, N, K, act=act, bias=b,
                            mul=m, residual=r)
    assert rq.rq_get_device_status() == 0
    cpu = [None if t is None else t.cpu() for t in (b, m, r)]
    want, tol = ref.product(x[:M].float(), xs, w.float(), ws, cpu[0], act, cpu[1], cpu[2],
                            ref.DTYPES[dtype])
    off = (y.cpu().double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    assert bool((room[:, N:] == 7).all())


# one tile split over K, one-CTA tiles, CTA pairs, and ragged edges of each
SIZES = [(1, 64, 128), (1, 1000, 2048), (5, 130, 896), (16, 3584, 512), (48, 257, 4096),
         (129, 384, 256), (300, 777, 384), (520, 2048, 256), (1000, 1500, 128), (64, 9728, 256)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes_and_types(rq, M, N, K, dtype):
    check(rq, M, N, K, dtype)
    check(rq, M, N, K, dtype, "silu", True, True, True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_parts(rq, act, dtype):
    for M, N, K in ((7, 200, 1024), (400, 1100, 256), (150, 20000, 128)):
        for parts in ((True, False, False), (False, True, False), (False, False, True)):
            check(rq, M, N, K, dtype, act, *parts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_apart(rq, dtype):
    for M, N, K in ((3, 96, 512), (200, 515, 128), (600, 1024, 256)):
        check(rq, M, N, K, dtype, "silu", True, True, True, stride=2 * N + 8, y_stride=N + 8)
        check(rq, M, N, K, dtype, "none", True, True, True, stride=N + 1, y_stride=N + 3)


@pytest.mark.parametrize("M,N,K", [(2, 300, 1024), (200, 515, 128), (700, 2048, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(rq, M, N, K, dtype):
    g = ref.gen(M)
    x, xs = codes(g, M, K, -M % 16)
    w, ws = codes(g, N, K)
    args = (x.cuda(), xs.cuda(), w.cuda(), ws.cuda())
    _, m, r = operands(g, M, N, dtype, False, True, True, None)
    y = torch.empty_like(r)
    rq.rq_fp8_gemm_epilogue(*args, y, M, N, K, act="gelu", mul=m, residual=r)
    onto_r, onto_m = r.clone(), m.clone()
    rq.rq_fp8_gemm_epilogue(*args, onto_r, M, N, K, act="gelu", mul=m, residual=onto_r)
    rq.rq_fp8_gemm_epilogue(*args, onto_m, M, N, K, act="gelu", mul=onto_m, residual=r)
    assert torch.equal(onto_r, y) and torch.equal(onto_m, y)


def test_without_an_epilogue_it_is_the_product(rq):
    g = ref.gen(1)
    for M, N, K in ((20, 640, 1024), (300, 1000, 256), (1024, 4096, 512)):
        x, xs = codes(g, M, K, -M % 16)
        w, ws = codes(g, N, K)
        args = (x.cuda(), xs.cuda(), w.cuda(), ws.cuda())
        plain, y = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        rq.rq_fp8_gemm(args[0].view(torch.uint8), args[1], args[2].view(torch.uint8), args[3], plain,
                       M, N, K)
        rq.rq_fp8_gemm_epilogue(*args, y, M, N, K)
        assert torch.equal(plain, y)
        # the C call without an epilogue at all
        y.zero_()
        assert rq.lib().rq_fp8_gemm_epilogue(*[t.data_ptr() for t in args], None, 0, y.data_ptr(), N,
                                             M, N, K, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(plain, y)


def test_activations_of_large_and_special_sums(rq):
    # sums of 0, +-large and NaN by way of the bias
    N, K = 8, 128
    x, w = torch.zeros(16, K), torch.zeros(N, K)
    bias = torch.tensor([0.0, 90.0, -90.0, 1e4, -1e4, float("inf"), float("nan"), -30.0]).cuda()
    args = (x.to(torch.float8_e4m3fn).cuda(), torch.ones(1).cuda(),
            w.to(torch.float8_e4m3fn).cuda(), torch.ones(1).cuda())
    for dtype in ("f32", "bf16"):
        for act in ACTS:
            y = torch.empty(1, N, dtype=ref.DTYPES[dtype], device="cuda")
            rq.rq_fp8_gemm_epilogue(*args, y, 1, N, K, act=act, bias=bias)
            want = ref.act(bias.double().cpu(), act)
            want[5] = float("inf")
            got = y[0].double().cpu()
            assert bool(got[6].isnan()) and got[5] == float("inf")
            tol = 2 * ref.ROUND[y.dtype] * want.abs() + 16 * ref.U * bias.double().cpu().abs()
            keep = [0, 1, 2, 3, 4, 7]
            assert bool(((got - want).abs() <= tol)[keep].all()), (act, got, want)


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_linear_route(rq, M):
    import synthetic
    N, K = 512, 1024
    ctx = rq.Context(gemm_threshold=1)
    w = torch.from_numpy(synthetic.weight_matrix(5, rq.RQ_Q4K, N, K).view("uint8").reshape(-1).copy()).cuda()
    x = torch.from_numpy(synthetic.activation(6, M, K)).cuda()
    g = ref.gen(7)
    b, m, r = operands(g, M, N, "f32", True, True, True, None)
    plain, y = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    ctx.rq_linear(rq.RQ_Q4K, w, x, plain, M, N, K)
    hits = ctx.stats()["act_hits"]
    ctx.rq_linear_epilogue(rq.RQ_Q4K, w, x, y, M, N, K, act="silu", bias=b, mul=m, residual=r)
    assert ctx.stats()["act_hits"] == hits + 1 and ctx.stats()["weights"] == 1
    z = plain.double() + b.double()
    want = r.double() + m.double() * (z * torch.sigmoid(z))
    # the product's own sums (rounded once less here), then as in ref.product
    tol = 8 * ref.U * (plain.abs() + z.abs()).double() * (1.13 * m.abs()) + \
        16 * ref.U * z.abs() * m.abs() + 2 * ref.U * want.abs()
    assert bool(((y.double() - want).abs() <= tol).all())
    # at every M, whatever the threshold
    ctx.set_gemm_threshold(1000)
    again = torch.empty_like(y)
    ctx.rq_linear_epilogue(rq.RQ_Q4K, w, x, again, M, N, K, act="silu", bias=b, mul=m, residual=r)
    assert torch.equal(again, y)
    ctx.close()


def test_graph_and_stream(rq):
    g = ref.gen(9)
    M, N, K = 64, 1024, 2048
    x, xs = codes(g, M, K)
    w, ws = codes(g, N, K)
    args = (x.cuda(), xs.cuda(), w.cuda(), ws.cuda())
    b, m, r = operands(g, M, N, "bf16", True, True, True, None)
    ys = [torch.empty_like(m) for _ in range(3)]
    rq.rq_fp8_gemm_epilogue(*args, ys[0], M, N, K, act="relu", bias=b, mul=m, residual=r)
    torch.cuda.synchronize()
    rq.rq_fp8_gemm_epilogue(*args, ys[1], M, N, K, act="relu", bias=b, mul=m, residual=r,
                            stream=torch.cuda.Stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.rq_fp8_gemm_epilogue(*args, ys[2], M, N, K, act="relu", bias=b, mul=m, residual=r)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
