"""GPU: norms, gate and residual sum between blocks against 64 bits."""
import numpy as np
import pytest
import torch

import pass_util as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def rows(g, t, n, dtype, stride=None):
    """Normal rows with a few large values, `stride` elements apart."""
    x = torch.randn(t, n, generator=g) * (1 + 15 * (torch.rand(n, generator=g) < 0.01))
    wide = torch.zeros(t, stride or n)
    wide[:, :n] = x
    return wide.to(ref.DTYPES[dtype]).cuda()[:, :n]


def check(rq, t, n, dtype, h_dtype=None, post=True, pre=True, weights=True, gate=None, scale=0.7,
          block=True, stream_out=True, x_out=True, absmax=False, stride=None, seed=0):
    g = ref.gen(seed + t * 31 + n)
    h_dtype = h_dtype or dtype
    y = rows(g, t, n, dtype, stride) if block else None
    h = rows(g, t, n, h_dtype, stride)
    wp = (1 + 0.2 * torch.randn(n, generator=g)).cuda() if weights else None
    wq = (1 + 0.2 * torch.randn(n, generator=g)).cuda() if weights else None
    gates = None
    if gate == "channel":
        gates = torch.randn(n, generator=g).to(ref.DTYPES[dtype]).cuda()
    elif gate == "token":
        gates = rows(g, t, n, dtype, stride)
    ho = torch.full((t, n), 9.0, dtype=h.dtype, device="cuda") if stream_out else None
    xo = torch.full((t, n), 9.0, dtype=ref.DTYPES[dtype], device="cuda") if x_out else None
    top = torch.full((1,), -1, dtype=torch.int32, device="cuda") if absmax else None
    p = rq.NormParams(n, post=post, pre=pre, post_weight=wp, pre_weight=wq, eps=EPS, scale=scale)
    rq.rq_residual_norm(p, y, h, ho, xo, t, gate=gates, absmax_bits=top)
    cpu = [None if v is None else v.cpu() for v in (y, h, wp, wq, gates)]
    H, X, eh, ex = ref.norm(cpu[0], cpu[1], post, pre, cpu[2], cpu[3], cpu[4], scale, EPS, n)
    for got, want, e in ((ho, H, eh), (xo, X, ex)):
        if got is None:
            continue
        tol = e + ref.ROUND[got.dtype] * (want.abs() + e) + ref.TINY[got.dtype]
        assert bool(((got.double().cpu() - want).abs() <= tol).all())
    if absmax:
        assert top.view(torch.float32).item() == xo.abs().max().item()


@pytest.mark.parametrize("dtype,h_dtype", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                           ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [1, 3, 32, 257, 1024, 3584, 4099, 8192, 16383, 16384])
def test_widths_and_types(rq, n, dtype, h_dtype):
    for t in (1, 5):
        check(rq, t, n, dtype, h_dtype)
    check(rq, 310, n, dtype, h_dtype, gate="token")  # more tokens than twice the SMs


@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_parts(rq, block, post, pre, gate):
    for dtype, n in (("f32", 640), ("bf16", 641)):
        for weights in (True, False):
            check(rq, 3, n, dtype, "f32", post, pre, weights, gate if block else None,
                  block=block, stream_out=block)
    if block:
        check(rq, 3, 640, "f16", "f16", post, pre, True, gate, x_out=False)
        check(rq, 3, 640, "f16", "f32", post, pre, True, gate, stream_out=False)


def test_rows_apart(rq):
    for dtype in ("f32", "bf16"):
        check(rq, 7, 512, dtype, "f32", gate="token", stride=1536)
        check(rq, 7, 512, dtype, "f32", gate="token", stride=517)
        check(rq, 400, 96, dtype, "f32", gate="token", stride=104)


@pytest.mark.parametrize("t", [0, 1, 4, 5, 311, 2000])
def test_largest_magnitude(rq, t):
    if t == 0:
        top = torch.full((1,), 5, dtype=torch.int32, device="cuda")
        x = torch.zeros(0, 64, device="cuda")
        rq.rq_residual_norm(rq.NormParams(64), x, x, x, x.clone(), 0, absmax_bits=top)
        assert top.item() == 0
        return
    for n in (64, 130, 1536):
        check(rq, t, n, "f32", absmax=True)


def test_largest_magnitude_feeds_the_quantization(rq):
    g = ref.gen(3)
    t, n = 40, 512
    y, h = rows(g, t, n, "f32"), rows(g, t, n, "f32")
    x, ho = torch.empty_like(y), torch.empty_like(h)
    bits = torch.empty(2, dtype=torch.int32, device="cuda")
    rq.rq_residual_norm(rq.NormParams(n), y, h, ho, x, t, absmax_bits=bits)
    rq.rq_absmax(x, x.numel(), bits[1:])
    assert bits[0].item() == bits[1].item()
    # NaNs are passed over by both
    y[3, 5] = float("nan")
    rq.rq_residual_norm(rq.NormParams(n), y, h, ho, x, t, absmax_bits=bits)
    rq.rq_absmax(x, x.numel(), bits[1:])
    assert bool(x[3].isnan().all()) and not bool(x[2].isnan().any())
    assert bits[0].item() == bits[1].item()


def test_in_place(rq):
    g = ref.gen(4)
    for t, n in ((1, 3584), (70, 1001)):
        y, h = rows(g, t, n, "bf16"), rows(g, t, n, "f32")
        p = rq.NormParams(n, scale=0.5)
        ho, x = torch.empty_like(h), torch.empty_like(y)
        rq.rq_residual_norm(p, y, h, ho, x, t)
        rq.rq_residual_norm(p, y, h, h, y, t)
        assert torch.equal(h, ho) and torch.equal(y, x)


def test_rows_of_zeros_and_infinities(rq):
    n = 256
    y, h = torch.zeros(3, n, device="cuda"), torch.zeros(3, n, device="cuda")
    h[1, 7] = float("inf")
    ho, x = torch.empty_like(h), torch.empty_like(y)
    rq.rq_residual_norm(rq.NormParams(n), y, h, ho, x, 3)
    assert torch.equal(ho, h)
    assert bool((x[0] == 0).all()) and bool((x[2] == 0).all())
    assert bool(x[1, 7].isnan())  # infinity over infinity


def test_rows_behind_the_last_are_left(rq):
    g = ref.gen(5)
    y, h = rows(g, 6, 96, "f32"), rows(g, 6, 96, "f32")
    ho, x = torch.full_like(h, 7.0), torch.full_like(y, 7.0)
    rq.rq_residual_norm(rq.NormParams(96), y, h, ho, x, 5)
    assert bool((ho[5] == 7).all()) and bool((x[5] == 7).all())
    assert not bool((ho[4] == 7).any())


def test_equal_calls_give_equal_bits_in_a_graph_and_on_a_stream(rq):
    g = ref.gen(6)
    y, h = rows(g, 33, 2048, "f32"), rows(g, 33, 2048, "f32")
    p = rq.NormParams(2048)
    outs = [(torch.empty_like(h), torch.empty_like(y),
             torch.empty(1, dtype=torch.int32, device="cuda")) for _ in range(3)]
    rq.rq_residual_norm(p, y, h, outs[0][0], outs[0][1], 33, absmax_bits=outs[0][2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    rq.rq_residual_norm(p, y, h, outs[1][0], outs[1][1], 33, absmax_bits=outs[1][2], stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.rq_residual_norm(p, y, h, outs[2][0], outs[2][1], 33, absmax_bits=outs[2][2])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    assert np.isfinite(outs[0][1].cpu().numpy()).all()
