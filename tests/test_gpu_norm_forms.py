"""GPU: every kernel form that widths and numbers of tokens choose, with a gate of
each channel and without, on dense rows of odd widths and on rows apart."""
import pytest
import torch

import pass_util as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def check(rq, t, n, dtype, h_dtype, gate, stride=None):
    g = ref.gen(t + 7 * n)

    def rows(kind):
        wide = torch.zeros(t, stride or n)
        wide[:, :n] = torch.randn(t, n, generator=g)
        return wide.to(ref.DTYPES[kind]).cuda()[:, :n]

    y, h = rows(dtype), rows(h_dtype)
    wp, wq = (1 + 0.2 * torch.randn(n, generator=g).cuda() for _ in range(2))
    gates = None
    if gate == "channel":
        gates = torch.randn(n, generator=g).to(ref.DTYPES[dtype]).cuda()
    elif gate == "token":
        gates = rows(dtype)
    # (rows behind the last stay as they were)
    ho = torch.full((t + 1, n), 9.0, dtype=h.dtype, device="cuda")
    xo = torch.full((t + 1, n), 9.0, dtype=y.dtype, device="cuda")
    p = rq.NormParams(n, post_weight=wp, pre_weight=wq, eps=EPS, scale=0.7)
    rq.rq_residual_norm(p, y, h, ho[:t], xo[:t], t, gate=gates)
    cpu = [None if v is None else v.cpu() for v in (y, h, wp, wq, gates)]
    H, X, eh, ex = ref.norm(cpu[0], cpu[1], True, True, cpu[2], cpu[3], cpu[4], 0.7, EPS, n)
    for got, want, e in ((ho, H, eh), (xo, X, ex)):
        tol = e + ref.ROUND[got.dtype] * (want.abs() + e) + ref.TINY[got.dtype]
        assert bool(((got[:t].double().cpu() - want).abs() <= tol).all())
        assert bool((got[t] == 9).all())


TYPES = [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")]


@pytest.mark.parametrize("dtype,h_dtype", TYPES)
@pytest.mark.parametrize("t", [3, 400])
@pytest.mark.parametrize("n", [31, 33, 129, 515, 1025, 2051, 4099, 8195, 16371])
def test_odd_widths_with_a_gate_of_each_channel(rq, n, t, dtype, h_dtype):
    # 400 tokens are more than twice the SMs: several groups a thread
    check(rq, t, n, dtype, h_dtype, "channel")


@pytest.mark.parametrize("dtype,h_dtype", TYPES)
@pytest.mark.parametrize("t", [2, 400])
@pytest.mark.parametrize("n", [16, 100, 200, 1000, 1030, 2000, 3000, 5000, 9000, 16384])
def test_rows_apart_of_every_number_of_groups(rq, n, t, dtype, h_dtype):
    # at an odd distance: one element at a time, 1 to 16 a thread
    check(rq, t, n, dtype, h_dtype, "token" if n % 16 else "channel", stride=n + 3)


@pytest.mark.parametrize("dtype,h_dtype", TYPES)
@pytest.mark.parametrize("n", [128, 256, 512, 1024, 4096, 4104, 8192, 16384])
def test_aligned_widths_with_a_gate_of_each_channel(rq, n, dtype, h_dtype):
    for t in (2, 400):
        check(rq, t, n, dtype, h_dtype, "channel")
