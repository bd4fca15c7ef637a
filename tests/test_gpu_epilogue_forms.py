"""GPU: what the epilogue's callers may rely on besides its sums: rows that are
rewritten in place are read anew."""
import pytest
import torch

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
