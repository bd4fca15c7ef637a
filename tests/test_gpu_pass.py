"""GPU: a pass's steps run together, as a serving loop uses them."""
import importlib.util
import os

import pytest
import torch

import pass_util as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Serving:
    """Three sequences through one layer and a vocabulary, a token each a pass:
    plan, norm, q/k/v, cache, attention, product onto the stream, norm,
    logits, draw.  The pass reads and writes fixed tensors only."""

    HIDDEN, HEADS, KV, D, VOCAB, PAGE, BATCH = 512, 4, 2, 128, 300, 16, 3

    def __init__(self, rq):
        import synthetic
        self.rq, self.ctx = rq, rq.Context()
        h, q, kv = self.HIDDEN, self.HEADS * self.D, self.KV * self.D

        def weight(seed, qtype, n, k):
            return torch.from_numpy(
                synthetic.weight_matrix(seed, qtype, n, k).view("uint8").reshape(-1).copy()).cuda()

        self.wq = [weight(1, rq.RQ_Q4K, q, h), weight(2, rq.RQ_Q4K, kv, h),
                   weight(3, rq.RQ_Q6K, kv, h)]
        self.wo, self.head = weight(4, rq.RQ_Q4K, h, q), weight(5, rq.RQ_Q6K, self.VOCAB, h)
        g = ref.gen(1)
        self.embedding = torch.randn(self.VOCAB, h, generator=g).cuda()
        self.cache = rq.KVCache(24, self.PAGE, self.KV, self.D)
        self.params = rq.QKParams(self.HEADS, self.KV, self.D)
        self.norm = rq.NormParams(h, post=False)
        self.free = torch.randperm(24, generator=g).int().cuda()
        b = self.BATCH

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device="cuda")

        self.table, self.position = i32(b, 8), i32(b)
        self.slot = torch.zeros(b, dtype=torch.int64, device="cuda")
        self.length, self.following = i32(b), i32(b)
        self.count, self.left = i32(1), i32(1)
        self.count += 24
        self.token = i32(b)
        self.token += torch.tensor([5, 6, 7], device="cuda", dtype=torch.int32)
        self.u = torch.zeros(b, device="cuda")
        self.temperature = torch.tensor([0.7, 1.0, 0.0], device="cuda")
        self.top_k = torch.tensor([40, 0, 0], dtype=torch.int32, device="cuda")
        self.top_p = torch.tensor([0.9, 0.8, 1.0], device="cuda")
        f = lambda n: torch.empty(b, n, device="cuda")  # noqa: E731
        self.x, self.normed, self.out, self.logits = f(h), f(h), f(q), f(self.VOCAB)
        self.qkv = [f(q), f(kv), f(kv)]

    def run(self):
        rq, b, h = self.rq, self.BATCH, self.HIDDEN
        torch.index_select(self.embedding, 0, self.token, out=self.x)
        rq.rq_batch_plan(self.length, self.table, self.free, self.count, self.left, self.slot,
                         self.position, self.PAGE, new_tokens=1, next_length=self.following)
        rq.rq_residual_norm(self.norm, None, self.x, None, self.normed, b)
        self.ctx.rq_linear_group([rq.RQ_Q4K, rq.RQ_Q4K, rq.RQ_Q6K], self.wq, self.normed, self.qkv,
                                 [t.shape[1] for t in self.qkv], b, h)
        q, k, v = (t.view(b, -1, self.D) for t in self.qkv)
        rq.rq_qkv_to_cache(self.params, q, k, v, self.position, q, self.cache, self.slot, b)
        self.ctx.rq_cache_attention(self.cache, q, self.out.view_as(q), self.table, self.length, b, 1,
                                    self.HEADS, self.D ** -0.5)
        self.ctx.rq_act_cache_invalidate()
        self.ctx.rq_linear_epilogue(rq.RQ_Q4K, self.wo, self.out, self.x, b, h, self.out.shape[1],
                                    residual=self.x)
        rq.rq_residual_norm(self.norm, None, self.x, None, self.normed, b)
        self.ctx.rq_linear(rq.RQ_Q6K, self.head, self.normed, self.logits, b, self.VOCAB, h)
        rq.rq_sample(self.logits, self.u, self.token, b, self.VOCAB, temperature=self.temperature,
                     top_k=self.top_k, top_p=self.top_p)
        self.length.copy_(self.following)
        self.count.copy_(self.left)


def texts(rq, captured, passes=40):
    s = Serving(rq)
    graph = None
    rows = []
    g = ref.gen(2)
    for i in range(passes):
        s.u.copy_(torch.rand(3, generator=g))
        if not captured or i < 2:
            s.run()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    s.run()
            graph.replay()
        rows.append(s.token.tolist())
    assert rq.rq_get_device_status() == 0
    assert s.length.tolist() == [passes] * 3
    held = -(-passes // 16)
    assert s.count.tolist() == [24 - 3 * held]
    used = s.table[:, :held].flatten().tolist()
    assert len(set(used)) == len(used)
    s.ctx.close()
    return rows


def test_a_captured_serving_loop_writes_the_same_texts(rq):
    eager = texts(rq, False)
    assert texts(rq, True) == eager
    assert texts(rq, False) == eager
    assert all(0 <= t < 300 for row in eager for t in row)


@pytest.mark.parametrize("filters", [dict(top_p=0.8), dict(top_k=5), dict(min_p=0.1),
                                     dict(top_k=40, top_p=0.9, min_p=0.01)])
def test_filtered_drafts_do_not_change_the_text(example, filters):
    prompt = [3, 141, 59, 26, 53, 3, 141, 59]
    plain, passes = example.generate(example.Decoder(), prompt, 48, "none", temperature=0.7,
                                     **filters)
    assert passes == 48
    text, fewer = example.generate(example.Decoder(), prompt, 48, "tree", temperature=0.7, **filters)
    assert text == plain and fewer <= passes


def test_a_long_prompt_takes_the_fused_product(example):
    # 100 tokens at once go by the FP8 route, gate with its epilogue
    g = ref.gen(3)
    prompt = torch.randint(0, 512, (101,), generator=g).tolist()
    text, passes = example.generate(example.Decoder(), prompt, 8, "none", temperature=0.5)
    again, _ = example.generate(example.Decoder(), prompt, 8, "none", temperature=0.5)
    assert text == again and passes == 8 and all(0 <= t < 512 for t in text)
