"""GPU: verification of drafted tokens against an integer restatement, exactly,
and the distribution that it leaves."""
import numpy as np
import pytest
import torch

from serving_util import gen, verify_chain, verify_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rq():
    import quantized_linear_layers_gb300 as rq
    return rq


def run_chain(rq, tok, p, q, u):
    b, n = u.shape[0], u.shape[1] - 1
    acc = torch.full((b + 2,), 77, dtype=torch.int32, device="cuda")
    nxt = torch.full((b + 2,), 77, dtype=torch.int32, device="cuda")
    rq.rq_verify_chain(tok.cuda() if n else None, p.cuda(), None if q is None else q.cuda(),
                       u.cuda(), acc[1:-1], nxt[1:-1], b, n, p.shape[-1])
    for x in (acc, nxt):
        assert int(x[0]) == 77 and int(x[-1]) == 77
    return acc[1:-1].cpu().tolist(), nxt[1:-1].cpu().tolist()


def chain_inputs(seed, b, n, v, sharp=2.0):
    g = gen(seed)
    lq = sharp * torch.randn((b, n + 1, v), generator=g)
    q = torch.softmax(lq, -1)[:, :n].contiguous()
    p = torch.softmax(lq + 0.5 * torch.randn(lq.shape, generator=g), -1)
    tok = torch.multinomial(q.view(b * n, v), 1, generator=g).view(b, n).int() if n else \
        torch.zeros((b, 0), dtype=torch.int32)
    return tok, p, q, torch.rand((b, n + 1), generator=g)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("b,n,v", [(1, 0, 1), (3, 0, 50), (5, 1, 2), (4, 3, 31), (2, 7, 4097),
                                   (6, 5, 33333), (1, 600, 100), (2, 4, 65536)])
def test_chains(rq, b, n, v, drawn):
    tok, p, q, u = chain_inputs(b + n + v, b, n, v)
    got = run_chain(rq, tok, p, q if drawn else None, u)
    want = [verify_chain(tok[i].numpy(), p[i].numpy(), q[i].numpy() if drawn else None,
                         u[i].numpy()) for i in range(b)]
    assert list(zip(*got)) == want


def test_chain_corners(rq):
    v = 77
    tok, p, q, u = chain_inputs(1, 12, 4, v)
    u[0, :] = 0.0                                    # keeps all; first token with weight
    u[1, :] = 1.0 - 2.0 ** -24                       # last unit of the last draw
    tok[2, 1], tok[3, 0] = -1, v                     # chains that end early
    p[4, 0, int(tok[4, 0])] = 0.0                    # surely rejected
    q[5, 0], p[5, 0] = p[5, 0].clone(), p[5, 0]
    u[5, 0] = 1.0                                    # rejected where p == q: falls back to p
    p[6, 0] = 0.0                                    # no weight at all
    p[7, 0] = 0.0
    p[7, 0, 40] = 1.0                                # one-hot target
    u[7, 0] = 0.999
    p[8, 0, 5] = float("nan")
    q[9, 0, 7] = float("inf")
    u[10, 4], u[10, 0] = float("nan"), 0.99999
    p[11] *= 2.0 ** -40                              # below the draw's unit
    got = run_chain(rq, tok, p, q, u)
    want = [verify_chain(tok[i].numpy(), p[i].numpy(), q[i].numpy(), u[i].numpy())
            for i in range(12)]
    assert list(zip(*got)) == want
    got = run_chain(rq, tok, p, None, u)
    want = [verify_chain(tok[i].numpy(), p[i].numpy(), None, u[i].numpy()) for i in range(12)]
    assert list(zip(*got)) == want


def run_tree(rq, tok, par, p, u):
    b, n = tok.shape
    acc = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    nxt = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    path = torch.full((b * n + 2,), 77, dtype=torch.int32, device="cuda")
    inner = path[1:-1].view(b, n)
    rq.rq_verify_tree(tok.cuda(), par.cuda(), p.cuda(), u.cuda(), acc, nxt, inner, b, n,
                      p.shape[-1])
    assert int(path[0]) == 77 and int(path[-1]) == 77
    return acc.cpu().tolist(), nxt.cpu().tolist(), inner.cpu().tolist()


@pytest.mark.parametrize("b,n,v", [(1, 1, 2), (3, 12, 5), (4, 64, 300), (2, 40, 20011),
                                   (1, 1024, 3), (5, 7, 1)])
def test_trees(rq, b, n, v):
    g = gen(n + v)
    p = torch.softmax(2 * torch.randn((b, n + 1, v), generator=g), -1)
    u = torch.rand((b, n + 1), generator=g)
    par = torch.stack([torch.tensor([int(torch.randint(-1, max(i, 1), (1,), generator=g)) if i else -1
                                     for i in range(n)]) for _ in range(b)]).int()
    top = p.topk(min(3, v), -1).indices
    pick = torch.randint(0, min(3, v), (b, n), generator=g)
    tok = torch.stack([top[i, par[i].long() + 1, pick[i]] for i in range(b)]).int()
    if n > 6:
        tok[0, 2], par[0, 3], par[0, 5] = -1, 3, -2          # a pad, and two bad parents
    acc, nxt, path = run_tree(rq, tok, par, p, u)
    some = 0
    for i in range(b):
        clean = [x if -1 <= x < j else -3 for j, x in enumerate(par[i].tolist())]
        want, y = verify_tree(tok[i].tolist(), clean, p[i].numpy(), u[i].numpy())
        assert nxt[i] == y and acc[i] == len(want)
        assert path[i] == want + [-1] * (n - len(want))
        some += len(want)
    if n == 64:                     # 4 x 64 likely drafts among 300 tokens
        assert some > 0


def test_a_sharp_tree_is_walked_to_its_leaves(rq):
    """Likely drafts of a sharp target over an odd, large vocabulary."""
    b, n, v = 3, 39, 20011
    g = gen(1)
    p = torch.softmax(12 * torch.randn((b, n + 1, v), generator=g), -1)
    u = torch.rand((b, n + 1), generator=g)
    par = torch.tensor([i // 3 - 1 for i in range(n)]).int().repeat(b, 1)
    top = p.topk(3, -1).indices
    tok = torch.stack([top[i, par[i].long() + 1, torch.arange(n) % 3] for i in range(b)]).int()
    acc, nxt, path = run_tree(rq, tok, par, p, u)
    for i in range(b):
        want, y = verify_tree(tok[i].tolist(), par[i].tolist(), p[i].numpy(), u[i].numpy())
        assert (acc[i], nxt[i], path[i]) == (len(want), y, want + [-1] * (n - len(want)))


def test_tree_without_drafts(rq):
    p = torch.softmax(torch.randn((2, 1, 40)), -1).cuda()
    u = torch.rand((2, 1)).cuda()
    acc, nxt = (torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2))
    rq.rq_verify_tree(None, None, p, u, acc, nxt, None, 2, 0, 40)
    want = run_chain(rq, torch.zeros((2, 0), dtype=torch.int32), p.cpu(), None, u.cpu())
    assert (acc.tolist(), nxt.tolist()) == want


@pytest.mark.parametrize("kind", ["drawn", "fixed", "tree"])
def test_first_token_is_distributed_as_the_target(rq, kind):
    """50000 sequences: the first token that comes out has the target's
    probabilities (chi-square of 7 degrees of freedom, below 40: 1e-6)."""
    b, v = 50000, 8
    g = gen(2)
    p1 = torch.softmax(torch.randn(v, generator=g), -1)
    q1 = torch.softmax(torch.randn(v, generator=g), -1)
    u = torch.rand((b, 3), generator=g)
    p = p1.repeat(b, 3, 1).contiguous()
    if kind == "tree":
        tok = torch.tensor([[2, 5]], dtype=torch.int32).repeat(b, 1)
        par = torch.full((b, 2), -1, dtype=torch.int32)
        acc, nxt, path = run_tree(rq, tok, par, p, u)
        path = torch.tensor(path)[:, 0].long()
        first = torch.where(path >= 0, tok[:, :].long().gather(1, path.clamp_min(0)[:, None])[:, 0],
                            torch.tensor(nxt).long())
    else:
        q = q1.repeat(b, 2, 1).contiguous()
        tok = torch.multinomial(q1.repeat(b, 1), 2, replacement=True, generator=g).int()
        if kind == "fixed":
            tok = torch.tensor([[3, 3]], dtype=torch.int32).repeat(b, 1)
            q = None
        acc, nxt = run_chain(rq, tok, p, q, u)
        first = torch.where(torch.tensor(acc) > 0, tok[:, 0].long(), torch.tensor(nxt).long())
    seen = np.bincount(first.numpy(), minlength=v)
    want = p1.double().numpy() * b
    assert ((seen - want) ** 2 / want).sum() < 40
