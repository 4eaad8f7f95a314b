"""Adapters and scores as they are used together: adapters of a sparse layer trained by a policy gradient, and served.

Tolerance of the training step: every sum of the library is within 1e-5 of its terms' magnitudes, and a gradient passes
through at most six of them (logits, softmax, its product, the adapter's two, the sparse layer), with magnitudes at most some
tens of times the result's: gradients agree to 1e-3 of the largest of their tensor, far below what a wrong or missing term
would change.
"""

import threading

import pytest
import torch

from spmm_row_sorted_gb300 import snack
from spmm_row_sorted_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

WIDTH, VOCAB, RANK, ADAPTERS = 80, 331, 8, 4


class Model:
    def __init__(self, n, seed):
        lay = wl.make_layer(WIDTH, WIDTH, density=0.2, val_std=0.2, seed=seed)
        row, col, val = (torch.from_numpy(t).cuda() for t in (lay.row, lay.col, lay.val))
        self.bias = torch.linspace(-0.5, 0.5, WIDTH, device="cuda")
        self.layer = snack.SparseLinear(WIDTH, WIDTH, row, col, val, self.bias, max_batch=n)
        self.dense = torch.zeros(WIDTH, WIDTH, dtype=torch.float64, device="cuda")
        self.dense[row.long(), col.long()] = val.double()
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=g)

        self.x, self.w = normal(n, WIDTH), normal(VOCAB, WIDTH, std=0.4)
        self.a, self.b = normal(ADAPTERS, RANK, WIDTH, std=WIDTH ** -0.5), normal(ADAPTERS, WIDTH, RANK, std=RANK ** -0.5)
        self.scales = torch.linspace(0.5, 2.0, ADAPTERS, device="cuda")
        self.which = torch.randint(-1, ADAPTERS, (n,), device="cuda", generator=g)
        self.targets = torch.randint(0, VOCAB, (n,), device="cuda", generator=g)
        self.targets[3::11] = -100
        self.advantage = normal(n)

    def hidden64(self, x, a, b):
        y = x @ self.dense.T + self.bias.double()
        rows = []
        for i, k in enumerate(self.which.tolist()):
            rows.append(y[i] if k < 0 else y[i] + self.scales[k].double() * (b[k] @ (a[k] @ x[i])))
        return torch.stack(rows)


@pytest.mark.parametrize("n", [7, 150, 400])
def test_a_policy_gradient_of_adapters(n):
    m = Model(n, seed=n)
    beta = 0.05
    want = [t.double().requires_grad_() for t in (m.x, m.a, m.b, m.w)]
    log_p = torch.log_softmax(m.hidden64(*want[:3]) @ want[3].T, 1)
    scored = m.targets >= 0
    logp = log_p[torch.arange(n, device="cuda"), m.targets.clamp(min=0)]
    entropy = -(log_p.exp() * log_p).sum(1)
    (-(m.advantage.double() * logp + beta * entropy)[scored].sum()).backward()

    leaves = [t.clone().requires_grad_() for t in (m.x, m.a, m.b, m.w)]
    hidden = snack.adapted(leaves[0], snack.sparse_linear(leaves[0], m.layer), leaves[1], leaves[2], m.which, m.scales)
    got_logp, got_entropy = snack.token_logprobs(hidden, leaves[3], m.targets)
    (-(m.advantage * got_logp + beta * got_entropy).sum()).backward()

    assert bool(((got_logp.double() - logp)[scored].abs() <= 1e-3).all()) and bool((got_logp[~scored] == 0).all())
    assert bool(((got_entropy.double() - entropy)[scored].abs() <= 1e-3).all()) and bool((got_entropy[~scored] == 0).all())
    for leaf, w in zip(leaves, want):
        assert float((leaf.grad.double() - w.grad).abs().max()) <= 1e-3 * float(w.grad.abs().max())
    m.layer.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_serving_picks_the_likeliest_tokens_and_replays(dtype):
    n, top = 40, 5
    m = Model(n, seed=2)
    x, w, a, b = (t.to(dtype) for t in (m.x, m.w, m.a, m.b))
    base = torch.empty(n, WIDTH, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)

    def step():
        hidden = snack.adapt(x, base, a, b, m.which, m.scales)
        return (hidden, *snack.score(hidden, w, top=top)[1:4])

    hidden, entropy, ids, top_logp = step()
    z = hidden.double() @ w.double().T
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(ids, order)
    log_p = torch.log_softmax(z, 1)
    assert bool(((top_logp.double() - log_p.gather(1, order)).abs() <= 1e-3).all())
    assert bool(((entropy.double() + (log_p.exp() * log_p).sum(1)).abs() <= 1e-3).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    m.which.copy_(m.which.flip(0))
    x.mul_(-1)
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(held, step()))
    m.layer.close()


def in_a_new_thread(call):
    out = []

    def run():
        try:
            out.append(call())
        except Exception as e:  # handed on to the test
            out.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if isinstance(out[0], Exception):
        raise out[0]
    return out[0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_calls_from_a_host_thread_of_their_own(dtype):
    """A thread's first call of CUDA, too: a server's threads start with any of them."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(r, 96, device="cuda", generator=g).to(dtype) for r in (200, 3000))
    t = torch.randint(0, 3000, (200,), device="cuda", generator=g)
    a, b = torch.randn(3, 8, 96, device="cuda", generator=g).to(dtype), torch.randn(3, 96, 8, device="cuda", generator=g).to(dtype)
    which = torch.randint(0, 3, (200,), device="cuda", generator=g)  # rows without one leave their h as it was
    up = torch.randn(200, device="cuda", generator=g)
    y, h = snack.adapt(x, x, a, b, which, keep=True)
    scored = snack.score(x, w, t, top=3)
    kept = snack.xent(x, w, t)
    calls = (lambda: snack.adapt(x, x, a, b, which, keep=True), lambda: snack.adapt_grad(x, x, a, b, which, h),
             lambda: snack.score(x, w, t, top=3), lambda: snack.score_grad(x, w, t, scored[4], up, up),
             lambda: snack.xent(x, w, t), lambda: snack.xent_grad(x, w, t, kept[1]))
    for call in calls:
        for p, q in zip(in_a_new_thread(call), call()):
            assert torch.equal(p, q)
