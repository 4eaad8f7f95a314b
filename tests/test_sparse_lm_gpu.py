"""The example language model: one training step against the same model written
densely in 64 bits, and a short training run with rewiring.

Tolerance of the step: every sum of the library is within 1e-5 of its terms'
magnitudes, and a gradient passes through at most six of them (projection,
softmax, its product, two sparse layers, the table's sum), with magnitudes at
most some tens of times the result's: updates agree to 1e-3 of the largest
update of their tensor, far below what a wrong or missing term would change.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_lm.py")


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("sparse_lm", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def dense(layer):
    w = torch.zeros(layer.out_f, layer.in_f, dtype=torch.float64, device="cuda")
    w[layer.row.long(), layer.col.long()] = layer.val.double()
    return w


def test_step_matches_a_dense_model_in_64_bits(lm):
    vocab, width, hidden, n = 157, 48, 96, 200
    model = lm.SparseLM(vocab, width, hidden, density=0.1, batch=n, seed=3)
    model.table.mul_(20.0)  # away from the uniform start, and enough gradient to be clipped
    ids = torch.from_numpy(lm.chain_text(vocab, n + 1, 1)).cuda()
    x_ids, targets = ids[:-1].clone(), ids[1:].clone()
    x_ids[5], targets[7] = -1, -100  # a padding token, and a position that is not trained on
    before = [t.double().clone() for t in (model.table, model.up.val, model.up.bias, model.down.val, model.down.bias)]
    table = before[0].clone().requires_grad_()
    up, down = dense(model.up).requires_grad_(), dense(model.down).requires_grad_()
    b_up, b_down = before[2].clone().requires_grad_(), before[4].clone().requires_grad_()
    x = table[x_ids.clamp(min=0)] * (x_ids >= 0)[:, None] * model.scale
    y = x + torch.nn.functional.gelu(x @ up.T + b_up) @ down.T + b_down
    want = torch.nn.functional.cross_entropy(y @ table.T, targets, ignore_index=-100)
    want.backward()
    grads = [table.grad, up.grad[model.up.row.long(), model.up.col.long()], b_up.grad,
             down.grad[model.down.row.long(), model.down.col.long()], b_down.grad]
    want_norm = float(torch.sqrt(sum((g ** 2).sum() for g in grads)))
    max_norm = want_norm / 3
    loss, norm = model.step(x_ids, targets, lr=0.5, max_norm=max_norm)
    assert abs(float(loss) - want.item()) <= 1e-5 * want.item()
    assert abs(float(norm) - want_norm) <= 1e-3 * want_norm
    after = (model.table, model.up.val, model.up.bias, model.down.val, model.down.bias)
    for b, a, g in zip(before, after, grads):
        update = 0.5 * g / 3
        # and the rounding of the updated parameter itself
        tol = 1e-3 * update.abs().max() + 2.0 ** -23 * b.abs().max()
        assert float((a.double() - (b - update)).abs().max()) <= float(tol)
    model.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_learns_the_chain(lm, dtype):
    losses = lm.train(steps=150, vocab=120, width=64, hidden=128, density=0.15, batch=512, rewire=60, dtype=dtype, seed=1)
    assert np.isfinite(losses).all()
    assert abs(losses[0] - np.log(120)) < 0.5
    assert np.mean(losses[-10:]) < 0.7 * losses[0]
