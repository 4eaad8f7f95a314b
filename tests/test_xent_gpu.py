"""Softmax cross entropy of a vocabulary projection, and its gradient, against
the definitions in 64 bits.

Tolerances, from the kernels' arithmetic.  A logit is a sum in fp32 of exact
products (bf16 operands; fp32 ones as parts that leave out less than 2^-23 of
a product): |err z| <= A T with A = 1e-5, the bound of every fp32 sum of this
library, and T the largest sum of magnitudes of the row.  The log of the sum
moves by at most the largest err z, plus the errors of 2^x (2^-21) and of the
sums (2^-17 over thousands of terms): |err loss| <= 2 A T + 2^-16 + 2^-22 |lse|.
With e = 2 A T + 2^-16 the relative error of a probability, dz is within
g (p e + the rounding to bf16, 2^-8 (p + [v = t])) for bf16 operands and within
g (e p + 2^-22 (p + [v = t])) for fp32 ones.  A product's sum adds A of its
magnitudes, and a bf16 output half an ulp.  E below is the sum over the
magnitudes g (p + [v = t]) |w| (or |x|).
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from spmm_row_sorted_gb300 import snack

from gpu_util import bf16_half_ulp, f64

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
A = 1e-5


def make(n, vocab, width, dtype, seed, gap=0, lead=0, ignored=0.1, itype=torch.int64, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def matrix(rows, std):
        buf = torch.full((rows * (width + gap) + lead,), float("nan"), device="cuda", dtype=DTYPES[dtype])
        m = buf[lead:].view(rows, width + gap)[:, :width]
        m.copy_(torch.empty(rows, width, device="cuda").normal_(0, std, generator=g))
        return m

    x, w = matrix(n, 1.0), matrix(vocab, spread / width ** 0.5)
    rng = np.random.default_rng(seed)
    t = rng.integers(0, vocab, n)
    t[rng.random(n) < ignored] = -100
    t[rng.random(n) < ignored / 4] = vocab
    if n > 1:
        t[0], t[-1] = 0, vocab - 1
    return x, w, torch.from_numpy(t).to(itype).cuda()


def reference(x, w, t, g):
    """loss per row, dx, dw and their magnitudes for per-row weights g (zero where not trained on)."""
    x, w, t = f64(x), f64(w), t.cpu().numpy().astype(np.int64)
    inside = (t >= 0) & (t < w.shape[0])
    z = x @ w.T
    T = (np.abs(x) @ np.abs(w).T).max(1)
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    at = np.where(inside, t, 0)
    rows = np.arange(len(t))
    loss = np.where(inside, lse - z[rows, at], 0.0)
    p = np.exp(z - lse[:, None])
    g = np.where(inside, g, 0.0)[:, None]
    hot = np.zeros_like(z)
    hot[rows[inside], at[inside]] = 1.0
    dz, mag = g * (p - hot), np.abs(g) * (p + hot)
    return dict(loss=loss, lse=lse, T=T, inside=inside, dx=dz @ w, dw=dz.T @ x,
                # magnitudes, and the same weighted by each row's relative error of a probability
                ex=mag @ np.abs(w), ew=mag.T @ np.abs(x), e=2 * A * T + 2.0 ** -16,
                eew=(mag * (2 * A * T + 2.0 ** -16)[:, None]).T @ np.abs(x))


def check_loss(loss, r):
    assert np.all(np.abs(f64(loss) - r["loss"]) <= 2 * A * r["T"] + 2.0 ** -16 + 2.0 ** -22 * np.abs(r["lse"]))
    assert not np.any(f64(loss)[~r["inside"]])


def check_grads(dx, dw, r, dtype):
    round_dz = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
    for got, ref, bound in ((dx, r["dx"], (r["e"][:, None] + round_dz + A) * r["ex"]),
                            (dw, r["dw"], r["eew"] + (round_dz + A) * r["ew"])):
        if got is None:
            continue
        if dtype == "bf16":
            bound = bound + bf16_half_ulp(np.abs(ref) + bound)
        assert np.all(np.abs(f64(got) - ref) <= bound + 1e-300)


SHAPES = [
    # n, vocab, width, gap, lead
    (1, 1, 1, 0, 0),
    (1, 2, 8, 0, 0),
    (1, 5000, 64, 0, 0),
    (3, 257, 16, 0, 0),
    (16, 1000, 128, 0, 0),
    (31, 129, 72, 0, 0),
    (127, 513, 65, 0, 0),      # rows that are laid out again
    (128, 512, 64, 0, 0),      # whole tiles
    (129, 511, 192, 0, 0),
    (200, 700, 100, 4, 0),     # 16-byte aligned rows with gaps for fp32, not for bf16
    (200, 700, 96, 8, 8),
    (200, 700, 96, 0, 1),      # off a 16-byte boundary
    (300, 4000, 320, 0, 0),
    (64, 40000, 40, 0, 0),     # wide tiles
    (1030, 3001, 259, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,width,gap,lead", SHAPES)
def test_xent_matches_definition(n, vocab, width, gap, lead, dtype):
    x, w, t = make(n, vocab, width, dtype, seed=n + vocab, gap=gap, lead=lead, itype=torch.int32 if n % 2 else torch.int64)
    rng = np.random.default_rng(n)
    dloss = torch.from_numpy(rng.normal(size=n).astype(np.float32)).cuda()
    r = reference(x, w, t, dloss.cpu().numpy().astype(np.float64))
    loss, state = snack.xent(x, w, t, reduction="none")
    check_loss(loss, r)
    dx, dw = snack.xent_grad(x, w, t, state, dloss, reduction="none")
    check_grads(dx, dw, r, dtype)
    assert not np.any(f64(dx)[~r["inside"]])
    again = snack.xent_grad(x, w, t, snack.xent(x, w, t, reduction="none")[1], dloss, reduction="none")
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])  # repeats bit for bit
    only_x, none_w = snack.xent_grad(x, w, t, state, dloss, reduction="none", want_dw=False)
    none_x, only_w = snack.xent_grad(x, w, t, state, dloss, reduction="none", want_dx=False)
    assert none_w is None and none_x is None and torch.equal(only_x, dx) and torch.equal(only_w, dw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
def test_xent_reductions(reduction, dtype):
    x, w, t = make(150, 900, 128, dtype, seed=4)
    inside = ((t >= 0) & (t < 900)).cpu().numpy()
    scale = 1.0 if reduction == "sum" else 1.0 / inside.sum()
    up = torch.tensor(0.3, device="cuda")
    r = reference(x, w, t, np.full(150, 0.3 * scale))
    loss, state = snack.xent(x, w, t, reduction=reduction)
    tol = (2 * A * r["T"] + 2.0 ** -16 + 2.0 ** -22 * np.abs(r["lse"]))[inside].sum() * scale
    want = r["loss"].sum() * scale
    assert loss.shape == () and abs(float(loss) - want) <= tol + 2.0 ** -23 * abs(want)
    dx, dw = snack.xent_grad(x, w, t, state, up, reduction=reduction)
    check_grads(dx, dw, r, dtype)
    if reduction == "mean":  # no upstream gradient: 1
        r1 = reference(x, w, t, np.full(150, scale))
        check_grads(*snack.xent_grad(x, w, t, state, reduction=reduction), r1, dtype)


def test_xent_nothing_to_train_on():
    x, w, t = make(40, 300, 64, "bf16", seed=6)
    t[:] = -100
    loss, state = snack.xent(x, w, t)
    assert float(loss) == 0.0
    dx, dw = snack.xent_grad(x, w, t, state)
    assert not dx.any() and not dw.any()
    loss, state = snack.xent(x[:0], w, t[:0])
    assert float(loss) == 0.0
    dx, dw = snack.xent_grad(x[:0], w, t[:0], state)
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_large_logits(dtype):
    """Logits of several hundred, of both signs: exponentials of the differences only."""
    x, w, t = make(70, 800, 64, dtype, seed=8, spread=200.0)
    r = reference(x, w, t, np.ones(70))
    loss, state = snack.xent(x, w, t, reduction="none")
    check_loss(loss, r)
    assert np.isfinite(f64(loss)).all()
    dx, dw = snack.xent_grad(x, w, t, state, reduction="sum")
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    w32 = w.clone()
    w32[:] = w[0]  # equal logits
    loss, _ = snack.xent(x, w32, t, reduction="none")
    inside = r["inside"]
    assert np.allclose(f64(loss)[inside], np.log(800.0), rtol=0, atol=2e-4)


def test_xent_not_finite_rows_stay_apart():
    x, w, t = make(140, 600, 64, "bf16", seed=9, ignored=0.0)
    clean, _ = snack.xent(x, w, t, reduction="none")
    bad = x.clone()
    bad[5, 3] = float("nan")
    bad[77, 0] = float("inf")
    loss, state = snack.xent(bad, w, t, reduction="none")
    assert torch.isnan(loss[5]) and torch.isnan(loss[77])
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[5] = keep[77] = False
    assert torch.equal(loss[keep], clean[keep])
    t2 = t.clone()
    t2[5] = t2[77] = -100  # not trained on: their dx is zero, the other rows' as before
    loss, state = snack.xent(bad, w, t2, reduction="none")
    assert float(loss[5]) == 0.0 and float(loss[77]) == 0.0
    ones = torch.ones(140, device="cuda")
    dx, _ = snack.xent_grad(bad, w, t2, state, ones, reduction="none", want_dw=False)
    want, _ = snack.xent_grad(x, w, t2, snack.xent(x, w, t2, reduction="none")[1], ones, reduction="none", want_dw=False)
    assert torch.equal(dx, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_rows_not_trained_on_may_hold_anything(dtype):
    x, w, t = make(140, 600, 72, dtype, seed=21, ignored=0.2)
    up = torch.rand(140, device="cuda") + 0.5
    up[3], t[3] = 0.0, 17  # a weight of zero leaves a row out too
    out = (t < 0) | (t >= 600)
    out[3] = True
    bad = x.clone()
    bad[out] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").repeat(24).to(x.dtype)
    loss, state = snack.xent(x, w, t, reduction="none")
    loss_bad, state_bad = snack.xent(bad, w, t, reduction="none")
    keep = ~out
    keep[3] = False
    assert torch.equal(loss[keep], loss_bad[keep])
    want = snack.xent_grad(x, w, t, state, up, reduction="none")
    got = snack.xent_grad(bad, w, t, state_bad, up, reduction="none")
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert not got[0][out].any()


def test_xent_in_pieces_of_the_vocabulary():
    """A workspace-bounded gradient: n * vocab large enough for several pieces of dz and of w's parts."""
    n, vocab, width = 8300, 40100, 64
    x, w, t = make(n, vocab, width, "bf16", seed=10)
    loss, state = snack.xent(x, w, t)
    dx, dw = snack.xent_grad(x, w, t, state)
    assert snack.snack_xent_workspace_size(x, w, True) < 2 * n * vocab  # less than dz whole
    # the first and last rows of x, and blocks of the vocabulary in every piece, against the definition
    inside = ((t >= 0) & (t < vocab)).cpu().numpy()
    scale = 1.0 / inside.sum()
    rows = np.r_[0:40, n - 40:n]
    r = reference(x[rows], w, t[rows], np.full(80, scale))
    check_grads(dx[rows], None, r, "bf16")
    zs = (x.float() @ w.float().T).double()
    lse = torch.logsumexp(zs, 1)
    p = torch.exp(zs - lse[:, None])
    del zs
    ok = torch.from_numpy(inside).cuda()
    p[ok, t[ok].long()] -= 1.0
    p *= ok[:, None] * scale
    ref = p.T @ x.double()
    mag = p.abs().T @ x.double().abs()
    T = float((x[:512].double().abs() @ w.double().abs().T).max()) * 1.5
    # p - 1 stands for p + 1 in the magnitudes: a factor of 1 + 2 p / (1 - p) <= 2 for p <= 1/3
    bound = 2 * (2 * A * T + 2.0 ** -16 + 2.0 ** -8 + 2 * A) * mag + 2.0 ** -8 * ref.abs() + 1e-12
    assert bool(((dw.double() - ref).abs() <= bound).all())


def test_linear_cross_entropy_autograd_matches_differences():
    n, vocab, width = 6, 11, 5
    x, w, t = make(n, vocab, width, "f32", seed=12)
    x, w = x.contiguous().requires_grad_(), w.contiguous().requires_grad_()
    (snack.linear_cross_entropy(x, w, t, reduction="sum") * 1.5).backward()
    h = 2.0 ** -6

    def loss(a, b):
        return 1.5 * float(snack.xent(a.detach(), b.detach(), t, reduction="sum")[0])

    # central differences: h^2 / 6 of a third derivative below 10 (softmax of logits with |x|, |w| < 4), and
    # 2^-22 of a loss below 64 over h
    for which in (x, w):
        for i in (0, which.numel() // 2, which.numel() - 1):
            lo, hi = which.detach().clone(), which.detach().clone()
            lo.view(-1)[i] -= h
            hi.view(-1)[i] += h
            pair = (loss(hi, w) - loss(lo, w)) if which is x else (loss(x, hi) - loss(x, lo))
            assert abs(pair / (2 * h) - float(which.grad.view(-1)[i])) < 10 * h * h / 6 * 1.5 + 64 * 2.0 ** -22 / h


def test_xent_on_another_stream():
    x, w, t = make(300, 2000, 128, "bf16", seed=14)
    loss, state = snack.xent(x, w, t)
    want = snack.xent_grad(x, w, t, state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l2, s2 = snack.xent(x, w, t, stream=side)
    got = snack.xent_grad(x, w, t, s2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(loss, l2) and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_xent_refusals():
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(10, 8, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    for args in ((x, w.bfloat16(), t), (x[:, :7], w, t), (x, w, t[:3]), (x.half(), w.half(), t), (x, w, t.float()),
                 (x.cpu(), w.cpu(), t.cpu()), (x, w, t.cpu())):
        with pytest.raises(ValueError):
            snack.xent(*args)
    with pytest.raises(ValueError):
        snack.xent(x, w, t, reduction="max")
    loss, state = snack.xent(x, w, t, reduction="none")
    with pytest.raises(ValueError):
        snack.xent_grad(x, w, t, state, reduction="none")  # no upstream gradient
    with pytest.raises(ValueError):
        snack.xent_grad(x, w, t, state[:4])
    with pytest.raises(ValueError):
        snack.xent_grad(x, w, t, state, torch.zeros(3, device="cuda"), reduction="none")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(snack.SnackError) as e:
        snack.snack_xent_fwd(x, w, t, 0, loss, state, ws)
    assert e.value.status == 4
    with pytest.raises(snack.SnackError) as e:  # dx on x
        snack.snack_xent_bwd(x, w, t, 1, state, None, x, None, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 1
    with pytest.raises(snack.SnackError) as e:
        snack.snack_xent_fwd(x, w, t, 7, loss, state, ws)
    assert e.value.status == 1


@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("n,vocab,width,gap,lead", [
    (1, 700, 513, 0, 0), (4, 64, 700, 0, 0), (5, 2100, 1100, 0, 0), (8, 129, 2050, 2, 2), (9, 1000, 128, 4, 0),
    (16, 333, 515, 0, 1), (17, 4097, 260, 0, 0), (32, 1000, 1030, 0, 0), (32, 65, 512, 0, 0),
])
def test_xent_few_fp32_tokens(n, vocab, width, gap, lead, reduction):
    x, w, t = make(n, vocab, width, "f32", seed=n * vocab, gap=gap, lead=lead, ignored=0.2 if n > 2 else 0.0)
    inside = ((t >= 0) & (t < vocab)).cpu().numpy()
    up = np.random.default_rng(n).normal(size=n).astype(np.float32)
    g = up.astype(np.float64) if reduction == "none" else np.full(n, 0.7 / max(1, inside.sum()))
    dloss = torch.from_numpy(up).cuda() if reduction == "none" else torch.tensor(0.7, device="cuda")
    r = reference(x, w, t, g)
    check_loss(snack.xent(x, w, t, reduction="none")[0], r)
    loss, state = snack.xent(x, w, t, reduction=reduction)
    dx, dw = snack.xent_grad(x, w, t, state, dloss, reduction=reduction)
    check_grads(dx, dw, r, "f32")
    only_x, _ = snack.xent_grad(x, w, t, state, dloss, reduction=reduction, want_dw=False)
    _, only_w = snack.xent_grad(x, w, t, state, dloss, reduction=reduction, want_dx=False)
    check_grads(only_x, only_w, r, "f32")
    again = snack.xent_grad(x, w, t, state, dloss, reduction=reduction)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("n,vocab,width,dtype", [(20, 3000, 129, "bf16"), (40, 700, 130, "bf16"), (300, 513, 77, "bf16"),
                                                 (33, 2000, 61, "f32"), (60, 5000, 30, "f32")])
def test_xent_grad_rows_off_every_boundary(n, vocab, width, dtype):
    """dw rows that start in the middle of a word, into a caller's matrix with gaps that stay as they are; products
    split many ways along the vocabulary."""
    x, w, t = make(n, vocab, width, dtype, seed=n)
    loss, state = snack.xent(x, w, t)
    scale = 1.0 / float(((t >= 0) & (t < vocab)).sum())
    r = reference(x, w, t, np.full(n, scale))
    check_grads(*snack.xent_grad(x, w, t, state), r, dtype)
    for gap, lead in ((0, 1), (3, 0), (1, 2)):
        buf = torch.full((vocab * (width + gap) + lead,), 7.0, device="cuda", dtype=DTYPES[dtype])
        dw = buf[lead:].view(vocab, width + gap)[:, :width]
        ws = torch.empty(snack.snack_xent_workspace_size(x, w, True), dtype=torch.uint8, device="cuda")
        snack.snack_xent_bwd(x, w, t, 2, state, None, None, dw, ws)
        check_grads(None, dw, r, dtype)
        if gap:
            assert torch.all(buf[lead:].view(vocab, width + gap)[:, width:] == 7.0)
        assert torch.all(buf[:lead] == 7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
@pytest.mark.parametrize("n", [1, 16, 17, 32, 33])
def test_xent_totals_of_a_few_rows(n, reduction, dtype):
    x, w, t = make(n, 900, 72, dtype, seed=100 + n, ignored=0.4)
    loss, state = snack.xent(x, w, t, reduction)
    r = reference(x, w, t, np.ones(n))
    count = max(1, int(r["inside"].sum()))
    over = count if reduction == "mean" else 1
    # the rows' bounds, and the total's rounding to fp32 (it is added in 64 bits)
    bound = (2 * A * r["T"] + 2.0 ** -16 + 2.0 ** -22 * np.abs(r["lse"]))[r["inside"]].sum() / over
    want = r["loss"].sum() / over
    assert abs(float(loss) - want) <= bound + 2.0 ** -23 * abs(want)
    assert float(state[n]) == (float(np.float32(1) / np.float32(count)) if reduction == "mean" else 1.0)


def test_linear_cross_entropy_refuses_a_second_derivative():
    x, w, t = make(4, 9, 8, "f32", seed=15)
    x = x.contiguous().requires_grad_()
    (g,) = torch.autograd.grad(snack.linear_cross_entropy(x, w.contiguous(), t), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("n,vocab,width,gap,lead", [
    (5, 1, 1, 0, 0), (6, 300, 31, 0, 0), (7, 257, 4101, 0, 0), (8, 4500, 64, 4, 4), (12, 255, 33, 0, 3), (13, 2049, 2052, 0, 0),
    (24, 513, 961, 0, 0), (31, 40000, 36, 0, 0), (33, 129, 449, 0, 1), (48, 3000, 100, 4, 0), (64, 1000, 1300, 0, 0),
    (64, 200, 2049, 0, 0), (65, 300, 64, 0, 0),
])
def test_xent_some_fp32_tokens(n, vocab, width, gap, lead):
    x, w, t = make(n, vocab, width, "f32", seed=n + vocab, gap=gap, lead=lead, ignored=0.2)
    up = torch.from_numpy(np.random.default_rng(n).normal(size=n).astype(np.float32)).cuda()
    r = reference(x, w, t, up.cpu().numpy().astype(np.float64))
    loss, state = snack.xent(x, w, t, reduction="none")
    check_loss(loss, r)
    assert torch.equal(loss, snack.xent(x, w, t, reduction="none")[0])
    check_grads(*snack.xent_grad(x, w, t, state, up, reduction="none"), r, "f32")


@pytest.mark.parametrize("n", [8, 30, 50, 70])
def test_xent_fp32_not_finite_rows_stay_apart(n):
    x, w, t = make(n, 700, 96, "f32", seed=n, ignored=0.0)
    clean, _ = snack.xent(x, w, t, reduction="none")
    bad = x.clone()
    bad[1, 3] = float("nan")
    bad[n - 2, 0] = float("inf")
    loss, _ = snack.xent(bad, w, t, reduction="none")
    assert torch.isnan(loss[1]) and not torch.isfinite(loss[n - 2])
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[1] = keep[n - 2] = False
    assert torch.equal(loss[keep], clean[keep])
    t[1] = t[n - 2] = -100
    loss, state = snack.xent(bad, w, t, reduction="none")
    assert float(loss[1]) == 0.0 and float(loss[n - 2]) == 0.0
    ones = torch.ones(n, device="cuda")
    dx, dw = snack.xent_grad(bad, w, t, state, ones, reduction="none")
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all()) and not dx[1].any() and not dx[n - 2].any()
    # a weight that is no number spoils every row's loss, and is not lost on the way
    w[5, 7] = float("nan")
    assert bool(torch.isnan(snack.xent(x, w, t, reduction="none")[0][t >= 0]).all())


@pytest.mark.parametrize("n", [4, 8, 16, 32, 64, 100])
def test_xent_fp32_losses_are_fp32(n):
    # the tensor core rounds sums towards zero: 750 instructions in a row (2000 of K, six part products) would lose
    # 750 / 2 * 1.4e-8 = 5e-6 of a logit, 1.6e-4 of a loss near 32.  Held to half of that: 2^-20 of lse and what
    # fp32 sums of this many terms round (2^-18 of a thirtieth of the magnitudes' sum, near the sum's own size)
    x, w, t = make(n, 2000, 2000, "f32", seed=n, ignored=0.0, spread=8.0)
    r = reference(x, w, t, np.ones(n))
    loss, _ = snack.xent(x, w, t, reduction="none")
    assert np.all(np.abs(f64(loss) - r["loss"]) <= 2.0 ** -18 * r["T"] / 30 + 2.0 ** -20 * np.abs(r["lse"]))


@pytest.mark.parametrize("n", [1, 3, 4])
@pytest.mark.parametrize("vocab", [1, 17, 19455, 19456, 19700])
def test_xent_a_few_fp32_tokens_of_any_vocabulary(n, vocab):
    x, w, t = make(n, vocab, 45, "f32", seed=n + vocab, ignored=0.0)
    r = reference(x, w, t, np.full(n, 0.5))
    loss, state = snack.xent(x, w, t, reduction="none")
    check_loss(loss, r)
    check_grads(*snack.xent_grad(x, w, t, state, torch.full((n,), 0.5, device="cuda"), reduction="none"), r, "f32")


def test_xent_first_calls_of_a_process():
    """Kernels whose shared memory lies near the limit that a launch may use without asking for more."""
    code = """
import torch
from spmm_row_sorted_gb300 import snack
for n, vocab, width in ((32, 257, 64), (30, 500, 250), (16, 300, 400), (8, 300, 900), (64, 100, 100), (2, 20000, 2900)):
    x, w = torch.randn(n, width, device="cuda"), torch.randn(vocab, width, device="cuda") / width
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, state = snack.xent(x, w, t)
    want = torch.nn.functional.cross_entropy(x.double() @ w.double().t(), t)
    assert abs(float(loss) - float(want)) < 1e-4
    snack.xent_grad(x, w, t, state)
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def confident(n, width, dtype, seed):
    """Rows of x along their own target's row of w, all operands positive: logits of 40 for the target and near 30 for the
    63 others, so 1 - p is some 1e-3."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.rand(64, width, device="cuda", generator=g).to(DTYPES[dtype])
    t = torch.arange(n, device="cuda") % 64
    x = (w[t].float() * (120.0 / width) * (1.0 + torch.rand(n, 1, device="cuda", generator=g) / 16)).to(DTYPES[dtype])
    return x, w, t


@pytest.mark.parametrize("n,width,dtype", [
    (64, 4096, "bf16"), (40, 2500, "bf16"), (150, 4160, "bf16"), (300, 1000, "bf16"),
    (4, 4096, "f32"), (16, 4096, "f32"), (64, 4096, "f32"), (100, 4096, "f32"),
    (17, 4096, "f32"), (32, 4096, "f32"), (64, 512, "f32"),
])
def test_xent_grad_of_confident_tokens(n, width, dtype):
    # At the target dz = p - 1 cancels to 1e-3, so the gradient's logits have to agree with the loss's far better than
    # each agrees with 64 bits.  Allowed of dz there: the rounding of lse (2^-19 below 64), of its logarithm, of the sum and of
    # the exponential (2^-21 each): 2^-18.
    # Elsewhere p moves by the differences of logits, 2^-14 relative; dz is rounded to bf16 (2^-9) or to fp32 parts;
    # products lose up to 2^-16 of their magnitudes on the way (2^-20 for fp32).
    x, w, t = confident(n, width, dtype, seed=n + width)
    up = torch.full((n,), 1.0, device="cuda")
    r = reference(x, w, t, np.ones(n))
    loss, state = snack.xent(x, w, t, reduction="none")
    dx, dw = snack.xent_grad(x, w, t, state, up, reduction="none")
    X, W, T = f64(x), f64(w), t.cpu().numpy()
    z = X @ W.T
    z -= z.max(1, keepdims=True)
    p = np.exp(z)
    p /= p.sum(1, keepdims=True)
    hot = np.zeros_like(p)
    hot[np.arange(n), T] = 1.0
    dz = p - hot
    dz[np.arange(n), T] = -(p * (1 - hot)).sum(1)  # 1 - p without cancellation
    assert 1e-4 < -dz[np.arange(n), T].max() and -dz[np.arange(n), T].min() < 5e-2
    err = (2.0 ** -14 + (2.0 ** -9 if dtype == "bf16" else 2.0 ** -22)) * np.abs(dz) + 2.0 ** -18 * hot
    product = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -20
    for got, ref, bound in ((dx, dz @ W, err @ np.abs(W) + product * (np.abs(dz) @ np.abs(W))),
                            (dw, dz.T @ X, err.T @ np.abs(X) + product * (np.abs(dz).T @ np.abs(X)))):
        if dtype == "bf16":
            bound = bound + bf16_half_ulp(np.abs(ref) + bound)
        off = np.abs(f64(got) - ref) / bound
        assert off.max() <= 1.0, off.max()
    assert np.all(np.abs(f64(loss) - r["loss"]) <= 2 * A * r["T"])


def operands_of_a_kind(kind, n, width, dtype):
    """Logits of about 40 for one of 63 rows of w, row 0 of which is zero: the loss of target 0 is lse."""
    g = torch.Generator(device="cuda").manual_seed(7)

    def some(rows):
        a = torch.randn(rows, width, device="cuda", generator=g)
        if kind == "positive":
            return a.abs()
        return a * (torch.rand(rows, width, device="cuda", generator=g) < 0.1) if kind == "nine of ten zero" else a

    w = some(64)
    w[0] = 0.0
    w = (w * (40.0 / width * (10.0 ** 0.5 if kind == "nine of ten zero" else 1.0))).to(DTYPES[dtype])
    owner = torch.arange(n, device="cuda") % 63 + 1
    x = (w[owner].float() * (width / 40.0) + some(n)).to(DTYPES[dtype])
    return x, w, torch.zeros(n, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("kind", ["random", "positive", "nine of ten zero"])
@pytest.mark.parametrize("n,dtype", [(256, "bf16"), (16, "f32"), (64, "f32"), (256, "f32")])
def test_xent_mean_error_of_the_logits(n, dtype, kind):
    # The accumulator rounds towards zero: an instruction (16 of K) costs a sum of positive products 3.6e-8 of itself at
    # most, and 32 of them run in a row (16 of fp32 operands), so a logit is up to 1.15e-6 (5.8e-7) too small; rounding
    # to nearest, elsewhere, leaves less than 1e-7 on average.  Never too large: nothing is put back by guess.
    x, w, t = operands_of_a_kind(kind, n, 4096, dtype)
    loss, _ = snack.xent(x, w, t, reduction="none")
    z = x.double() @ w.double().T
    mean = float(((loss.double() - torch.logsumexp(z, 1)) / z.amax(1)).mean())
    assert -(1.15e-6 if dtype == "bf16" else 5.8e-7) <= mean <= 1e-7, mean


@pytest.mark.parametrize("n,dtype", [(1, "bf16"), (200, "bf16"), (4, "f32"), (16, "f32"), (64, "f32"), (200, "f32")])
def test_xent_logits_of_few_bits_are_exact(n, dtype):
    # whole numbers below 2^9 as logits, and all their partial sums: only lse, its logarithm and the sum of
    # exponentials round, 2^-24 of lse each at most, and 2^-20 of the loss's other terms
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randint(-2, 3, (300, 2048), device="cuda", generator=g) * (torch.rand(300, 2048, device="cuda", generator=g) < 0.1)
    w[0] = 0
    owner = torch.arange(n, device="cuda") % 299 + 1
    x = w[owner]
    z = x.double() @ w.double().T
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, state = snack.xent(x.to(DTYPES[dtype]), w.to(DTYPES[dtype]), t, reduction="none")
    lse = torch.logsumexp(z, 1)
    assert 200.0 < float(lse.amin()) and float(lse.amax()) < 512.0
    assert bool(((loss.double() - lse).abs() <= 2.0 ** -23 * lse + 2.0 ** -20).all())


@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("n,vocab,dtype", [(1, 64, "bf16"), (20, 64, "bf16"), (64, 300, "bf16"), (200, 1000, "bf16"), (3, 64, "f32"),
                                           (4, 20000, "f32"), (16, 64, "f32"), (64, 64, "f32"), (100, 300, "f32")])
def test_xent_loss_of_confident_tokens(n, vocab, dtype, reduction):
    """A loss far below the logits it is the difference of: not rounded to the spacing of lse."""
    # Operands of few bits, so that every product and sum is exact: logits of 384 + d for the target and 384 and less for
    # the others.  What is left: differences of logits, each within two fp32 spacings at 384 (2^-14) relative of a
    # loss; 2^-20 for the exponentials, the sum near 1 and its logarithm.  lse alone has spacing 2^-15.
    rng = np.random.default_rng(n + vocab)
    d = rng.integers(14, 26, n) / 2.0
    x, w = np.zeros((n, 16)), np.zeros((vocab, 16))
    x[:, 0], w[:, 0] = 24.0, 16.0
    x[:, 1] = 1.0
    w[1:, 1] = -rng.integers(0, 9, vocab - 1) / 2.0
    x[:, 2], w[0, 2] = d, 1.0
    x, w = (torch.from_numpy(a).to(DTYPES[dtype]).cuda() for a in (x, w))
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    X, W = f64(x), f64(w)
    z = X @ W.T
    rest = np.exp(z[:, 1:] - z[:, :1]).sum(1)
    want = np.log1p(rest)
    bound = 2.0 ** -14 * want + 2.0 ** -20
    loss, state = snack.xent(x, w, t, reduction=reduction)
    if reduction == "mean":
        assert abs(float(loss) - want.mean()) <= bound.mean()
    else:
        assert np.all(np.abs(f64(loss) - want) <= bound)
    assert np.all(np.abs(f64(state)[:n] - (z[:, 0] + want)) <= 2.0 ** -20 * z[:, 0])


def test_calls_on_the_default_stream_by_its_handle():
    """The default stream's handle is 0: the call runs there, not on a stream of its own."""
    x, w, t = make(40, 300, 64, "bf16", seed=3)
    for handle in (0, torch.cuda.default_stream().cuda_stream, torch.cuda.default_stream()):
        with snack._On(x.device, handle):
            assert torch.cuda.current_stream().cuda_stream == 0
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        with snack._On(x.device, handle):
            assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
    loss, _ = snack.xent(x, w, t)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # from another stream
        assert torch.equal(snack.xent(x, w, t, stream=0)[0].cpu(), loss.cpu())
    torch.cuda.synchronize()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
@pytest.mark.parametrize("n,dtype", [(3, "f32"), (12, "f32"), (40, "f32"), (90, "f32"), (5, "bf16"), (140, "bf16")])
def test_xent_rows_not_trained_on_stay_out_whatever_the_upstream_gradient(n, dtype, reduction, value):
    x, w, t = make(n, 300, 72, dtype, seed=n, ignored=0.0)
    t[n // 2] = -100
    up = torch.tensor(value, device="cuda")
    loss, state = snack.xent(x, w, t, reduction=reduction)
    dx, dw = snack.xent_grad(x, w, t, state, up, reduction=reduction)
    keep = (t >= 0) & (t < 300)
    assert not torch.isfinite(dx[keep]).any()
    assert not dx[~keep].any()  # a NaN counts as not zero
    assert not torch.isfinite(dw).all()
    t[:] = -100  # nothing to train on
    loss, state = snack.xent(x, w, t, reduction=reduction)
    dx, dw = snack.xent_grad(x, w, t, state, up, reduction=reduction)
    assert float(loss) == 0.0 and not dx.any() and not dw.any()


def piece_targets(n, vocab, seed):
    """Targets over the whole vocabulary, many of them on either side of multiples of 256: where pieces of it may end."""
    rng = np.random.default_rng(seed)
    t = rng.integers(0, vocab, n)
    edges = np.arange(1, (vocab + 255) // 256) * 256
    near = rng.choice(edges, n // 2) - rng.integers(0, 2, n // 2)
    t[:n // 2] = near
    for pair in (19456, 77824):  # whole waves of tiles of a GPU of 152 multiprocessors
        e = np.arange(pair, vocab, pair)
        k = min(len(e), n // 8)
        t[n // 2:n // 2 + k], t[n // 2 + k:n // 2 + 2 * k] = e[:k], e[:k] - 1
    t[-1], t[-2], t[-3] = vocab - 1, 0, -100
    return torch.from_numpy(t).cuda()


@pytest.mark.parametrize("n,vocab,width,dtype,spread", [
    (70, 120000, 512, "f32", 3.0),     # w's three parts, 369 MB: two pieces of the loss and of the gradient
    (70, 120000, 512, "f32", 0.03),    # nearly equal logits: what the products round shows
    (60, 120000, 512, "f32", 3.0),     # the same with w cut as it is read
    (3000, 40000, 64, "f32", 3.0),     # dz's three parts, 720 MB: several pieces of the gradient alone
    (80, 300001, 513, "bf16", 3.0),    # rows that are laid out again, 346 MB: several pieces of both
    (4200, 70000, 136, "bf16", 3.0),   # dz of 588 MB; rows off 128-byte lines
])
def test_xent_in_several_pieces_of_every_kind(n, vocab, width, dtype, spread):
    x, w, _ = make(n, vocab, width, dtype, seed=n + width, spread=spread)
    t = piece_targets(n, vocab, n)
    inside = (t >= 0) & (t < vocab)
    count = int(inside.sum())
    X, W = x.double(), w.double()
    at = torch.where(inside, t, 0)[:, None]
    loss, state = snack.xent(x, w, t, reduction="none")
    mean, kept = snack.xent(x, w, t)
    dx, dw = snack.xent_grad(x, w, t, kept)
    T = float(w.abs().double().sum(1).max()) * float(x.abs().max())  # above every row's sum of magnitudes
    T = min(T, float((X[:64].abs() @ W.abs().T).max()) * 1.5)
    want, lse = torch.empty(n, device="cuda", dtype=torch.float64), torch.empty(n, device="cuda", dtype=torch.float64)
    ref_x, mag_x = torch.zeros_like(X), torch.zeros_like(X)
    ref_w, mag_w = torch.zeros_like(W), torch.zeros_like(W)
    for a in range(0, n, 512):  # rows at a time: the logits in 64 bits are large
        s = slice(a, min(n, a + 512))
        z = X[s] @ W.T
        lse[s] = torch.logsumexp(z, 1)
        want[s] = torch.where(inside[s], lse[s] - z.gather(1, at[s])[:, 0], 0.0)
        p = torch.exp(z - lse[s][:, None])
        del z
        weight = (inside[s].double() / count)[:, None]
        p *= weight
        mag = p.clone().scatter_add_(1, at[s], weight)
        p.scatter_add_(1, at[s], -weight)
        ref_x[s], mag_x[s] = p @ W, mag @ W.abs()
        ref_w += p.T @ X[s]
        mag_w += mag.T @ X[s].abs()
        del p, mag
    bound = 2 * A * T + 2.0 ** -16 + 2.0 ** -22 * lse.abs()
    assert bool(((loss.double() - want).abs() <= bound).all())
    assert abs(float(mean) - float(want.sum()) / count) <= float(bound.max()) + 2.0 ** -23 * abs(float(mean))
    e = 2 * A * T + 2.0 ** -16 + A + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22)
    for got, ref, mag in ((dx, ref_x, mag_x), (dw, ref_w, mag_w)):
        tol = e * mag
        if dtype == "bf16":
            tol = tol + torch.from_numpy(bf16_half_ulp((ref.abs() + tol).cpu().numpy())).cuda()
        assert bool(((got.double() - ref).abs() <= tol + 1e-300).all())
    assert not dx[~inside].any()


@pytest.mark.parametrize("n,vocab,width", [(64, 300, 513), (64, 300, 1000), (130, 700, 4160), (20, 1000, 2048), (260, 513, 1100)])
def test_xent_bf16_widths_of_several_units(n, vocab, width):
    """More of K than the tensor core sums at a time."""
    x, w, t = make(n, vocab, width, "bf16", seed=n + width)
    up = torch.from_numpy(np.random.default_rng(n).normal(size=n).astype(np.float32)).cuda()
    r = reference(x, w, t, up.cpu().numpy().astype(np.float64))
    loss, state = snack.xent(x, w, t, reduction="none")
    check_loss(loss, r)
    check_grads(*snack.xent_grad(x, w, t, state, up, reduction="none"), r, "bf16")


def few_terms(n, vocab, width, seed):
    """Nearly equal logits (sums of tiny values), so that dz is known to fp32 and a gradient shows what its products round:
    two rows that are trained on (dw's sums have two terms), and a vocabulary of `vocab` (dx's)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, width, device="cuda", generator=g)
    w = torch.randn(vocab, width, device="cuda", generator=g) * 2.0 ** -10
    t = torch.full((n,), -100, dtype=torch.int64, device="cuda")
    t[1], t[n - 1] = 0, vocab - 1
    return x, w, t


def parts_of(a, parts):
    """a as a sum of `parts` bf16 values, each the rounding of what the ones before leave over."""
    out = np.zeros_like(a)
    for _ in range(parts):
        out += torch.from_numpy((a - out).astype(np.float32)).to(torch.bfloat16).double().numpy()
    return out


@pytest.mark.parametrize("n,vocab,width", [
    (2, 3, 64), (4, 20000, 40), (4, 3, 300), (8, 2, 64), (16, 3, 129),   # the CUDA cores
    (17, 3, 64), (33, 2, 100), (64, 3, 520), (65, 3, 64), (100, 2, 777), (300, 3, 256), (100, 200, 64),  # the tensor cores
])
def test_xent_fp32_gradients_are_fp32(n, vocab, width):
    # p = exp(z - lse): lse and its logarithm round to 2^-24 of lse < 16 each, the exponent's argument to as much, 2^x to 2^-22:
    # 2^-19.5 of p at lse = 10, 2^-21 near log 3.  At the target the difference rounds once more, 2^-24.
    # A product of parts leaves out 2^-23 of itself, its sum of a few terms rounds to 2^-22 of the magnitudes, the
    # factor and the output to 2^-23.
    x, w, t = few_terms(n, vocab, width, seed=n + vocab)
    X, W, T = f64(x), f64(w), t.cpu().numpy()
    inside = T >= 0
    z = X @ W.T
    lse = np.log(np.exp(z).sum(1))
    p = np.where(inside[:, None], np.exp(z - lse[:, None]), 0.0)
    hot = np.zeros_like(p)
    hot[np.arange(n)[inside], T[inside]] = 1.0
    dz = (p - hot) / inside.sum()
    err = (2.0 ** -23 * (4 + 1.5 * np.abs(lse))[:, None] * p + 2.0 ** -24 * hot) / inside.sum()
    product = 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -23
    loss, state = snack.xent(x, w, t)
    dx, dw = snack.xent_grad(x, w, t, state)
    for got, a, b, e in ((dx, dz, W, err), (dw, dz.T, X, err.T)):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        bound = e @ np.abs(b) + product * mag + 2.0 ** -149
        off = np.abs(f64(got) - ref) / bound
        assert off.max() <= 1.0, off.max()
        # the same with two parts of either operand would be outside: of dz where its terms are few and its values several
        assert (np.abs(a @ parts_of(b, 2) - ref) > bound).any()
        assert n < 8 or (np.abs(parts_of(a, 2) @ b - ref) > bound).any()


@pytest.mark.parametrize("n,width,dtype", [(100, 4096, "bf16"), (100, 4096, "f32"), (40, 2048, "bf16"), (300, 1001, "f32")])
def test_xent_loss_does_not_take_the_accumulators_bias_of_the_target(n, width, dtype):
    # a target's logit near 8 above others of about 1: on the tensor core it would come out 6e-7 of itself too small, 5e-6
    # of the loss.  In fp32 it rounds to either side; what remains is the others' bias, at most 1.15e-6 of their average in
    # lse, which is below 1.5
    g = torch.Generator(device="cuda").manual_seed(width)
    w = (torch.randn(20000, width, device="cuda", generator=g) / width ** 0.5).to(DTYPES[dtype])
    t = torch.randint(0, 20000, (n,), device="cuda", generator=g)
    x = (torch.randn(n, width, device="cuda", generator=g) + 8.0 * w[t].float()).to(DTYPES[dtype])
    z = x.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    rest = torch.exp(z - lse[:, None])
    assert float((rest * z).sum(1).sub((rest * z).gather(1, t[:, None])[:, 0]).mean()) < 1.5
    want = lse - z.gather(1, t[:, None])[:, 0]
    loss, _ = snack.xent(x, w, t, reduction="none")
    assert abs(float((loss.double() - want).mean())) <= 1.15e-6 * 1.5


@pytest.mark.parametrize("n,vocab,dtype", [(3, 20000, "f32"), (3, 500, "bf16"), (70, 500, "bf16"), (300, 700, "bf16")])
def test_xent_logits_of_minus_infinity(n, vocab, dtype):
    """Vocabulary rows that an infinite weight takes out: as fp32 arithmetic has it, where the products are not over parts.
    (The smallest vocabulary of the fp32 case's kernel is 128 rows for each of a GPU's multiprocessors.)"""
    x, w, t = make(n, vocab, 64, dtype, seed=n + vocab, ignored=0.0)
    x, w = x.abs().contiguous(), w.clone()
    gone = torch.arange(vocab, device="cuda") % 3 == 1
    w[gone, 5] = -float("inf")
    t[t % 3 == 1] = 2
    r = reference(x, w[~gone].contiguous(), t - (t + 1) // 3, np.ones(n))
    loss, state = snack.xent(x, w, t, reduction="none")
    check_loss(loss, r)
    t[0] = 1  # a target that is out
    loss, state = snack.xent(x, w, t, reduction="none")
    assert float(loss[0]) == float("inf") and torch.isfinite(loss[1:]).all() and torch.isfinite(state).all()


@pytest.mark.parametrize("n,vocab,width,gap,lead", [(100, 300, 128, 0, 0), (5, 64, 1000, 0, 0), (70, 500, 77, 0, 0), (300, 1500, 96, 4, 4),
                                                    (64, 200, 100, 3, 1)])
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_xent_dx_of_bf16_has_the_targets_entry_unrounded(n, vocab, width, gap, lead, reduction):
    # logits with probabilities near a half at the target, whose dz is most of the row's: its rounding to bf16 would be
    # up to 2^-9 of dx.  Left: every other entry's (2^-9 p), fp32 sums (2^-20 of T for a logit, 2^-16 of a product's
    # magnitudes) and dx's own rounding
    x, w, t = make(n, vocab, width, "bf16", seed=n + vocab, gap=gap, lead=lead, ignored=0.1, spread=1.0)
    inside = (t >= 0) & (t < vocab)
    at = torch.where(inside, t, 0)
    aim = w.float()[at]
    x.copy_((x.float() * 0.1 + aim * (float(np.log(vocab)) / aim.square().sum(1, keepdim=True))))
    up = torch.rand(n, device="cuda") + 0.5
    weight = f64(up) if reduction == "none" else np.full(n, 1.0 / max(1, int(inside.sum())))
    r = reference(x, w, t, weight)
    loss, state = snack.xent(x, w, t, reduction=reduction)
    dx, dw = snack.xent_grad(x, w, t, state, up if reduction == "none" else None, reduction=reduction)
    X, W, T = f64(x), f64(w), at.cpu().numpy()
    z = X @ W.T
    p = np.exp(z - r["lse"][:, None])
    hot = np.zeros_like(p)
    hot[np.arange(n), T] = r["inside"]
    assert 0.2 < np.median(p[hot > 0]) < 0.8
    g = np.where(r["inside"], weight, 0.0)[:, None]
    noise = (2.0 ** -20 * r["T"] + 2.0 ** -16)[:, None]
    bound = (g * (p * (noise + 2.0 ** -9 * (1 - hot)) + 2.0 ** -16 * (p + hot))) @ np.abs(W)
    bound = bound + bf16_half_ulp(np.abs(r["dx"]) + bound)
    off = np.abs(f64(dx) - r["dx"]) / (bound + 1e-300)
    assert off.max() <= 1.0, off.max()
    check_grads(None, dw, r, "bf16")
