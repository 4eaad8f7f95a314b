"""Log probabilities of tokens, entropies and likeliest tokens of a vocabulary projection, and the gradients, against the
definitions in 64 bits.

Tolerances.  A logit is within A T of its value, A = 1e-5 (the bound of every fp32 sum of this library) and T the largest sum
of magnitudes of the row.  The log of the sum moves by at most the largest of these, plus the errors of 2^x (2^-21) and of
the sums (2^-17 over thousands of terms): |err logp| <= 2 A T + 2^-16 + 2^-22 |lse|; with e = 2 A T + 2^-16 a probability is
within e of itself.  H = log S - sum e^(z - M) (z - M) / S: the second part is at most H and a sum of terms of one sign, each
within e of itself; dH/dz_v = -p (log p + H), the sum of which over v is at most 2 H: |err H| <= e (1 + 4 H).
dz = g [v = t] - p (g + h (log p + H)) is within e of the magnitude of each part, p |h| (err logp + err H) and its rounding,
2^-8 of it (bf16; not of the target's entry where g is not 0, which goes unrounded into both products: with g = 0 it is
an entry like the others, -p h (log p + H) rounded to bf16, by half an ulp and so up to 2^-8 of it) or 2^-22 (fp32 parts).  A product's sum adds A of its magnitudes, a bf16 output half an ulp.
Ids: where the logits' order is not clear in fp32 the products are summed in twice its precision, so ids are equal to the
order of the 64-bit logits, whose differences are far above 2^-45 of them here.
"""

import pytest
import torch

from spmm_row_sorted_gb300 import snack

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
A = 1e-5


def make(n, vocab, width, dtype, seed, gap=0, lead=0, ignored=0.1, itype=torch.int64, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def matrix(rows, std):
        buf = torch.full((rows * (width + gap) + lead,), float("nan"), device="cuda", dtype=DTYPES[dtype])
        m = buf[lead:].view(rows, width + gap)[:, :width]
        m.copy_(torch.empty(rows, width, device="cuda").normal_(0, std, generator=g))
        return m

    x, w = matrix(n, 1.0), matrix(vocab, spread / width ** 0.5)
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    t[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    t[torch.rand(n, generator=g, device="cuda") < ignored / 4] = vocab
    if n > 1:
        t[0], t[-1] = 0, vocab - 1
    return x, w, t.to(itype)


class Want:
    def __init__(self, x, w, t, top=0):
        x, w = x.double(), w.double()
        n, vocab = len(x), len(w)
        self.x, self.w = x, w
        self.scored = torch.ones(n, dtype=torch.bool, device="cuda") if t is None else (t >= 0) & (t < vocab)
        z = x @ w.T
        self.T = (x.abs() @ w.abs().T).amax(1)
        self.lse = torch.logsumexp(z, 1)
        self.log_p = z - self.lse[:, None]
        self.p = self.log_p.exp()
        self.H = -(self.p * self.log_p).sum(1)
        self.e = 2 * A * self.T + 2.0 ** -16
        self.logp_tol = self.e + 2.0 ** -22 * self.lse.abs()
        self.H_tol = self.e * (1 + 4 * self.H)
        if t is not None:
            self.at = torch.where(self.scored, t.long(), 0)
            self.logp = self.log_p.gather(1, self.at[:, None])[:, 0]
        if top:
            self.ids = z.sort(dim=1, descending=True, stable=True).indices[:, :top]
            self.top_logp = self.log_p.gather(1, self.ids)

    def check(self, got):
        logp, entropy, ids, top_logp, state = got
        s = self.scored
        if logp is not None:
            assert bool(((logp - self.logp).abs() <= self.logp_tol)[s].all()) and bool((logp[~s] == 0).all())
        assert bool(((entropy - self.H).abs() <= self.H_tol)[s].all()) and bool((entropy[~s] == 0).all())
        if ids is not None:
            assert torch.equal(ids[s], self.ids[s]) and bool((ids[~s] == -1).all())
            assert bool(((top_logp - self.top_logp).abs() <= self.logp_tol[:, None])[s].all()) and bool((top_logp[~s] == 0).all())
            assert bool((top_logp[:, 1:] <= top_logp[:, :-1]).all())
        assert bool(((state[0] - self.lse).abs() <= self.logp_tol)[s].all()) and torch.equal(state[1], entropy)

    def check_grads(self, dx, dw, g, h):
        bf = dx.dtype == torch.bfloat16
        zero = torch.zeros(len(self.x), device="cuda", dtype=torch.float64)
        g, h = (torch.where(self.scored, zero if d is None else d.double(), 0.0)[:, None] for d in (g, h))
        dz, H = -self.p * (g + h * (self.log_p + self.H[:, None])), self.H[:, None]
        mag = self.p * (g.abs() + h.abs() * ((self.log_p + H).abs() + 2 + 8 * H))
        rel = self.e[:, None] + A
        mag = mag * (rel + (2.0 ** -8 if bf else 2.0 ** -22))
        if hasattr(self, "at"):
            dz.scatter_add_(1, self.at[:, None], g)
            if bf:  # its own part of p, too
                own = mag.gather(1, self.at[:, None])
                mag.scatter_(1, self.at[:, None], torch.where(g != 0, own * (rel + 2.0 ** -22) / (rel + 2.0 ** -8), own))
            mag.scatter_add_(1, self.at[:, None], g.abs() * (rel + 2.0 ** -22))
        for got, want, tol in ((dx, dz @ self.w, mag @ self.w.abs()), (dw, dz.T @ self.x, mag.T @ self.x.abs())):
            tol = tol + HALF_ULP[got.dtype] * (want.abs() + tol) + 2.0 ** -133
            assert bool(((got - want).abs() <= tol).all())


SHAPES = [
    # n, vocab, width, gap, lead, top
    (1, 1, 1, 0, 0, 1),
    (1, 2, 8, 0, 0, 2),
    (2, 31, 8, 0, 0, 5),
    (1, 5000, 64, 0, 0, 24),
    (3, 257, 16, 0, 0, 1),
    (4, 30000, 40, 0, 0, 8),   # few fp32 tokens on the CUDA cores
    (7, 1003, 33, 3, 1, 24),
    (16, 1000, 128, 0, 0, 20),
    (31, 129, 72, 0, 0, 3),
    (64, 700, 264, 0, 0, 5),   # fp32 logits by warps that share rows
    (65, 300, 264, 0, 0, 5),
    (127, 513, 65, 0, 0, 8),   # rows that are laid out again
    (128, 512, 64, 0, 0, 0),
    (129, 511, 192, 0, 0, 24),
    (200, 700, 100, 4, 0, 7),
    (200, 700, 96, 0, 1, 2),
    (300, 4000, 320, 0, 0, 16),
    (64, 40000, 40, 0, 0, 10),
    (1030, 3001, 259, 0, 0, 4),
    (257, 33, 600, 0, 0, 24),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,width,gap,lead,top", SHAPES)
def test_score_matches_definition(n, vocab, width, gap, lead, top, dtype):
    x, w, t = make(n, vocab, width, dtype, seed=n + vocab, gap=gap, lead=lead, itype=torch.int32 if n % 2 else torch.int64)
    want = Want(x, w, t, top)
    got = snack.score(x, w, t, top)
    want.check(got)
    for a, b in zip(got, snack.score(x, w, t, top)):  # repeats bit for bit
        assert a is b is None or torch.equal(a, b)
    # without tokens every row is scored; results do not depend on what else is asked for
    free = snack.score(x, w, top=top)
    Want(x, w, None, top).check(free)
    assert free[0] is None
    alone = snack.score(x, w, t)
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1]) and alone[2] is None and alone[3] is None
    gen = torch.Generator(device="cuda").manual_seed(n)
    g, h = (torch.randn(n, device="cuda", generator=gen) for _ in range(2))
    h[::3] = 0
    g[::5] = 0
    dx, dw = snack.score_grad(x, w, t, got[4], g, h)
    want.check_grads(dx, dw, g, h)
    assert bool((dx[~want.scored] == 0).all()) and bool((dx[(g == 0) & (h == 0)] == 0).all())
    again = snack.score_grad(x, w, t, got[4], g, h)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    only_x, no_w = snack.score_grad(x, w, t, got[4], g, h, want_dw=False)
    no_x, only_w = snack.score_grad(x, w, t, got[4], g, h, want_dx=False)
    assert no_w is None and no_x is None and torch.equal(only_x, dx) and torch.equal(only_w, dw)
    want.check_grads(*snack.score_grad(x, w, t, got[4], g), g, None)
    want.check_grads(*snack.score_grad(x, w, t, got[4], dentropy=h), None, h)
    Want(x, w, None).check_grads(*snack.score_grad(x, w, None, free[4], dentropy=h), None, h)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_log_probability_s_gradient_is_the_loss_s_negative(dtype):
    """Bit for bit, but for the rows of dw that are targets of bf16 operands: those take the target's entry of dz, g (1 - p),
    unrounded.  The loss's are off by its rounding (2^-8 |g| of a row of x each), and both by their own (half an ulp)."""
    x, w, t = make(90, 900, 128, dtype, seed=5)
    g = torch.randn(90, device="cuda")
    state = snack.score(x, w, t)[4]
    kept = snack.xent(x, w, t, reduction="none")[1]
    kept[:90] = state[0]
    (dx, dw), (lx, lw) = snack.score_grad(x, w, t, state, g), snack.xent_grad(x, w, t, kept, -g, reduction="none")
    assert torch.equal(dx, lx)
    if dtype == "f32":
        assert torch.equal(dw, lw)
        return
    inside = (t >= 0) & (t < 900)
    tol = torch.zeros(900, 128, device="cuda", dtype=torch.float64)
    tol.index_add_(0, t[inside].long(), 2.0 ** -8 * (g[:, None] * x).double().abs()[inside])
    hit = torch.zeros(900, dtype=torch.bool, device="cuda")
    hit[t[inside].long()] = True
    assert torch.equal(dw[~hit], lw[~hit])
    assert bool(((dw.double() - lw.double()).abs() <= tol + 2.0 ** -8 * (dw.abs() + lw.abs()).double()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 20, 100])
def test_equal_logits_rank_by_id(n, dtype):
    vocab, width = 3000, 64
    x, w, _ = make(n, vocab, width, dtype, seed=1)
    x[0] = 0  # every logit 0
    got = snack.score(x, w, top=24)
    assert torch.equal(got[2][0], torch.arange(24, device="cuda"))
    assert bool(((got[3][0] + torch.log(torch.tensor(float(vocab)))).abs() <= 2.0 ** -16).all())
    w[:] = w[torch.arange(vocab, device="cuda") % 700]  # each row four or five times, far apart
    Want(x, w, None, 13).check(snack.score(x, w, top=13))
    w[:] = w[5]  # all of them
    ids = snack.score(x, w, top=10)[2]
    assert torch.equal(ids, torch.arange(10, device="cuda").expand(n, 10))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 40, 200])
def test_order_where_fp32_cannot_tell(n, dtype):
    """Fourteen logits near 40 that differ by 2^-26: below an fp32 step of them (2^-18), seen in sums of 64 bits.  The
    products are exact and their sums' partial ones need 40 + 26 - ... bits: 64-bit sums hold them all."""
    vocab, width = 5000, 128
    x = torch.zeros(n, width, device="cuda")
    w = torch.zeros(vocab, width, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(n)
    x[:, :100] = torch.randint(1, 9, (n, 100), generator=gen, device="cuda") / 4.0
    x[:, 101] = 2.0 ** -13
    w[:, :100] = torch.randint(-2, 3, (vocab, 100), generator=gen, device="cuda") / 16.0
    near = torch.randperm(vocab, generator=gen, device="cuda")[:14]
    w[near, :100] = 0.25
    w[near, 101] = torch.randperm(14, generator=gen, device="cuda").float() * 2.0 ** -13
    x, w = x.to(DTYPES[dtype]), w.to(DTYPES[dtype])
    want = Want(x, w, None, 6)
    assert torch.equal(snack.score(x, w, top=6)[2], want.ids)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 30, 150])
def test_a_confident_row_keeps_the_digits_of_what_is_below_one(n, dtype):
    """Logits of whole numbers are exact: what is left are the errors of exp and of the sums, relative to 1 - p and H."""
    vocab, width = 2000, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.zeros(n, width, device="cuda", dtype=DTYPES[dtype])
    w = torch.randint(-8, 9, (vocab, width), generator=gen, device="cuda").to(DTYPES[dtype])
    x[:, 0] = 1
    x[:, 1] = 1
    t = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    w[t, 0] = 30 + torch.arange(n, device="cuda").to(DTYPES[dtype]) % 3
    for targets in (t, None):
        want = Want(x, w, targets, 2)
        got = snack.score(x, w, targets, 2)
        want.check(got)
        assert bool(((got[1] - want.H).abs() <= 2.0 ** -16 * want.H).all())
        first = got[0] if targets is not None else got[3][:, 0]
        other = want.logp if targets is not None else want.top_logp[:, 0]
        assert bool(((first - other).abs() <= 2.0 ** -16 * other.abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 30, 150])
def test_rows_that_are_not_scored_stay_out_whatever_they_hold(n, dtype):
    x, w, t = make(n, 600, 64, dtype, seed=3)
    t[1] = -100
    want = snack.score(x, w, t, 4)
    g = torch.randn(n, device="cuda")
    grads = snack.score_grad(x, w, t, want[4], g, g)
    x[1] = float("nan")
    got = snack.score(x, w, t, 4)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    g[1] = float("inf")
    for a, b in zip(snack.score_grad(x, w, t, got[4], g, g), grads):
        assert torch.equal(a, b)
    # a row of its own NaN is NaN, and its ids are of the vocabulary; the others stay
    t[1] = 5
    ids = snack.score(x, w, t, 4)
    assert all(bool(torch.isnan(ids[k][1]).all()) for k in (0, 1, 3)) and bool(((ids[2][1] >= 0) & (ids[2][1] < 600)).all())
    keep = torch.arange(n, device="cuda") != 1
    for k in range(4):
        assert torch.equal(ids[k][keep], want[k][keep])


def test_a_row_with_the_lowest_logits_has_them_last():
    """-inf logits (bf16 operands follow fp32 arithmetic) take no part in sums, entropies and gradients."""
    x, w, t = make(70, 300, 64, "bf16", seed=7, ignored=0)
    x[:, 0], w[:, 0] = 1, 0
    gone = torch.arange(300, device="cuda") % 3 == 0
    w[gone, 0] = float("-inf")
    t = torch.where(t % 3 == 0, (t + 1) % 300, t)
    x0, w0 = x.clone(), w.clone()
    logp, entropy, ids, top_logp, state = snack.score(x, w, t, 24)
    kept = (~gone).nonzero()[:, 0]
    back = torch.full((300,), -1, device="cuda")
    back[kept] = torch.arange(len(kept), device="cuda")
    want = Want(x0, w0[kept].contiguous(), back[t], 24)
    want.check((logp, entropy, back[ids], top_logp, state))


def test_score_in_pieces_of_the_vocabulary():
    x, w, t = make(8200, 50000, 64, "bf16", seed=9)  # 1.6 GB of logits
    got = snack.score(x, w, t, 6)
    for a in range(0, 8200, 1025):
        rows = slice(a, a + 1025)
        Want(x[rows], w, t[rows], 6).check([g[rows] for g in got[:4]] + [got[4][:, rows]])
    x, w, t = make(5000, 30000, 32, "f32", seed=10)
    got = snack.score(x, w, t, 3)
    for a in range(0, 5000, 1000):
        rows = slice(a, a + 1000)
        Want(x[rows], w, t[rows], 3).check([g[rows] for g in got[:4]] + [got[4][:, rows]])


def test_gradients_against_differences():
    """Of L = sum g logp + h H in the direction of a random step of w: a central difference of the 64-bit definition."""
    x, w, t = make(60, 200, 48, "f32", seed=11)
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, h = (torch.randn(60, device="cuda", generator=gen) for _ in range(2))
    state = snack.score(x, w, t)[4]
    dx, dw = snack.score_grad(x, w, t, state, g, h)

    def loss(x, w):
        v = Want(x, w, t)
        return (torch.where(v.scored, g * v.logp + h * v.H, 0.0)).sum()

    for k, grad in ((0, dx), (1, dw)):
        step = torch.randn(grad.shape, device="cuda", generator=gen, dtype=torch.float64)
        eps = 1e-5  # truncation eps^2 and rounding 1e-16 / eps, both 1e-10 of the third derivative and the value
        ends = [loss(*(p.double() + (s * eps * step if i == k else 0) for i, p in enumerate((x, w)))) for s in (1, -1)]
        got, want = float((grad.double() * step).sum()), float((ends[0] - ends[1]) / (2 * eps))
        size = float((grad.double() * step).abs().sum())
        assert abs(got - want) <= 1e-4 * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_gives_autograd_the_gradients(dtype):
    x, w, t = make(50, 400, 64, dtype, seed=12)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    logp, entropy = snack.token_logprobs(a, b, t)
    g, h = torch.randn(50, device="cuda"), torch.randn(50, device="cuda")
    (g * logp + h * entropy).sum().backward()
    ref = snack.score(x, w, t)
    assert torch.equal(logp, ref[0]) and torch.equal(entropy, ref[1])
    dx, dw = snack.score_grad(x, w, t, ref[4], g, h)
    assert torch.equal(a.grad, dx) and torch.equal(b.grad, dw)
    a.grad = None
    snack.token_logprobs(a, w, t)[0].sum().backward()  # one output and one input alone
    assert torch.equal(a.grad, snack.score_grad(x, w, t, ref[4], torch.ones(50, device="cuda"), torch.zeros(50, device="cuda"))[0])


@pytest.mark.parametrize("dtype,n", [("bf16", 100), ("f32", 100), ("f32", 10), ("f32", 3)])
def test_score_on_another_stream_and_in_a_graph(dtype, n):
    x, w, t = make(n, 900, 64, dtype, seed=13)
    g = torch.randn(n, device="cuda")

    def step(stream=None):
        got = snack.score(x, w, t, 5, stream=stream)
        return (*got, *snack.score_grad(x, w, t, got[4], g, g, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.mul_(0.5)
    t.copy_(t.flip(0))
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(held, step()))


def test_score_without_rows_and_refusals():
    x, w, t = make(6, 30, 16, "bf16", seed=14)
    none = snack.score(x[:0], w, t[:0], 3)
    assert [tuple(v.shape) for v in none] == [(0,), (0,), (0, 3), (0, 3), (2, 0)]
    dx, dw = snack.score_grad(x[:0], w, t[:0], none[4], none[0], none[1])
    assert dx.shape == (0, 16) and bool((dw == 0).all())
    state = snack.score(x, w, t)[4]
    g = torch.ones(6, device="cuda")
    for bad in (lambda: snack.score(x, w.float(), t), lambda: snack.score(x, w[:, :8], t), lambda: snack.score(x, w, t[:5]),
                lambda: snack.score(x, w, t.float()), lambda: snack.score(x.half(), w.half(), t), lambda: snack.score(x, w.cpu(), t),
                lambda: snack.score_grad(x, w, None, state, g), lambda: snack.score_grad(x, w, t, state[0], g),
                lambda: snack.score_grad(x, w, t, state, g[:3]), lambda: snack.score_grad(x, w, t, state.double(), g)):
        with pytest.raises(ValueError):
            bad()
    for top, status in ((-1, 1), (31, 1), (25, 7)):
        with pytest.raises(snack.SnackError) as e:
            snack.score(x, w, t, top)
        assert e.value.status == status


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2, 40, 200])
def test_order_of_logits_that_are_small_against_their_terms(n, dtype):
    """Terms whose sums reach 2^13 or so cancel: a rounding of such a sum to fp32 (2^-11) is larger than the steps between the
    fourteen largest logits (2^-12, near 2^-3), which differ by far more than roundings of numbers of their own size would.
    The products are multiples of 2^-14 and 64-bit sums of them exact."""
    vocab, width = 5000, 512
    gen = torch.Generator(device="cuda").manual_seed(n)
    half = width // 2 - 2
    x, w = torch.zeros(n, width, device="cuda"), torch.zeros(vocab, width, device="cuda")

    def eight_bits(*shape):  # from 1 to 16
        return torch.randint(128, 256, shape, generator=gen, device="cuda") / 2.0 ** torch.randint(4, 8, shape, generator=gen, device="cuda")

    big, terms = eight_bits(half), eight_bits(vocab, half)
    turn = torch.randperm(half, generator=gen, device="cuda")
    sign = 1 - 2 * torch.randint(0, 2, (n, 1), generator=gen, device="cuda")
    x[:, :half], x[:, half:2 * half] = sign * big, sign * big[turn]
    w[:, :half], w[:, half:2 * half] = terms, -terms[:, turn]
    x[:, -1] = 2.0 ** -6
    x[:, -2] = 2.0 ** -3
    near = torch.randperm(vocab, generator=gen, device="cuda")[:14]
    w[:, -2] = -8.0  # the others: -1
    w[near, -2] = 1.0
    w[near, -1] = torch.randperm(14, generator=gen, device="cuda").float() * 2.0 ** -6
    x, w = x.to(DTYPES[dtype]), w.to(DTYPES[dtype])
    want = Want(x, w, None, 6)
    assert torch.equal(want.ids[0], near[w[near, -1].float().argsort(descending=True)][:6])
    got = snack.score(x, w, top=6)
    assert torch.equal(got[2], want.ids)
    assert bool((got[3][:, 1:] <= got[3][:, :-1]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(1, 9000), (5, 40000), (40, 9000), (70, 40000), (200, 9000), (200, 40000)])
def test_equal_logits_of_many_groups_rank_by_id(n, vocab, dtype):
    """More groups of 32 equal logits than are ranked by counting (256), and than there is room for (1024)."""
    x, w, _ = make(n, vocab, 64, dtype, seed=1)
    x[0] = 0  # every logit 0
    got = snack.score(x, w, top=24)
    assert torch.equal(got[2][0], torch.arange(24, device="cuda"))
    assert bool(((got[3][0] + torch.log(torch.tensor(float(vocab)))).abs() <= 2.0 ** -15).all())
    Want(x, w, None, 24).check(got)
    w[:] = w[5]  # all of them, in every row
    w[vocab - 3:] *= 2  # and three beside, the largest or the lowest
    Want(x, w, None, 10).check(snack.score(x, w, top=10))


def test_equal_logits_in_pieces_of_the_vocabulary_rank_by_id():
    n, vocab = 8200, 50000  # 1.6 GB of logits
    x, w, _ = make(n, vocab, 64, "bf16", seed=2)
    x[::7] = 0
    w[:] = w[torch.arange(vocab, device="cuda") % 20000]
    ids = snack.score(x, w, top=24)[2]
    assert torch.equal(ids[::7], torch.arange(24, device="cuda").expand(len(ids[::7]), 24))
    for rows in (slice(0, 600), slice(n - 600, n)):
        assert torch.equal(ids[rows], Want(x[rows], w, None, 24).ids)


def test_gradients_where_logits_are_the_lowest():
    """Tokens with -inf logits get no probability: their rows of dw are 0, the others' as if they were not there.  dx is dz w, a
    product with their rows in it: 0 times -inf, NaN, in the column that has them, and the others' sum elsewhere."""
    x, w, t = make(70, 300, 64, "bf16", seed=7, ignored=0)
    x[:, 0], w[:, 0] = 1, 0
    gone = torch.arange(300, device="cuda") % 3 == 0
    t = torch.where(t % 3 == 0, (t + 1) % 300, t)
    kept = (~gone).nonzero()[:, 0]
    back = torch.full((300,), -1, device="cuda")
    back[kept] = torch.arange(len(kept), device="cuda")
    want = Want(x, w[kept].contiguous(), back[t])
    w[gone, 0] = float("-inf")
    g, h = (torch.randn(70, device="cuda", generator=torch.Generator(device="cuda").manual_seed(s)) for s in (1, 2))
    dx, dw = snack.score_grad(x, w, t, snack.score(x, w, t)[4], g, h)
    assert bool(torch.isnan(dx[:, 0]).all()) and bool((dw[gone] == 0).all())
    dx[:, 0] = 0  # w's kept entries of the column are 0
    want.check_grads(dx, dw[kept], g, h)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 12, 30, 130, 300])
def test_the_entropy_s_gradient_adds_up_to_nothing(n, dtype):
    """sum_v dz = -sum_v p (log p + H) = 0: dx in a column where every token has 1.  Logits near 640 that differ by 0.2: what
    log p + H is off by is common to all of a row, so logits that the gradient sums in another way than the statistics did (off
    by 10^-7 of themselves for each truncated addition) would show.  What may be left: the roundings of lse and H (2^-24 of each),
    H's own error (2^-17 of its two parts), dz's (2^-8 of each entry, or 2^-22) and dx's."""
    vocab, width = 8192, 4096
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = (torch.rand(n, width, device="cuda", generator=gen) + 0.5) * 0.4
    w = (0.75 + 0.5 * torch.rand(1, width, device="cuda", generator=gen)) * 0.4 + torch.randn(vocab, width, device="cuda", generator=gen) * 0.008
    x[:, 0], w[:, 0] = 0, 1
    x, w = x.to(DTYPES[dtype]), w.to(DTYPES[dtype])
    state = snack.score(x, w)[4]
    dx = snack.score_grad(x, w, None, state, dentropy=torch.ones(n, device="cuda"), want_dw=False)[0]
    want = Want(x, w, None)
    size = (want.p * (want.log_p + want.H[:, None]).abs()).sum(1)
    tol = 2.0 ** -24 * (want.lse + want.H) + 2.0 ** -17 * 2 * (1 + want.H) + size * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22)
    assert float(want.lse.min()) > 400 and 0.05 < float(size.mean()) < 0.5
    assert bool((dx[:, 0].abs().double() <= tol * (1 + HALF_ULP[dx.dtype])).all()), float((dx[:, 0].abs().double() / tol).max())
