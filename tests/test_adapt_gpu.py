"""Low-rank adapters beside a shared projection, and their gradients, against the definitions in 64 bits.

Tolerances, relative to T, the same expression of magnitudes (|s| |B| |A| |x| and so on).

A sum of K products (`sums(K)`): 16 products of bf16 operands and what is there go through one tensor core addition,
which keeps at least 23 bits of the largest and cuts the rest off: 2^-22 T each with the sum's own truncation, ceil(K / 16)
of them in a row at most, and up to 16 more additions of warps and blocks.  fp32 operands are three parts of 8 bits: what
is left out are products of a part below 2^-7 and one below 2^-15 of its operand, twice (2^-21 T with the smaller ones);
the six part products of 16 of K run through one such chain (6 additions of 2^-22 T at most, of which five move small sums:
12 2^-23 T), and are added in fp32, ceil(K / 16) + 16 times (2^-24 T).

h and dh enter their products as two bf16 parts (bf16 operands; each rounding leaves at most 2^-9 of what it rounds:
2^-18 T) or as three that hold all bits.  An output goes through two or three sums (of K and of the rank; of the rows for dA
and dB), the scale (2^-24) and one addition (2^-24 of base and product).  The result is rounded once: half an ulp of its type.
"""

import os
import sys

import pytest
import torch

from spmm_row_sorted_gb300 import snack

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # relative, at most (of a power of two)


def sums(k, dtype):
    steps = (k + 15) // 16 + 16
    return steps * 2.0 ** -22 if dtype == torch.bfloat16 else 2.0 ** -21 + 12 * 2.0 ** -23 + steps * 2.0 ** -24


def make_which(n, adapters, kind, seed, itype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "own":        # every row another one
        w = torch.arange(n) % adapters
    elif kind == "mixed":    # in any order, some rows without one, at both ends of the range
        w = torch.randint(-1, adapters + 1, (n,), generator=g)
        w[::7] = -100
    elif kind == "none":
        w = torch.where(torch.arange(n) % 2 == 0, -1, adapters)
    elif kind == "one":      # all the same one; the others have no rows
        w = torch.full((n,), adapters // 2)
    else:                    # "runs": requests' rows lie together
        w = torch.randint(-1, adapters, (max(1, n // 37 + 1),), generator=g).repeat_interleave(37)[:n]
    return w.to(itype).cuda()


def strided(n, width, gap, lead, dtype, seed, std=1.0):
    """[n, width] whose rows lie width + gap apart and start `lead` elements into a buffer of NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((n * (width + gap) + lead,), float("nan"), device="cuda", dtype=dtype)
    v = buf[lead:].view(n, width + gap)[:, :width]
    v.copy_(torch.empty(n, width, device="cuda").normal_(0, std, generator=g))
    return v


class Case:
    def __init__(self, n, adapters, rank, width, out, dtype, kind, gap=0, lead=0, scales=True, itype=torch.int64, seed=0):
        kind_t = DTYPES[dtype]
        self.x = strided(n, width, gap, lead, kind_t, seed + 1)
        self.base = strided(n, out, gap, lead, kind_t, seed + 2)
        self.dy = strided(n, out, gap, lead, kind_t, seed + 3)
        self.a = strided(adapters * rank, width, 0, lead, kind_t, seed + 4, width ** -0.5).view(adapters, rank, width)
        self.b = strided(adapters * out, rank, 0, lead, kind_t, seed + 5, rank ** -0.5).view(adapters, out, rank)
        self.scales = torch.linspace(-0.5, 2.0, adapters, device="cuda") if scales else None
        self.which = make_which(n, adapters, kind, seed, itype)

    def args(self):
        return self.a, self.b, self.which

    def want(self):
        """y, dx, da, db and their T, in 64 bits."""
        x, base, dy, a, b = (t.double() for t in (self.x, self.base, self.dy, self.a, self.b))
        k = len(a)
        s = self.scales.double() if self.scales is not None else torch.ones(k, dtype=torch.float64, device="cuda")
        val = [base.clone(), torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)]
        mag = [base.abs(), torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)]
        for j in range(k):
            rows = (self.which == j).nonzero()[:, 0]
            for out, f in ((val, lambda t: t), (mag, torch.abs)):
                xs, g, aj, bj, sj = f(x[rows]), f(dy[rows]), f(a[j]), f(b[j]), f(s[j])
                h, dh = xs @ aj.T, sj * (g @ bj)
                out[0][rows] += sj * (h @ bj.T)
                out[1][rows] = dh @ aj
                out[2][j] = dh.T @ xs
                out[3][j] = sj * (g.T @ h)
        return val, mag


def check(got, want, mag, rel, what):
    tol = rel * mag + HALF_ULP[got.dtype] * (want.abs() + rel * mag) + 2.0 ** -133  # the last: bf16's smallest step, halved
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float((got.double() - want).abs().max()))


def bounds(case):
    dtype, (n, width), out, rank = case.x.dtype, case.x.shape, case.base.shape[1], case.a.shape[1]
    down, back, across, rows = sums(width, dtype), sums(out, dtype), sums(rank, dtype), sums(n, dtype)
    one = 2.0 ** -17  # parts of h and dh, the scale and the addition
    return down + across + one, back + across + one, back + rows + one, down + rows + one


CASES = [
    # n, adapters, rank, width, out, dtype, kind, gap, lead
    (1, 1, 1, 1, 1, "f32", "one", 0, 0),
    (1, 1, 1, 1, 1, "bf16", "one", 0, 0),
    (1, 8, 16, 512, 384, "bf16", "one", 0, 0),
    (1, 3, 16, 512, 384, "bf16", "none", 0, 0),
    (2, 2, 8, 64, 64, "f32", "own", 0, 0),
    (16, 1, 16, 128, 96, "bf16", "one", 0, 0),
    (17, 1, 16, 128, 96, "bf16", "one", 0, 0),
    (63, 1, 8, 130, 62, "f32", "one", 0, 0),
    (64, 32, 16, 1024, 768, "bf16", "mixed", 0, 0),
    (64, 64, 16, 1024, 768, "bf16", "own", 0, 0),
    (65, 2, 32, 256, 520, "bf16", "one", 8, 0),
    (65, 2, 32, 256, 520, "f32", "one", 4, 0),
    (129, 5, 64, 320, 200, "bf16", "runs", 0, 0),
    (129, 5, 64, 320, 200, "f32", "runs", 0, 0),
    (200, 3, 100, 96, 333, "bf16", "mixed", 1, 1),
    (200, 3, 100, 96, 333, "f32", "mixed", 1, 1),
    (150, 4, 20, 1001, 77, "bf16", "runs", 3, 0),
    (150, 4, 20, 1001, 77, "f32", "runs", 3, 0),
    (100, 2, 128, 264, 136, "bf16", "mixed", 0, 0),
    (100, 2, 128, 264, 136, "f32", "mixed", 0, 0),
    (90, 2, 256, 72, 80, "bf16", "runs", 0, 8),
    (90, 2, 256, 72, 80, "f32", "runs", 0, 4),
    (90, 2, 255, 72, 80, "f32", "runs", 0, 0),
    (300, 700, 4, 40, 48, "f32", "mixed", 0, 0),      # more adapters than rows
    (300, 1500, 8, 40, 48, "bf16", "mixed", 0, 0),    # more than one block of the scan, fewer warps
    (50, 20000, 2, 8, 8, "f32", "mixed", 0, 0),       # a warp's counts fill the shared memory
    (3000, 3, 8, 72, 40, "bf16", "mixed", 0, 0),
    (9001, 2, 16, 64, 64, "bf16", "one", 0, 0),       # more rounds than a lane keeps keys
    (9001, 6, 5, 33, 65, "f32", "mixed", 0, 0),
    (70, 1, 16, 4096, 4096, "bf16", "one", 0, 0),     # clusters
    (70, 1, 16, 4096, 4096, "f32", "one", 0, 0),
    (2000, 1, 64, 256, 128, "bf16", "one", 0, 0),
]


@pytest.mark.parametrize("n,adapters,rank,width,out,dtype,kind,gap,lead", CASES)
def test_adapt_matches_definition(n, adapters, rank, width, out, dtype, kind, gap, lead):
    c = Case(n, adapters, rank, width, out, dtype, kind, gap, lead, itype=torch.int32 if n % 2 else torch.int64, seed=n)
    val, mag = c.want()
    rel = bounds(c)
    y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)
    check(y, val[0], mag[0], rel[0], "y")
    assert torch.equal(snack.adapt(c.x, c.base, *c.args(), c.scales), y)  # without h, and again the same bits
    outside = (c.which < 0) | (c.which >= adapters)
    assert torch.equal(y[outside], c.base[outside])
    dx, da, db = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
    check(dx, val[1], mag[1], rel[1], "dx")
    check(da, val[2], mag[2], rel[2], "da")
    check(db, val[3], mag[3], rel[3], "db")
    again = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
    assert all(torch.equal(p, q) for p, q in zip((dx, da, db), again))
    assert bool((dx[outside] == 0).all())
    unused = torch.ones(adapters, dtype=torch.bool, device="cuda")
    unused[c.which[~outside].long()] = False
    assert bool((da[unused] == 0).all()) and bool((db[unused] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adapt_in_place_without_a_base_and_into_wider_rows(dtype):
    c = Case(77, 5, 12, 90, 51, dtype, "mixed", gap=3, seed=4)
    y = snack.adapt(c.x, c.base, *c.args(), c.scales)
    buf = c.base.new_full((77, 60), 7.0)
    out = buf[:, 4:55]
    assert snack.adapt(c.x, c.base, *c.args(), c.scales, out=out) is out
    assert torch.equal(out, y) and bool((buf[:, :4] == 7).all()) and bool((buf[:, 55:] == 7).all())
    held = c.base.clone()
    mark = held._version
    snack.adapt(c.x, held, *c.args(), c.scales, out=held)
    assert torch.equal(held, y) and held._version > mark
    view = out[:]  # the same rows by another tensor
    out.copy_(c.base)
    snack.adapt(c.x, out, *c.args(), c.scales, out=view)
    assert torch.equal(out, y) and bool((buf[:, 55:] == 7).all())
    alone = snack.adapt(c.x, None, *c.args(), c.scales)
    assert torch.equal(alone, snack.adapt(c.x, torch.zeros_like(c.base), *c.args(), c.scales))
    ones = torch.ones(5, device="cuda")
    assert torch.equal(snack.adapt(c.x, c.base, *c.args()), snack.adapt(c.x, c.base, *c.args(), ones))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adapt_grad_adds_to_dx_and_leaves_out_what_is_not_asked_for(dtype):
    c = Case(130, 4, 16, 200, 72, dtype, "mixed", seed=8)
    h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)[1]
    dx, da, db = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
    buf = torch.full((130, 209), 3.0, device="cuda", dtype=c.x.dtype)
    into = buf[:, :200]
    start = strided(130, 200, 0, 0, c.x.dtype, 9)
    into.copy_(start)
    got = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, dx=into)[0]
    assert got is into and bool((buf[:, 200:] == 3).all())
    val, mag = c.want()
    check(into, val[1] + start.double(), mag[1] + start.double().abs(), bounds(c)[1], "dx added")
    outside = (c.which < 0) | (c.which >= 4)
    assert torch.equal(into[outside], start[outside])
    only = snack.adapt_grad(c.x, c.dy, *c.args(), None, c.scales, want_db=False)
    assert torch.equal(only[0], dx) and torch.equal(only[1], da) and only[2] is None
    only = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, want_dx=False, want_da=False)
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)
    assert snack.adapt_grad(c.x, c.dy, *c.args(), h, want_dx=False, want_da=False, want_db=False) == (None, None, None)


def test_rows_without_an_adapter_stay_out_whatever_they_hold():
    for dtype in ("f32", "bf16"):
        c = Case(100, 3, 8, 64, 64, dtype, "mixed", seed=2)
        outside = (c.which < 0) | (c.which >= 3)
        want = snack.adapt(c.x, c.base, *c.args(), keep=True)
        grads = snack.adapt_grad(c.x, c.dy, *c.args(), want[1])
        c.x[outside] = float("nan")
        c.dy[outside] = float("inf")
        y, h = snack.adapt(c.x, c.base, *c.args(), keep=True)
        assert torch.equal(y, want[0])
        h[outside] = float("nan")
        for p, q in zip(grads, snack.adapt_grad(c.x, c.dy, *c.args(), h)):
            assert torch.equal(p, q)
        # and one bad row spoils its own results, no other row's
        bad = int((c.which == 1).nonzero()[0])
        c.x[bad, 3] = float("inf")
        y2 = snack.adapt(c.x, c.base, *c.args())
        rest = torch.arange(100, device="cuda") != bad
        assert torch.equal(y2[rest], y[rest]) and not torch.isfinite(y2[bad]).all()


def test_adapt_without_rows():
    for dtype in DTYPES.values():
        x, base = torch.empty(0, 24, device="cuda", dtype=dtype), torch.empty(0, 40, device="cuda", dtype=dtype)
        a, b = torch.ones(3, 4, 24, device="cuda", dtype=dtype), torch.ones(3, 40, 4, device="cuda", dtype=dtype)
        which = torch.empty(0, device="cuda", dtype=torch.int64)
        y, h = snack.adapt(x, base, a, b, which, keep=True)
        assert y.shape == (0, 40) and h.shape == (0, 4)
        dx, da, db = snack.adapt_grad(x, base, a, b, which, h)
        assert dx.shape == (0, 24) and bool((da == 0).all()) and bool((db == 0).all()) and da.shape == a.shape and db.shape == b.shape


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adapted_gives_autograd_the_gradients(dtype):
    c = Case(70, 3, 8, 48, 56, dtype, "mixed", seed=6)
    leaves = [t.clone().requires_grad_() for t in (c.x, c.base, c.a, c.b)]
    y = snack.adapted(*leaves, c.which, c.scales)
    h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)[1]
    y.backward(c.dy)
    dx, da, db = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
    for leaf, want in zip(leaves, (dx, c.dy, da, db)):
        assert torch.equal(leaf.grad, want)
    # only what is needed
    a = c.a.clone().requires_grad_()
    snack.adapted(c.x, c.base, a, c.b, c.which, c.scales).backward(c.dy)
    assert torch.equal(a.grad, da)


def test_gradients_against_differences():
    """The outputs are linear in each of x, A and B: central differences with steps of any size are exact but for the
    roundings of y, which check's tolerance of y bounds (twice, over twice the step 1, in the sum over dy)."""
    c = Case(60, 3, 8, 40, 44, "f32", "mixed", seed=5)
    h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)[1]
    grads = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i, grad in zip((0, 2, 3), grads):
        parts = [c.x, c.base, c.a, c.b]
        step = torch.randn(parts[i].shape, device="cuda", generator=g)
        side = []
        for sign in (1.0, -1.0):
            moved = list(parts)
            moved[i] = parts[i] + sign * step
            side.append(snack.adapt(*moved, c.which, c.scales).double())
        got = ((side[0] - side[1]) / 2 * c.dy.double()).sum()
        want = (grad.double() * step.double()).sum()
        # magnitudes: |dy| |y| with every factor's magnitude doubled at most, at 2^-17 of each term (bounds() of these sizes)
        m = Case(60, 3, 8, 40, 44, "f32", "mixed", seed=5)
        m.x, m.a, m.b = (t.abs() + (step.abs() if k == i else 0) for k, t in ((0, c.x), (2, c.a), (3, c.b)))
        size = (m.want()[1][0] * c.dy.double().abs()).sum()
        assert abs(float(got - want)) <= 2 * sum(bounds(c)) * float(size)


def test_adapt_on_another_stream_and_in_a_graph():
    c = Case(200, 6, 16, 256, 192, "bf16", "runs", seed=3)

    def step(stream=None):
        y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True, stream=stream)
        return (y, *snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    c.which.copy_(c.which.flip(0))  # the captured call reads the adapters of its rows anew
    c.x.mul_(2)
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(held, step()))


def test_sparse_layer_with_adapters():
    from spmm_row_sorted_gb300 import workloads as wl

    lay = wl.make_layer(96, 80, density=0.2, val_std=0.2, seed=1)
    row, col, val = (torch.from_numpy(t).cuda() for t in (lay.row, lay.col, lay.val))
    layer = snack.SparseLinear(96, 80, row, col, val, torch.ones(96, device="cuda"), max_batch=64)
    c = Case(50, 4, 8, 80, 96, "f32", "mixed", seed=7)
    y, h = layer.forward_adapted(c.x, *c.args(), c.scales, keep=True)
    base = layer.forward(c.x)
    want, h2 = snack.adapt(c.x, base, *c.args(), c.scales, keep=True)
    inside = (c.which >= 0) & (c.which < 4)
    assert torch.equal(y, want) and torch.equal(h[inside], h2[inside])
    assert torch.equal(layer.forward_adapted(c.x, *c.args(), c.scales), want)
    # both parts' gradients: the layer's, and the adapters' added to it
    x, a, b = (t.clone().requires_grad_() for t in (c.x, c.a, c.b))
    snack.adapted(x, snack.sparse_linear(x, layer), a, b, c.which, c.scales).backward(c.dy)
    dx = layer.grad_input(c.dy)
    got = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, dx=dx)
    assert torch.equal(a.grad, got[1]) and torch.equal(b.grad, got[2])
    # autograd adds two rounded parts where the call adds once: an addition's rounding apart
    assert bool(((x.grad - got[0]).abs() <= 2.0 ** -22 * (x.grad.abs() + 2 * layer.grad_input(c.dy).abs())).all())
    layer.close()


# rows by the hundred: tiles of 128, several columns' units and tiles per block, tails of columns, every step of the rank
MANY = [
    # n, adapters, rank, width, out, dtype, kind, gap
    (700, 3, 4, 72, 1160, "bf16", "mixed", 0),
    (513, 2, 12, 136, 1032, "bf16", "runs", 0),
    (1030, 4, 16, 200, 2048, "bf16", "mixed", 8),
    (700, 3, 48, 264, 1043, "bf16", "runs", 5),      # the last columns of a row short of an access
    (641, 2, 64, 128, 3080, "bf16", "mixed", 0),
    (700, 3, 100, 1000, 520, "bf16", "runs", 0),     # the matrix's rows on 8 bytes
    (513, 2, 128, 192, 264, "bf16", "mixed", 0),
    (400, 2, 192, 96, 392, "bf16", "runs", 0),
    (400, 2, 256, 264, 392, "bf16", "mixed", 0),
    (700, 3, 7, 200, 264, "bf16", "runs", 0),        # the matrix's rows on 2
    (600, 2, 20, 161, 333, "bf16", "mixed", 3),
    (600, 2, 20, 161, 333, "f32", "mixed", 3),
    (600, 2, 40, 160, 334, "f32", "runs", 2),
]


@pytest.mark.parametrize("n,adapters,rank,width,out,dtype,kind,gap", MANY)
def test_adapt_of_many_rows_matches_definition(n, adapters, rank, width, out, dtype, kind, gap):
    c = Case(n, adapters, rank, width, out, dtype, kind, gap, seed=n)
    val, mag = c.want()
    rel = bounds(c)
    y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)
    check(y, val[0], mag[0], rel[0], "y")
    outside = (c.which < 0) | (c.which >= adapters)
    assert torch.equal(y[outside], c.base[outside])
    held = strided(n, out, gap, 0, c.x.dtype, n + 2)  # the base's values, to be overwritten
    wide = held._base if held._base is not None else held
    gaps = torch.isnan(wide).sum()
    assert torch.equal(snack.adapt(c.x, held, *c.args(), c.scales, out=held), y) and torch.isnan(wide).sum() == gaps
    assert torch.equal(snack.adapt(c.x, None, *c.args(), c.scales), snack.adapt(c.x, torch.zeros_like(c.base), *c.args(), c.scales))
    dx, da, db = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
    for got, i, what in ((dx, 1, "dx"), (da, 2, "da"), (db, 3, "db")):
        check(got, val[i], mag[i], rel[i], what)
    assert bool((dx[outside] == 0).all())
    into = strided(n, width, gap, 0, c.x.dtype, n + 9)
    start = into.clone()
    snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, dx=into)
    check(into, val[1] + start.double(), mag[1] + start.double().abs(), rel[1], "dx added")
    assert torch.equal(into[outside], start[outside])


@pytest.mark.parametrize("lead", [1, 2, 3, 4, 5, 6, 7])
def test_adapt_of_rows_that_lie_anywhere(lead):
    """Starts at every element of an access, rows of odd and even steps, matrices too."""
    for n, rank, width, out, gap in ((300, 9, 133, 141, 0), (270, 33, 65, 130, 1), (290, 3, 130, 71, 2)):
        c = Case(n, 3, rank, width, out, "bf16", "runs", gap, lead, seed=lead)
        val, mag = c.want()
        rel = bounds(c)
        y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)
        grads = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)
        for got, i, what in ((y, 0, "y"), (grads[0], 1, "dx"), (grads[1], 2, "da"), (grads[2], 3, "db")):
            check(got, val[i], mag[i], rel[i], what)
        buf = torch.full((n * (out + gap) + lead + 9,), 7.0, device="cuda", dtype=torch.bfloat16)
        into = buf[lead:lead + n * (out + gap)].view(n, out + gap)[:, :out]
        snack.adapt(c.x, c.base, *c.args(), c.scales, out=into)
        assert torch.equal(into, y)
        into.fill_(7.0)
        assert bool((buf == 7).all())  # nothing beside the rows was written


@pytest.mark.parametrize("rank", [192, 193, 208, 240, 241, 255])
@pytest.mark.parametrize("n", [3, 70, 300])
def test_adapt_of_the_highest_ranks(n, rank):
    for dtype in ("f32", "bf16"):
        c = Case(n, 2, rank, 72, 80, dtype, "runs", 0, 0, seed=n)
        val, mag = c.want()
        rel = bounds(c)
        y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)
        for got, i, what in zip((y, *snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)), range(4), ("y", "dx", "da", "db")):
            check(got, val[i], mag[i], rel[i], what)


@pytest.mark.parametrize("n,adapters", [(257, 255), (257, 256), (511, 1), (1024, 9), (2047, 255), (2048, 40), (2049, 40), (2049, 3)])
@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
def test_adapt_files_rows_by_every_way(n, adapters, kind):
    """Around the sizes up to which the first product's blocks file the rows themselves."""
    for dtype, rank in (("f32", 3), ("bf16", 8), ("f32", 40)):
        c = Case(n, adapters, rank, 40, 24, dtype, kind, 0, 0, seed=n, itype=torch.int32 if n % 2 else torch.int64)
        val, mag = c.want()
        rel = bounds(c)
        y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)
        for got, i, what in zip((y, *snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales)), range(4), ("y", "dx", "da", "db")):
            check(got, val[i], mag[i], rel[i], what)
        only = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, want_dx=False, want_da=False)[2]
        check(only, val[3], mag[3], rel[3], "db alone")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_row_in_place_by_another_tensor(dtype):
    """Of one row the step means nothing: a view of a wider buffer is the same row, whatever its step."""
    c = Case(1, 2, 12, 90, 51, dtype, "one", gap=3, seed=4)
    y = snack.adapt(c.x, c.base, *c.args(), c.scales)
    buf = c.base.new_full((1, 60), 7.0)
    out, view = buf[:, 4:55], buf[:, 4:55]
    out.copy_(c.base)
    snack.adapt(c.x, out, *c.args(), c.scales, out=view)
    assert torch.equal(out, y) and bool((buf[:, :4] == 7).all()) and bool((buf[:, 55:] == 7).all())
    out.copy_(c.base)
    without = torch.full_like(c.which, -1)  # no adapter: the base stays
    snack.adapt(c.x, out, c.a, c.b, without, c.scales, out=view)
    assert torch.equal(out, c.base) and bool((buf[:, 55:] == 7).all())


def positive(rows, width, seed, dtype=torch.bfloat16):
    """Values from 1/2 to 3/2, of one sign: truncated sums of them are all off to the same side."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(rows, width, device="cuda", dtype=dtype)
    for part in out.split(max(1, (1 << 26) // width)):
        part.copy_(torch.rand(part.shape, device="cuda", generator=g) + 0.5)
    return out


# additions of a run on the tensor core: its sum is added, rounded to nearest, to what came before
RUN_OUTER = 528


@pytest.mark.parametrize("rank", [32, 64])
def test_matrices_gradients_over_millions_of_rows_are_sums_in_fp32(rank):
    """dA and dB of one adapter over 2^21 rows of one sign, bf16.  Their mean relative error has none of the roundings to
    bf16 in it: those of m entries, independent (every row and column has a scale of its own) and at most 2^-8 each, add up
    to a mean above 2^-8 sqrt(2 ln(2e12) / m) once in 10^12 (Hoeffding).  What is left is off to one side: a run's additions,
    2^-22 each at most, the second parts of h and dh (2^-17), and h and dh themselves (20 additions of 2^-22)."""
    n, width, out = 1 << 21, 512, 256
    g = torch.Generator(device="cuda").manual_seed(5)

    def scales(k):
        return 1 + torch.rand(k, device="cuda", generator=g)

    x, dy = positive(n, width, 1).mul_(scales(width)), positive(n, out, 2).mul_(scales(out))
    a, b = positive(rank, width, 3).mul_(scales(rank)[:, None]).view(1, rank, width), positive(out, rank, 4).mul_(scales(rank)).view(1, out, rank)
    which = torch.zeros(n, device="cuda", dtype=torch.int64)
    h = snack.adapt(x, dy, a, b, which, keep=True)[1]
    _, da, db = snack.adapt_grad(x, dy, a, b, which, h, want_dx=False)
    want_a, want_b = torch.zeros(rank, width, device="cuda", dtype=torch.float64), torch.zeros(out, rank, device="cuda", dtype=torch.float64)
    for i in range(0, n, 1 << 17):
        xs, gs = x[i:i + (1 << 17)].double(), dy[i:i + (1 << 17)].double()
        want_a += (gs @ b[0].double()).T @ xs
        want_b += gs.T @ (xs @ a[0].double().T)
    for got, want in ((da[0], want_a), (db[0], want_b)):
        chance = 2.0 ** -8 * (2 * 28.33 / want.numel()) ** 0.5
        assert abs(float(((got - want) / want).mean())) <= chance + RUN_OUTER * 2.0 ** -22 + 2.0 ** -17 + 20 * 2.0 ** -22


@pytest.mark.parametrize("n,adapters,rank,gap,kind", [(33792, 1, 64, 0, "one"), (33793, 1, 20, 0, "one"), (33856, 1, 64, 1, "one"), (70001, 2, 32, 3, "mixed"),
                                                      (70001, 2, 65, 0, "runs"), (101377, 3, 8, 0, "one")])
def test_matrices_gradients_around_the_ends_of_runs(n, adapters, rank, gap, kind):
    """A cluster of eight blocks has 33792 rows in whole runs: one more run with no, one or a few rows, and several."""
    c = Case(n, adapters, rank, 40, 24, "bf16", kind, gap, 0, seed=n)
    val, mag = c.want()
    rel = bounds(c)
    h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)[1]
    _, da, db = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, want_dx=False)
    check(da, val[2], mag[2], rel[2], "da")
    check(db, val[3], mag[3], rel[3], "db")
    again = snack.adapt_grad(c.x, c.dy, *c.args(), h, c.scales, want_dx=False)
    assert torch.equal(again[1], da) and torch.equal(again[2], db)


@pytest.mark.parametrize("n,adapters,rank,run,chain", [(300, 1, 16, 64, 1 << 13), (300, 2, 160, 64, 1 << 13), (100, 64, 2, 1, 1 << 12), (3, 1, 16, 1, 1 << 10)])
def test_h_of_the_widest_rows_is_a_sum_in_fp32(n, adapters, rank, run, chain):
    """Nearly 2^20 terms of one sign per entry, bf16, 16 of them at a time: `chain` such additions one after the other by a
    cluster's block (of eight, by 128 rows) or a warp (eight in each of two or eight blocks, by few rows).  Of each `run` of
    them the tensor core cuts off at most 2^-22 per addition; the runs, and the sums of warps and blocks (16), are added in
    fp32, 2^-24 each."""
    width = (1 << 20) - 8
    x, a = positive(n, width, 1), positive(adapters * rank, width, 2).view(adapters, rank, width)
    b = torch.zeros(adapters, 1, rank, device="cuda", dtype=torch.bfloat16)
    which = torch.arange(n, device="cuda") % adapters
    h = snack.adapt(x, None, a, b, which, keep=True)[1]
    want = torch.zeros(n, rank, device="cuda", dtype=torch.float64)
    for c in range(0, width, 1 << 16):
        for k in range(adapters):
            want[which == k] += x[which == k, c:c + (1 << 16)].double() @ a[k, :, c:c + (1 << 16)].double().T
    assert float(((h - want) / want).abs().max()) <= run * 2.0 ** -22 + (chain / run + 17) * 2.0 ** -24


@pytest.mark.parametrize("n,adapters,rank,width", [(*c, w) for c in ((257, 1, 20), (600, 40, 64), (300, 2, 130), (300, 1, 256))
                                                   for w in (8128, 8192, 8256, 16400, 33001)] + [(20000, 2, 16, 2112), (9000, 3, 100, 4097)])
def test_h_around_the_ends_of_runs(n, adapters, rank, width):
    """Clusters of eight, one and two blocks with steps of 64 in runs of sixteen: the last run full, with one step, alone."""
    c = Case(n, adapters, rank, width, 24, "bf16", "mixed", seed=n)
    val, mag = c.want()
    rel = bounds(c)
    y, h = snack.adapt(c.x, c.base, *c.args(), c.scales, keep=True)
    check(y, val[0], mag[0], rel[0], "y")
    own = (c.which >= 0) & (c.which < adapters)
    x, a = c.x[own].double(), c.a.double()[c.which[own].long()]
    tol = sums(width, torch.bfloat16) * torch.einsum("ni,nri->nr", x.abs(), a.abs()) if n * rank * width < 1 << 28 else None
    if tol is not None:
        assert bool(((h[own] - torch.einsum("ni,nri->nr", x, a)).abs() <= tol).all())
    c = Case(n, adapters, rank, 24, width, "bf16", "mixed", seed=n)  # dh
    val, mag = c.want()
    dx, da, _ = snack.adapt_grad(c.x, c.dy, *c.args(), None, c.scales, want_db=False)
    check(dx, val[1], mag[1], bounds(c)[1], "dx")
    check(da, val[2], mag[2], bounds(c)[2], "da")
