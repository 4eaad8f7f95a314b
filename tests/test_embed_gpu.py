"""Embedding lookup and its gradient against the definitions in 64 bits.

Tolerances.  Forward: one product of the scale (rounded to fp32) and a stored
value, rounded once more: |err| <= 2^-23 |y| in fp32 (two roundings of half an
ulp), and half a bf16 ulp more in bf16.  Gradient: a row of m terms summed in
fp32, in any grouping, is within m 2^-24 of the sum of its terms' magnitudes
T (one rounding per addition), plus two roundings for the scale: (m + 2) 2^-24
T; a bf16 result adds half a bf16 ulp.
"""

import numpy as np
import pytest
import torch

from spmm_row_sorted_gb300 import snack

from gpu_util import assert_close_T, bf16_half_ulp, f64

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def make_ids(n, vocab, kind, seed, itype):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        ids = rng.integers(0, vocab, n)
    elif kind == "skewed":  # a few ids take most tokens
        ids = np.minimum((vocab * rng.random(n) ** 6).astype(np.int64), vocab - 1)
    elif kind == "one":
        ids = np.full(n, vocab // 2)
    elif kind == "outside":  # no token names a row
        ids = np.where(rng.random(n) < 0.5, -1, vocab)
    else:  # "padded": some ids outside, at both ends
        ids = rng.integers(0, vocab, n)
        ids[rng.random(n) < 0.3] = -1
        ids[rng.random(n) < 0.1] = vocab
        ids[rng.random(n) < 0.05] = -100
    return torch.from_numpy(ids.astype(np.int64)).to(itype).cuda()


def strided(n, width, gap, lead, dtype, seed, std=1.0):
    """[n, width] whose rows lie width + gap apart and start `lead` elements into their buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((n * (width + gap) + lead,), float("nan"), device="cuda", dtype=DTYPES[dtype])
    v = buf[lead:].view(n, width + gap)[:, :width]
    v.copy_(torch.empty(n, width, device="cuda").normal_(0, std, generator=g))
    return v


LOOKUPS = [
    # n, vocab, width, dtype, kind, gap, lead
    (1, 7, 8, "f32", "uniform", 0, 0),
    (1, 1, 1, "bf16", "uniform", 0, 0),
    (5, 100, 64, "bf16", "padded", 0, 0),
    (33, 1000, 4096, "bf16", "uniform", 0, 0),
    (257, 1000, 1001, "f32", "padded", 0, 0),
    (257, 1000, 1001, "bf16", "padded", 0, 0),
    (100, 333, 770, "bf16", "skewed", 0, 0),     # 4-byte accesses
    (100, 333, 772, "bf16", "skewed", 0, 0),     # 8-byte accesses
    (100, 333, 770, "f32", "skewed", 2, 0),      # 8-byte accesses
    (100, 333, 768, "f32", "padded", 3, 1),      # rows off every boundary
    (64, 50, 128, "bf16", "outside", 8, 8),
]


@pytest.mark.parametrize("itype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("n,vocab,width,dtype,kind,gap,lead", LOOKUPS)
def test_embed_matches_definition(n, vocab, width, dtype, kind, gap, lead, itype):
    table = strided(vocab, width, gap, lead, dtype, seed=n)
    ids = make_ids(n, vocab, kind, n, itype)
    scale = 1.7
    y = snack.embed(ids, table, scale)
    t, i = f64(table), ids.cpu().numpy().astype(np.int64)
    inside = (i >= 0) & (i < vocab)
    ref = np.where(inside[:, None], scale * t[np.where(inside, i, 0)], 0.0)
    assert y.shape == (n, width)
    err = np.abs(f64(y) - ref)
    bound = 2.0 ** -23 * np.abs(ref)
    if dtype == "bf16":
        bound = bound + bf16_half_ulp(np.abs(ref) * (1 + 2.0 ** -23))
    assert np.all(err <= bound)
    assert not np.any(f64(y)[~inside])


def test_embed_scale_one_copies_bits_and_shapes():
    table = strided(50, 96, 0, 0, "bf16", seed=3)
    ids = make_ids(24, 50, "uniform", 1, torch.int64).view(2, 3, 4)
    y = snack.embed(ids, table)
    assert y.shape == (2, 3, 4, 96)
    assert torch.equal(y, table[ids])
    assert snack.embed(ids[:0], table).shape == (0, 3, 4, 96)


def test_embed_leaves_the_gaps_of_its_output():
    table = strided(20, 30, 0, 0, "f32", seed=5)
    ids = make_ids(9, 20, "padded", 2, torch.int64)
    buf = torch.full((9, 37), 7.0, device="cuda")
    snack.embed(ids, table, 2.0, out=buf[:, 4:34])
    assert torch.all(buf[:, :4] == 7.0) and torch.all(buf[:, 34:] == 7.0)
    assert torch.equal(buf[:, 4:34].contiguous(), snack.embed(ids, table, 2.0))


GRADS = [
    # n, vocab, width, dtype, kind, gap, lead
    (0, 10, 16, "f32", "uniform", 0, 0),
    (1, 5, 8, "f32", "uniform", 0, 0),
    (1, 1, 1, "bf16", "uniform", 0, 0),
    (7, 3, 40, "bf16", "uniform", 0, 0),
    (8, 1000, 64, "f32", "outside", 0, 0),
    (31, 100, 1001, "f32", "padded", 0, 0),
    (32, 100, 1001, "bf16", "padded", 0, 0),
    (1023, 500, 768, "f32", "skewed", 5, 0),
    (1024, 500, 770, "bf16", "skewed", 0, 0),
    (1025, 500, 772, "bf16", "skewed", 0, 0),
    (4097, 37, 128, "bf16", "uniform", 0, 0),
    (3000, 100, 256, "f32", "one", 0, 0),        # one run over every chunk
    (8192, 4000, 512, "bf16", "padded", 0, 0),   # the last size that counts places
    (8193, 4000, 512, "bf16", "padded", 0, 0),   # the first that sorts by digits
    (20001, 255, 130, "f32", "skewed", 0, 1),    # one digit
    (20000, 256, 136, "bf16", "uniform", 0, 0),  # keys of nine bits
    (50000, 70000, 33, "f32", "skewed", 0, 0),   # three digits
    (70001, 300, 64, "f32", "one", 0, 0),
]


def grad_ref(ids, dout, vocab, scale):
    i = ids.cpu().numpy().astype(np.int64)
    inside = (i >= 0) & (i < vocab)
    d = f64(dout)
    out, mag, m = np.zeros((vocab, d.shape[1])), np.zeros((vocab, d.shape[1])), np.zeros(vocab)
    np.add.at(out, i[inside], d[inside])
    np.add.at(mag, i[inside], np.abs(d[inside]))
    np.add.at(m, i[inside], 1.0)
    return scale * out, abs(scale) * mag, m


def check_grad(got, ref, mag, m, dtype):
    bound = (m[:, None] + 2) * U * mag
    if dtype == "bf16":
        bound = bound + bf16_half_ulp(np.abs(ref) + bound)
    assert np.all(np.abs(f64(got) - ref) <= bound)
    assert not np.any(f64(got)[m == 0])


@pytest.mark.parametrize("n,vocab,width,dtype,kind,gap,lead", GRADS)
def test_embed_grad_matches_definition(n, vocab, width, dtype, kind, gap, lead):
    ids = make_ids(n, vocab, kind, n + 1, torch.int64 if n % 2 else torch.int32)
    dout = strided(n, width, gap, lead, dtype, seed=n)
    out = torch.full((vocab, width), float("nan"), device="cuda", dtype=DTYPES[dtype])
    g = snack.embed_grad(ids, dout, vocab, 0.7, out=out)
    ref, mag, m = grad_ref(ids, dout, vocab, 0.7)
    check_grad(g, ref, mag, m, dtype)
    assert torch.equal(g, snack.embed_grad(ids, dout, vocab, 0.7))  # repeats bit for bit


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_grad_accumulates(dtype):
    n, vocab, width = 500, 90, 200
    ids = make_ids(n, vocab, "skewed", 3, torch.int32)
    ids[ids > 60] = -1  # rows that no token names
    dout = strided(n, width, 0, 0, dtype, seed=4)
    start = strided(vocab, width, 0, 0, dtype, seed=5)
    out = start.clone()
    snack.embed_grad(ids, dout, vocab, 0.5, out=out, accumulate=True)
    ref, mag, m = grad_ref(ids, dout, vocab, 0.5)
    check = f64(out)
    s = f64(start)
    bound = (m[:, None] + 3) * U * (mag + np.abs(s))
    if dtype == "bf16":
        bound = bound + bf16_half_ulp(np.abs(ref + s) + bound)
    assert np.all(np.abs(check - (ref + s)) <= bound)
    assert torch.equal(out[torch.from_numpy(m == 0).cuda()], start[torch.from_numpy(m == 0).cuda()])


def test_embedding_autograd_matches_differences():
    vocab, width = 12, 6
    table = strided(vocab, width, 0, 0, "f32", seed=8).contiguous().requires_grad_()
    ids = make_ids(40, vocab, "padded", 9, torch.int64).view(4, 10)
    weight = torch.randn(4, 10, width, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    (snack.embedding(ids, table, 1.5) * weight).sum().backward()
    # linear in the table: central differences are exact but for rounding (values below 16, sums of 240 terms)
    base = table.detach()
    for r, c in [(0, 0), (5, 3), (11, 5)]:
        lo, hi = base.clone(), base.clone()
        lo[r, c] -= 0.5
        hi[r, c] += 0.5
        diff = (snack.embed(ids, hi, 1.5).double() * weight).sum() - (snack.embed(ids, lo, 1.5).double() * weight).sum()
        assert abs(float(diff) - float(table.grad[r, c])) < 1e-4


def test_embed_on_another_stream():
    n, vocab, width = 2000, 700, 256
    ids = make_ids(n, vocab, "skewed", 1, torch.int64)
    table, dout = strided(vocab, width, 0, 0, "bf16", 1), strided(n, width, 0, 0, "bf16", 2)
    want = snack.embed(ids, table), snack.embed_grad(ids, dout, vocab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = snack.embed(ids, table, stream=side), snack.embed_grad(ids, dout, vocab, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_embed_refusals():
    table = torch.zeros(10, 8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        snack.embed(ids.float(), table)
    with pytest.raises(ValueError):
        snack.embed(ids, table.half())
    with pytest.raises(ValueError):
        snack.embed(ids.cpu(), table)
    with pytest.raises(ValueError):
        snack.embed(ids, table, out=torch.zeros(4, 7, device="cuda"))
    with pytest.raises(snack.SnackError):
        snack.embed(ids, table, out=table[:4])  # overlaps its table
    with pytest.raises(ValueError):
        snack.embed_grad(ids, torch.zeros(3, 8, device="cuda"), 10)
    with pytest.raises(ValueError):
        snack.embed_grad(ids, torch.zeros(4, 8, device="cuda"), 10, accumulate=True)
    with pytest.raises(snack.SnackError):
        snack.embed_grad(ids, torch.zeros(4, 8, device="cuda"), 0)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    d = torch.zeros(4000, 8, device="cuda")
    with pytest.raises(snack.SnackError) as e:
        snack.snack_embed_grad(torch.zeros(4000, dtype=torch.int64, device="cuda"), d, 1.0, False, table, ws)
    assert e.value.status == 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_grad_leaves_the_gaps_of_its_output(dtype):
    n, vocab, width = 700, 300, 52
    ids = make_ids(n, vocab, "padded", 4, torch.int64)
    dout = strided(n, width, 0, 0, dtype, seed=9)
    want = snack.embed_grad(ids, dout, vocab, 0.5)
    for lead, gap in ((0, 4), (1, 3), (8, 12)):
        buf = torch.full((vocab * (width + gap) + lead,), 7.0, device="cuda", dtype=DTYPES[dtype])
        out = buf[lead:].view(vocab, width + gap)[:, :width]
        snack.embed_grad(ids, dout, vocab, 0.5, out=out)
        assert torch.equal(out.contiguous(), want)
        assert torch.all(buf[lead:].view(vocab, width + gap)[:, width:] == 7.0) and torch.all(buf[:lead] == 7.0)


def test_embedding_refuses_a_second_derivative():
    table = torch.randn(10, 8, device="cuda", requires_grad=True)
    y = snack.embedding(torch.arange(4, device="cuda"), table)
    up = torch.ones(4, 8, device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad(y, table, up, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_outputs_given_are_seen_by_autograd():
    table = strided(30, 16, 0, 0, "f32", seed=1)
    ids = make_ids(8, 30, "uniform", 1, torch.int64)
    buf = torch.zeros(8, 16, device="cuda")
    before = buf._version
    snack.embed(ids, table, out=buf)
    assert buf._version > before
    grad = torch.zeros(30, 16, device="cuda")
    for accumulate in (False, True):
        before = grad._version
        snack.embed_grad(ids, buf, 30, out=grad, accumulate=accumulate)
        assert grad._version > before
    with torch.inference_mode():
        held = torch.zeros(8, 16, device="cuda")
        snack.embed(ids, table, out=held)
    snack.embed(ids, table, out=held)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,width,dtype,kind", [
    (4095, 3000, 24, "f32", "skewed"), (4096, 3000, 24, "f32", "padded"),  # places counted up to 4096 tokens,
    (4097, 3000, 24, "f32", "padded"), (9000, 511, 24, "bf16", "skewed"),  # from there sorted by one cluster of blocks:
    (20000, 512, 16, "f32", "uniform"),                                    #  keys of nine bits, of ten (two passes),
    (30000, 2 ** 18 - 1, 8, "bf16", "skewed"),                             #  of 18 (two passes of nine),
    (30000, 2 ** 18, 8, "bf16", "padded"), (65535, 2 ** 21, 2, "f32", "uniform"),  # of 19 and 22 (three),
    (5000, 2 ** 27 + 1, 1, "bf16", "skewed"), (65536, 2 ** 28, 1, "bf16", "padded"),  # of 28 and 29 (four);
    (65536, 700, 16, "f32", "one"), (65536, 700, 16, "f32", "padded"),
    (65537, 700, 16, "f32", "padded"), (65537, 2 ** 18, 8, "bf16", "skewed"),  # and over the whole device above 65536:
    (200001, 70000, 4, "f32", "uniform"), (70000, 2 ** 27 + 1, 1, "bf16", "uniform"),  # three and four bytes of a key
    (300000, 9, 40, "f32", "skewed"),                                          # long runs over many chunks
])
def test_embed_grad_sorts_of_every_size(n, vocab, width, dtype, kind, accumulate):
    ids = make_ids(n, vocab, kind, n + vocab, torch.int64 if n % 2 else torch.int32)
    dout = strided(n, width, 0, 0, dtype, seed=n)
    start = torch.full((vocab, width), 0.75, device="cuda", dtype=DTYPES[dtype])
    out = start.clone()
    snack.embed_grad(ids, dout, vocab, 0.5, out=out, accumulate=accumulate)
    inside = (ids >= 0) & (ids < vocab)
    rows, at, m = torch.unique(ids[inside].long(), return_inverse=True, return_counts=True)
    d = dout[inside].double()
    ref = torch.zeros(len(rows), width, device="cuda", dtype=torch.float64).index_add_(0, at, d) * 0.5
    mag = torch.zeros(len(rows), width, device="cuda", dtype=torch.float64).index_add_(0, at, d.abs()) * 0.5
    bound = (m[:, None] + 2) * U * mag
    if accumulate:
        ref, bound = ref + 0.75, bound + U * (mag + 0.75)
    got = out[rows]
    if dtype == "bf16":
        bound = bound + torch.from_numpy(bf16_half_ulp((ref.abs() + bound).cpu().numpy())).cuda()
    assert bool(((got.double() - ref).abs() <= bound).all())
    out[rows] = start[0, 0] if accumulate else 0  # every other row: as it was, or zero
    assert torch.equal(out, start if accumulate else torch.zeros_like(start))
