"""Global gradient norm and clipping against the definition in 64 bits.

Tolerances.  The norm: a thread adds at most 128 squares in fp32 (a block's
piece of a tensor is 64 KB, for 256 threads; the tests' sizes give each block
one piece, or a few small ones), and 13 additions join the threads of a block, each
rounding within 2^-24 of the running sum; blocks are joined in fp64.  So the
sum of squares is within 141 * 2^-24 and its root within half of that.  An
output is one product with a factor within 3 roundings and the norm's error of
the exact one, rounded once: that and 2^-22 relative, and half a bf16 ulp in
bf16.
"""

import numpy as np
import pytest
import torch

from spmm_row_sorted_gb300 import snack

from gpu_util import bf16_half_ulp, f64

pytestmark = pytest.mark.gpu

REL = 141 * 2.0 ** -25


def tensors(sizes, types, seed, std=1.0, lead=0):
    """Gradients of the sizes given; with `lead` each starts that many elements off its allocation."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for s, t in zip(sizes, types):
        buf = torch.empty(s + lead, device="cuda").normal_(0, std, generator=g)
        out.append(buf.to(torch.float32 if t == "f" else torch.bfloat16)[lead:])
    return out


def norm_of(grads):
    return float(np.sqrt(sum(float((f64(g) ** 2).sum()) for g in grads)))


def check(grads, outs, norm, got_norm, max_norm):
    assert abs(float(got_norm) - norm) <= REL * norm
    f = min(1.0, max_norm / (norm + 1e-6))
    for g, o in zip(grads, outs):
        ref = f64(g) * f
        bound = (REL + 2.0 ** -22) * np.abs(ref) + 2.0 ** -149
        if g.dtype == torch.bfloat16:
            bound = bound + bf16_half_ulp(np.abs(ref) * (1 + 1e-5))
        assert np.all(np.abs(f64(o) - ref) <= bound)


CASES = [
    # sizes, types, max_norm, lead of the gradients, lead of the outputs
    ([1], "f", 0.5, 0, 0),
    ([1], "b", 100.0, 0, 0),
    ([7, 0, 9], "fbf", 1.0, 0, 0),
    ([23593, 768, 23593, 1024], "ffff", 1.0, 0, 0),
    ([16384, 16385, 32768, 32769, 65537], "fbfbf", 3.0, 0, 0),  # pieces of one tensor end inside and at its end
    ([40000, 40001], "fb", 1.0, 1, 0),                          # gradients off a 16-byte boundary, outputs on it
    ([40000, 40001], "bf", 1.0, 3, 3),
    ([100003, 5, 70001], "bbb", 1e6, 1, 2),                     # not clipped: a copy
    ([300 + 17 * i for i in range(40)], "fb" * 20, 2.0, 0, 1),
    ([37 + i % 50 for i in range(900)], "bff" * 300, 2.0, 0, 0),  # more tensors than one launch's arguments hold
    ([3000001], "f", 1.0, 0, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sizes,types,max_norm,lead,out_lead", CASES, ids=range(len(CASES)))
def test_clip_matches_definition(sizes, types, max_norm, lead, out_lead, in_place):
    grads = tensors(sizes, types, seed=len(sizes), lead=lead)
    norm = norm_of(grads)
    if in_place:
        outs = [g.clone() if lead == 0 else g for g in grads]
        grads = [g.clone() for g in grads]
        got = snack.clip_grad_norm(outs, max_norm)
    else:
        outs = tensors(sizes, types, seed=99, lead=out_lead)
        got = snack.clip_grad_norm(grads, max_norm, out=outs)
    check(grads, outs, norm, got, max_norm)


@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e-12, 1e18, 1e25])
def test_clip_norm_holds_where_squares_leave_fp32(std):
    grads = tensors([50000, 123], "ff", seed=4, std=std)
    outs = [torch.empty_like(g) for g in grads]
    got = snack.clip_grad_norm(grads, 1.0, out=outs)
    check(grads, outs, norm_of(grads), got, 1.0)


def test_clip_not_finite():
    a, b = tensors([1000, 500], "fb", seed=1)
    a[17] = float("inf")
    outs = [torch.empty_like(a), torch.empty_like(b)]
    assert float(snack.clip_grad_norm([a, b], 1.0, out=outs)) == float("inf")
    assert torch.isnan(outs[0][17]) and int(torch.isnan(outs[0]).sum()) == 1  # inf * 0
    assert int((outs[0] != 0).sum()) == 1 and not outs[1].any()
    a[17] = float("nan")
    assert torch.isnan(snack.clip_grad_norm([a, b], 1.0, out=outs))
    assert torch.isnan(outs[0]).all() and torch.isnan(outs[1]).all()


def test_clip_zero_gradients_and_unclipped_in_place():
    z = torch.zeros(1000, device="cuda")
    assert float(snack.clip_grad_norm([z], 1.0)) == 0.0 and not z.any()
    (g,) = tensors([5000], "b", seed=2, std=1e-4)
    before = g.clone()
    snack.clip_grad_norm([g], 10.0)
    assert torch.equal(g, before)


def test_clip_repeats_and_runs_on_another_stream():
    grads = tensors([200001, 77], "fb", seed=6)
    outs = [[torch.empty_like(g) for g in grads] for _ in range(2)]
    n0 = snack.clip_grad_norm(grads, 1.0, out=outs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n1 = snack.clip_grad_norm(grads, 1.0, out=outs[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(*outs))


def test_clip_refusals():
    g = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError):
        snack.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        snack.clip_grad_norm([g.half()], 1.0)
    with pytest.raises(ValueError):
        snack.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError):
        snack.clip_grad_norm([g], 1.0, out=[torch.zeros(99, device="cuda")])
    with pytest.raises(ValueError):
        snack.clip_grad_norm([g.view(10, 10).t()], 1.0)
    with pytest.raises(ValueError):
        snack.clip_grad_norm([g.cpu()], 1.0)
    for bad in (-1.0, float("nan")):
        with pytest.raises(snack.SnackError) as e:
            snack.clip_grad_norm([g], bad)
        assert e.value.status == 1
    with pytest.raises(snack.SnackError):  # shifted on itself
        snack.clip_grad_norm([g[:50]], 1.0, out=[g[10:60]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_clip_norm_of_elements_that_are_alike(dtype):
    # every rounding of a running sum of equal terms errs to the same side.  A thread's longest chain: 32 squares
    # of a batch, 4 batches of a piece, 5 pieces of a block (2^26 elements are 4096 at most), 13 additions of threads;
    # the root halves that, and rounds twice (4)
    g = torch.full((2 ** 26,), 0.1, device="cuda", dtype=dtype)
    want = float(g[0]) * 2.0 ** 13
    assert abs(float(snack.clip_grad_norm([g], 1e9)) - want) <= (32 + 4 + 5 + 13 + 4) * 2.0 ** -25 * want


def test_clip_refuses_a_gradient_given_twice():
    buf = torch.ones(200, device="cuda")
    g, h = buf[:100], buf[100:]
    apart = [torch.empty_like(g) for _ in range(2)]
    snack.clip_grad_norm([g, g], 1e9, out=apart)  # twice as a gradient alone is well defined
    assert torch.equal(apart[0], g) and torch.equal(apart[1], g)
    for grads, out in (([g, g], None), ([g, buf[50:150]], None), ([g, h], [h, g]), ([g, h], [apart[0], apart[0]]),
                       ([g, h], [apart[0], g])):
        with pytest.raises(snack.SnackError) as e:
            snack.clip_grad_norm(grads, 1.0, out=out)
        assert e.value.status == 1
    assert bool((buf == 1).all())


def test_tensors_written_in_place_are_seen_by_autograd():
    g = torch.rand(100, device="cuda")
    h = torch.rand(50, device="cuda").bfloat16()
    weight = torch.ones(100, device="cuda", requires_grad=True)
    y = (weight * g).sum()  # keeps g for its gradient
    before = g._version, h._version
    snack.clip_grad_norm([g, h], 1.0)
    assert g._version > before[0] and h._version > before[1]
    with pytest.raises(RuntimeError):
        y.backward()
    out = [torch.empty_like(g), torch.empty_like(h)]
    marks = g._version, h._version, out[0]._version, out[1]._version
    snack.clip_grad_norm([g, h], 1.0, out=out)  # the gradients are read only
    assert (g._version, h._version) == marks[:2] and out[0]._version > marks[2] and out[1]._version > marks[3]
    with torch.inference_mode():
        held = torch.rand(10, device="cuda")
        snack.clip_grad_norm([held], 1.0)
    snack.clip_grad_norm([held, g], 1.0)  # no version to keep: as before
