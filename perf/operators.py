"""The operators at the two ends of a sparse language model, and the cases they are measured on.

embed       rows of a table looked up by token, times a scale; an id outside the table gives a row of zeros
embed_grad  the table's gradient: for every id the sum of its tokens' rows, times the scale, in the table's type
xent        softmax cross entropy of a projection to the vocabulary, the mean over the tokens whose target is in it;
            "eval" gives each token's loss, "train" the mean loss and both gradients
clip        the 2-norm over many gradient tensors, and copies scaled so that it is at most max_norm
"""

import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
INDEX = {"i32": torch.int32, "i64": torch.int64}
PAD = -1        # the id of a padding token
IGNORE = -100   # the target of a position that is not trained on


def listed():
    return [
        # eight sequences of a server take their next token's row: a launch and 32 KB
        dict(name="embed_next_token", op="embed", tokens=8, vocab=32768, width=1024, type="f32", index="i64", gap=0),
        # a long training batch's lookup
        dict(name="embed_batch", op="embed", tokens=32768, vocab=131072, width=4096, type="bf16", index="i64", gap=0),
        # the backward pass of a small model's embedding; the rows lie in a wider buffer
        dict(name="embed_grad_small", op="embed_grad", tokens=1023, vocab=16384, width=768, type="f32", index="i32", gap=5),
        # the same of a large vocabulary and a long batch: most of the table's rows get no token
        dict(name="embed_grad_batch", op="embed_grad", tokens=32768, vocab=131072, width=4096, type="bf16", index="i64", gap=0),
        # scoring a handful of candidate tokens against a vocabulary: W is read once, for 16 rows
        dict(name="xent_eval_few", op="xent", pass_="eval", tokens=16, vocab=32768, width=1024, type="bf16", index="i64", gap=0),
        # perplexity over a stretch of text
        dict(name="xent_eval_text", op="xent", pass_="eval", tokens=2048, vocab=65536, width=4096, type="bf16", index="i64", gap=0),
        # a training step's head in 32 bits, at the 768-wide sparse MLP's batch
        dict(name="xent_train_f32", op="xent", pass_="train", tokens=1024, vocab=16384, width=768, type="f32", index="i64", gap=0),
        # odd sizes all round, 16 bits
        dict(name="xent_train_odd", op="xent", pass_="train", tokens=1999, vocab=50001, width=1000, type="bf16", index="i32", gap=3),
        # a training step's head over a large vocabulary: the largest case
        dict(name="xent_train_batch", op="xent", pass_="train", tokens=4096, vocab=131072, width=2048, type="bf16", index="i64", gap=0),
        # the gradients of one sparse MLP (two layers of 23,593 weights and their biases)
        dict(name="clip_mlp", op="clip", tensors=4, elements=51026, type="f32"),
        # a deep sparse model: hundreds of tensors from a bias of a few hundred to a few million weights
        dict(name="clip_deep", op="clip", tensors=288, elements=150_000_001, type="mixed"),
        # a few large dense tables
        dict(name="clip_tables", op="clip", tensors=6, elements=1_000_000_000, type="bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "xent", "xent", "clip"))
    if op == "clip":
        tensors = _log(rng, 1, 400)
        return dict(op=op, tensors=tensors, elements=max(tensors, _log(rng, 1000, 1_000_000_000)), type=rng.choice(("f32", "bf16", "mixed")))
    case = dict(op=op, tokens=_log(rng, 1, 32768), vocab=_log(rng, 1000, 131072), width=_log(rng, 64, 4096), type=rng.choice(("f32", "bf16")),
                index=rng.choice(("i32", "i64")), gap=rng.choice((0, 0, 0, 1, 8)))
    if rng.random() < 0.7:  # a model's width is mostly a multiple of 64; the others stay as drawn, odd ones among them
        case["width"] = max(64, case["width"] // 64 * 64)
    if op == "xent":
        case["pass_"] = rng.choice(("eval", "train"))
        case["tokens"] = min(case["tokens"], 8192)
        most = 4096 * 131072 * 2048 // (8 if case["type"] == "f32" else 1)
        while case["tokens"] * case["vocab"] * case["width"] > most:
            case["tokens"] = case["tokens"] // 2 + 1
    return case


def _tokens(case, gen, outside, share):
    """Ids whose frequencies fall as 1 / rank, as words' do, the ranks spread over the vocabulary; a share of them outside it."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    ids = (rank * 7919 + 13) % vocab
    gone = torch.rand(n, generator=gen, device="cuda") < share
    gone[:1] = False
    return torch.where(gone, outside, ids).to(INDEX[case["index"]])


def _rows(n, width, gap, type_, gen, std=1.0):
    """[n, width] normal values whose rows lie width + gap elements apart."""
    buf = torch.empty(n, width + gap, device="cuda", dtype=torch.float32)
    buf.normal_(0.0, std, generator=gen)
    return buf.to(TYPES[type_])[:, :width]


def _sizes(case):
    """The tensors' sizes: from a bias to a table, spread evenly over their logarithm and scaled to the sum."""
    n, total = case["tensors"], case["elements"]
    weight = np.exp(np.linspace(0.0, math.log(2000.0), n)) if n > 1 else np.ones(1)
    weight = weight[(np.arange(n) * 7) % n] if n % 7 else weight
    sizes = np.maximum(1, np.floor(weight / weight.sum() * (total - n))).astype(np.int64)
    sizes[int(np.argmax(sizes))] += total - int(sizes.sum())
    return [int(s) for s in sizes]


def _is_wide(case, i):
    return case["type"] == "f32" or (case["type"] == "mixed" and i % 2 == 0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case=case)
    if case["op"] == "clip":
        sizes = _sizes(case)
        wide = [_is_wide(case, i) for i in range(len(sizes))]
        # gradients of the layers differ in size: a factor of their own each
        state["grads"] = [torch.empty(s, device="cuda", dtype=torch.float32).normal_(0.0, 1e-3 * (1 + i % 5), generator=gen).to(TYPES["f32" if f else "bf16"])
                          for i, (s, f) in enumerate(zip(sizes, wide))]
        # what the optimizer reads: one flat buffer for each type, a view for each tensor
        flat, views = {}, [None] * len(sizes)
        for f in (True, False):
            at = [i for i in range(len(sizes)) if wide[i] == f]
            if at:
                flat[f] = torch.zeros(sum(sizes[i] for i in at), device="cuda", dtype=TYPES["f32" if f else "bf16"])
                for i, v in zip(at, flat[f].split([sizes[i] for i in at])):
                    views[i] = v
        state.update(flat=[flat[f] for f in (True, False) if f in flat], out=views, wide=wide, max_norm=1.0)
        return state
    n, vocab, width = case["tokens"], case["vocab"], case["width"]
    state["scale"] = math.sqrt(width)
    if case["op"] == "embed":
        state["ids"] = _tokens(case, gen, PAD, 0.03)
        state["table"] = _rows(vocab, width, case["gap"], case["type"], gen, 0.02)
    elif case["op"] == "embed_grad":
        state["ids"] = _tokens(case, gen, PAD, 0.03)
        state["dout"] = _rows(n, width, case["gap"], case["type"], gen, 1e-2)
    else:
        targets = _tokens(case, gen, IGNORE, 0.05)
        w = _rows(vocab, width, 0, case["type"], gen, 1.0 / math.sqrt(width))
        x = torch.empty(n, width + case["gap"], device="cuda", dtype=torch.float32).normal_(generator=gen)
        x[:, :width] += 9.0 * w[targets.long().clamp(0, vocab - 1)].float()  # a model that has learnt something
        state.update(targets=targets, w=w, x=x.to(TYPES[case["type"]])[:, :width])
    return state


def _plain_embed(s):
    ids = s["ids"].long()
    inside = (ids >= 0) & (ids < s["case"]["vocab"])
    rows = s["table"][torch.where(inside, ids, 0)].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s):
    c, ids = s["case"], s["ids"].long()
    inside = (ids >= 0) & (ids < c["vocab"])
    rows = torch.where(inside[:, None], s["dout"].float(), 0.0)
    grad = torch.zeros(c["vocab"], c["width"], device="cuda").index_add_(0, torch.where(inside, ids, 0), rows)
    return (grad * s["scale"]).to(s["dout"].dtype)


def _plain_xent(s):
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"].long()
    inside = (targets >= 0) & (targets < w.shape[0])
    at = torch.where(inside, targets, 0)[:, None]
    z = x @ w.T
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    loss = torch.where(inside, (torch.log(total) + top - picked)[:, 0], 0.0)
    if s["case"]["pass_"] == "eval":
        return loss
    weight = torch.where(inside, 1.0 / inside.sum().clamp(min=1).float(), 0.0)[:, None]
    dz = (e / total * weight).scatter_add(1, at, -weight)
    return (loss * weight[:, 0]).sum(), (dz @ w).to(s["x"].dtype), (dz.T @ x).to(s["w"].dtype)


def _plain_clip(s):
    norm = torch.cat([g.float() for g in s["grads"]]).square().sum().sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    parts = [torch.cat([g.float() for g, f in zip(s["grads"], s["wide"]) if f == kind]) * scale for kind in (True, False) if kind in s["wide"]]
    return [norm] + [p.to(o.dtype) for p, o in zip(parts, s["flat"])]


def run(state):
    op, case = state["case"]["op"], state["case"]
    if not own:
        return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "xent": _plain_xent, "clip": _plain_clip}[op](state)
    from spmm_row_sorted_gb300 import snack

    if op == "embed":
        return snack.embed(state["ids"], state["table"], state["scale"])
    if op == "embed_grad":
        return snack.embed_grad(state["ids"], state["dout"], case["vocab"], state["scale"])
    if op == "clip":
        return [snack.clip_grad_norm(state["grads"], state["max_norm"], out=state["out"])] + state["flat"]
    if case["pass_"] == "eval":
        return snack.xent(state["x"], state["w"], state["targets"], reduction="none")[0]
    loss, kept = snack.xent(state["x"], state["w"], state["targets"], reduction="mean")
    return (loss,) + snack.xent_grad(state["x"], state["w"], state["targets"], kept, reduction="mean")


def _distinct(case):
    """How many different rows a batch of tokens touches, on average."""
    rank = np.arange(1, case["vocab"] + 1, dtype=np.float64)
    p = np.log1p(1.0 / rank) / math.log(case["vocab"] + 1)
    return float((1.0 - (1.0 - p) ** case["tokens"]).sum())


def work(case):
    if case["op"] == "clip":
        sizes = _sizes(case)
        moved = sum(s * (4 if _is_wide(case, i) else 2) for i, s in enumerate(sizes))
        return {"bytes": 2 * moved, "flops": 3 * case["elements"]}
    n, vocab, width = case["tokens"], case["vocab"], case["width"]
    size, ids = (4 if case["type"] == "f32" else 2), n * (4 if case["index"] == "i32" else 8)
    if case["op"] == "embed":
        return {"bytes": int((n + _distinct(case)) * width * size) + ids, "flops": n * width}
    if case["op"] == "embed_grad":
        return {"bytes": (n + vocab) * width * size + ids, "flops": n * width}
    if case["pass_"] == "eval":
        return {"bytes": (n + vocab) * width * size + ids + 4 * n, "flops": 2 * n * vocab * width}
    return {"bytes": 2 * (n + vocab) * width * size + ids, "flops": 6 * n * vocab * width}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        flat = []
        for o in s["flat"]:
            whole, at = torch.empty(o.numel(), device="cuda", dtype=torch.float64), 0
            for g in s["grads"]:
                if g.dtype == o.dtype:
                    whole[at:at + g.numel()] = g.double() * scale
                    at += g.numel()
            flat.append(whole)
        return [torch.tensor(norm, dtype=torch.float64)] + flat
    n, vocab, width = case["tokens"], case["vocab"], case["width"]
    if case["op"] == "embed":
        out = torch.zeros(n, width, device="cuda", dtype=torch.float64)
        real = ((s["ids"] >= 0) & (s["ids"] < vocab)).nonzero()[:, 0]
        out[real] = s["table"].double()[s["ids"][real].long()] * s["scale"]
        return out
    if case["op"] == "embed_grad":
        out = torch.zeros(vocab, width, device="cuda", dtype=torch.float64)
        real = ((s["ids"] >= 0) & (s["ids"] < vocab)).nonzero()[:, 0]
        return out.index_put_((s["ids"][real].long(),), s["dout"][real].double() * s["scale"], accumulate=True)
    if (6 if case["pass_"] == "train" else 2) * n * vocab * width > 1.4e13:
        return None
    x, w = s["x"].double(), s["w"].double()
    real = ((s["targets"] >= 0) & (s["targets"] < vocab)).nonzero()[:, 0]
    t = s["targets"][real].long()
    z = torch.mm(x[real], w.t())
    log_p = torch.log_softmax(z, dim=1)
    loss = torch.zeros(n, device="cuda", dtype=torch.float64)
    loss[real] = -log_p[torch.arange(len(t), device="cuda"), t]
    if case["pass_"] == "eval":
        return loss
    count = max(1, len(t))
    dz = log_p.exp_()
    dz[torch.arange(len(t), device="cuda"), t] -= 1.0
    dz /= count
    dx = torch.zeros(n, width, device="cuda", dtype=torch.float64)
    dx[real] = torch.mm(dz, w)
    return loss.sum() / count, dx, torch.mm(dz.t(), x[real])
