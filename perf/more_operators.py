"""Adapting and scoring a sparse language model: low-rank adapters of many requests beside a shared projection, and the
log probabilities that a projection to the vocabulary gives to tokens.  The operators and the cases they are measured on.

adapt        base[i] + scale[a] B_a (A_a x[i]) for every row i, with the adapter a = which[i] of the row's request; a row
             whose adapter is none of them keeps its base
adapt_train  the same, and the gradients of x (this path's), A and B for an upstream gradient
score        of the logits x w^T: the log probability of each row's token, the entropy of the row's distribution, and the
             ids and log probabilities of its `top` likeliest tokens (of equal ones the lowest id first); a row whose token
             is outside the vocabulary is not scored: zeros, and the id -1
score_train  log probabilities and entropies, and the gradients of x and w for upstream gradients of both
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
INDEX = {"i32": torch.int32, "i64": torch.int64}
NONE = -1      # the adapter of a request without one
IGNORE = -100  # the token of a position that is not scored


def listed():
    return [
        # a server's step for one request: launches, and an adapter of 256 KB
        dict(name="adapt_one_token", op="adapt", tokens=1, requests=1, adapters=8, rank=16, width=4096, out=4096, type="bf16", index="i64", gap=0),
        # a server's step: a token of each of 64 requests, 32 adapters held
        dict(name="adapt_next_tokens", op="adapt", tokens=64, requests=64, adapters=32, rank=16, width=4096, out=4096, type="bf16", index="i64", gap=0),
        # prompts of some requests together
        dict(name="adapt_prompts", op="adapt", tokens=8192, requests=23, adapters=16, rank=32, width=4096, out=4096, type="bf16", index="i64", gap=0),
        # odd sizes all round, 32 bits; the rows lie in wider buffers
        dict(name="adapt_odd", op="adapt", tokens=1999, requests=61, adapters=9, rank=20, width=1001, out=1777, type="f32", index="i32", gap=3),
        # adapters of a small model trained in 32 bits, many tasks in a batch
        dict(name="adapt_train_small", op="adapt_train", tokens=1023, requests=40, adapters=12, rank=8, width=768, out=768, type="f32", index="i32", gap=0),
        # adapters of a wide layer's up projection: a long batch
        dict(name="adapt_train_batch", op="adapt_train", tokens=8192, requests=16, adapters=4, rank=64, width=4096, out=16384, type="bf16", index="i64", gap=0),
        # the next token of eight sequences: the likeliest ones to choose from
        dict(name="score_next_token", op="score", tokens=8, vocab=32768, width=1024, top=20, given=False, type="bf16", index="i64", gap=0),
        # a stretch of text scored, with the alternatives at each place
        dict(name="score_text", op="score", tokens=2048, vocab=65536, width=4096, top=8, given=True, type="bf16", index="i64", gap=0),
        # odd sizes in 32 bits, the log probabilities and entropies alone
        dict(name="score_odd", op="score", tokens=301, vocab=16411, width=771, top=0, given=True, type="f32", index="i32", gap=5),
        # a policy gradient's step of a small model, in 32 bits
        dict(name="score_train_f32", op="score_train", tokens=512, vocab=16384, width=768, top=0, given=True, type="f32", index="i64", gap=0),
        # odd sizes, 16 bits
        dict(name="score_train_odd", op="score_train", tokens=1021, vocab=50001, width=1000, top=0, given=True, type="bf16", index="i32", gap=3),
        # a policy gradient's step over a large vocabulary: the largest case
        dict(name="score_train_batch", op="score_train", tokens=4096, vocab=131072, width=2048, top=0, given=True, type="bf16", index="i64", gap=0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A model's width is mostly a multiple of 64; the others stay as drawn, odd ones among them."""
    w = _log(rng, low, high)
    return max(64, w // 64 * 64) if rng.random() < 0.7 else w


def draw(rng):
    op = rng.choice(("adapt", "adapt_train", "score", "score_train"))
    case = dict(op=op, tokens=_log(rng, 1, 8192), type=rng.choice(("f32", "bf16")), index=rng.choice(("i32", "i64")), gap=rng.choice((0, 0, 0, 1, 8)))
    if op.startswith("adapt"):
        case.update(requests=min(case["tokens"], _log(rng, 1, 256)), adapters=_log(rng, 1, 64), rank=rng.choice((1, 4, 8, 8, 16, 16, 16, 32, 64, 100, 128)),
                    width=_width(rng, 64, 8192), out=_width(rng, 64, 16384))
        while case["adapters"] * case["rank"] * (case["width"] + case["out"]) > 1 << 28:
            case["adapters"] = case["adapters"] // 2 + 1
        return case
    case.update(vocab=_log(rng, 1000, 131072), width=_width(rng, 64, 4096), given=True, top=0)
    if op == "score":
        case.update(top=rng.choice((0, 1, 5, 8, 20)), given=rng.random() < 0.7)
        if not case["given"] and not case["top"]:
            case["top"] = 1
    most = 4096 * 131072 * 2048 // (8 if case["type"] == "f32" else 1)
    while case["tokens"] * case["vocab"] * case["width"] > most:
        case["tokens"] = case["tokens"] // 2 + 1
    return case


def _rows(n, width, gap, type_, gen, std=1.0):
    """[n, width] normal values whose rows lie width + gap elements apart."""
    buf = torch.empty(n, width + gap, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=gen)
    return buf.to(TYPES[type_])[:, :width]


def _requests(case, gen):
    """Each token's adapter: the requests' tokens lie together, a tenth of the requests has no adapter."""
    n, r = case["tokens"], case["requests"]
    owner = torch.randint(0, case["adapters"], (r,), generator=gen, device="cuda")
    owner = torch.where(torch.rand(r, generator=gen, device="cuda") < 0.1, NONE, owner)
    owner[:1] = owner[:1].clamp(min=0)
    cuts = torch.randperm(n - 1, generator=gen, device="cuda")[:r - 1] + 1 if n > 1 else torch.empty(0, dtype=torch.int64, device="cuda")
    first = torch.zeros(n, dtype=torch.int64, device="cuda")
    first[cuts] = 1
    return owner[first.cumsum(0)].to(INDEX[case["index"]])


def _tokens(case, gen):
    """Ids whose frequencies fall as 1 / rank, as words' do, the ranks spread over the vocabulary; a share is not scored."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    ids = (rank * 7919 + 13) % vocab
    gone = torch.rand(n, generator=gen, device="cuda") < 0.05
    gone[:1] = False
    return torch.where(gone, IGNORE, ids).to(INDEX[case["index"]]), ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, width, type_ = case["tokens"], case["width"], case["type"]
    state = dict(case=case)
    if case["op"].startswith("adapt"):
        k, r, out = case["adapters"], case["rank"], case["out"]
        state["which"] = _requests(case, gen)
        state["x"] = _rows(n, width, case["gap"], type_, gen)
        state["base"] = _rows(n, out, case["gap"], type_, gen)
        state["a"] = _rows(k * r, width, 0, type_, gen, 1.0 / math.sqrt(width)).view(k, r, width)
        state["b"] = _rows(k * out, r, 0, type_, gen, 0.5 / math.sqrt(r)).view(k, out, r)
        state["scales"] = 0.5 + torch.rand(k, generator=gen, device="cuda")  # alpha / rank of each
        if case["op"] == "adapt_train":
            state["dy"] = _rows(n, out, case["gap"], type_, gen, 1e-2)
        return state
    state["targets"], likely = _tokens(case, gen)
    w = _rows(case["vocab"], width, 0, type_, gen, 1.0 / math.sqrt(width))
    x = torch.empty(n, width + case["gap"], device="cuda", dtype=torch.float32).normal_(generator=gen)
    x[:, :width] += 9.0 * w[likely].float()  # a model that has learnt something
    state.update(w=w, x=x.to(TYPES[type_])[:, :width])
    if case["op"] == "score_train":
        # advantages, and a bonus for entropy, of the mean over the batch
        state["dlogp"] = torch.empty(n, device="cuda").normal_(0.0, 1.0 / n, generator=gen)
        state["dentropy"] = torch.full((n,), 0.01 / n, device="cuda")
    return state


def _plain_adapt(s):
    x, base, a, b = s["x"].float(), s["base"].float(), s["a"].float(), s["b"].float()
    which, train = s["which"].long(), s["case"]["op"] == "adapt_train"
    y = base.clone()
    if train:
        dy, dx, da, db = s["dy"].float(), torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
    for k in range(len(a)):
        rows = (which == k).nonzero()[:, 0]
        h = x[rows] @ a[k].T
        y[rows] += s["scales"][k] * (h @ b[k].T)
        if train:
            g = s["scales"][k] * dy[rows]
            dh = g @ b[k]
            dx[rows] = dh @ a[k]
            da[k] = dh.T @ x[rows]
            db[k] = g.T @ h
    kind = s["x"].dtype
    return [t.to(kind) for t in ((y, dx, da, db) if train else (y,))]


def _best(z, x, w, top):
    """Ids of the largest logits, and what they have over the largest of them.  Where they lie as close as their roundings
    the order needs 64 bits: some more than asked for are ranked again by them."""
    some = z.topk(min(top + 8, z.shape[1]), dim=1).indices.sort(dim=1).values
    exact = torch.cat([(w[i].double() @ r.double()[:, :, None])[:, :, 0] for i, r in zip(some.split(256), x.split(256))])
    order = exact.sort(dim=1, descending=True, stable=True).indices[:, :top]
    value = exact.gather(1, order)
    return some.gather(1, order), (value - value[:, :1]).float()


def _plain_score(s):
    case, x, w = s["case"], s["x"].float(), s["w"].float()
    targets = s["targets"].long() if case["given"] else torch.zeros(len(x), dtype=torch.int64, device="cuda")
    scored = (targets >= 0) & (targets < len(w))
    at = torch.where(scored, targets, 0)[:, None]
    z = x @ w.T
    high = z.amax(1, keepdim=True)
    d = z - high
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = (log_total - (e * d).sum(1, keepdim=True) / total)[:, 0]
    logp = (d.gather(1, at) - log_total)[:, 0]
    out = [torch.where(scored, entropy, 0.0)]
    if case["given"]:
        out = [torch.where(scored, logp, 0.0)] + out
    if case["top"]:
        ids, below = _best(z, s["x"], s["w"], case["top"])
        out += [torch.where(scored[:, None], ids, -1), torch.where(scored[:, None], below - log_total, 0.0)]
    if case["op"] == "score":
        return out
    g, h = (torch.where(scored, s[k], 0.0)[:, None] for k in ("dlogp", "dentropy"))
    dz = -(e / total) * (g + h * (d - log_total + entropy[:, None]))
    dz = dz.scatter_add(1, at, g)
    return out + [(dz @ w).to(s["x"].dtype), (dz.T @ x).to(s["w"].dtype)]


def run(state):
    s, case = state, state["case"]
    if not own:
        return _plain_adapt(s) if case["op"].startswith("adapt") else _plain_score(s)
    from spmm_row_sorted_gb300 import snack

    if case["op"] == "adapt":
        return [snack.adapt(s["x"], s["base"], s["a"], s["b"], s["which"], s["scales"])]
    if case["op"] == "adapt_train":
        y, h = snack.adapt(s["x"], s["base"], s["a"], s["b"], s["which"], s["scales"], keep=True)
        return [y, *snack.adapt_grad(s["x"], s["dy"], s["a"], s["b"], s["which"], h, s["scales"])]
    targets = s["targets"] if case["given"] else None
    logp, entropy, ids, top_logp, kept = snack.score(s["x"], s["w"], targets, top=case["top"])
    out = [t for t in (logp, entropy, ids, top_logp) if t is not None]
    if case["op"] == "score":
        return out
    return out + list(snack.score_grad(s["x"], s["w"], targets, kept, s["dlogp"], s["dentropy"]))


def work(case):
    n, width, size = case["tokens"], case["width"], 4 if case["type"] == "f32" else 2
    ids = n * (4 if case["index"] == "i32" else 8)
    if case["op"].startswith("adapt"):
        k, r, out = case["adapters"], case["rank"], case["out"]
        used = k * (1.0 - (1.0 - 0.9 / k) ** case["requests"])  # adapters that a batch touches, on average
        rows = 0.9 * n if case["requests"] > 1 else n           # rows that have one
        moved = (rows * width + 2 * n * out + used * r * (width + out)) * size + ids
        flops = 2 * rows * r * (width + out)
        if case["op"] == "adapt":
            return {"bytes": int(moved), "flops": int(flops)}
        return {"bytes": int(moved + (rows * out + n * width + k * r * (width + out)) * size), "flops": int(3 * flops)}
    vocab, rows = case["vocab"], 4 * n * (2 if case["given"] else 1) + n * case["top"] * 12
    if case["op"] == "score":
        return {"bytes": (n + vocab) * width * size + (ids if case["given"] else 0) + rows, "flops": 2 * n * vocab * width}
    return {"bytes": 2 * (n + vocab) * width * size + ids + 2 * rows, "flops": 6 * n * vocab * width}


def exact(case, seed):
    s = prepare(case, seed)
    n, width = case["tokens"], case["width"]
    if case["op"].startswith("adapt"):
        k, r, out = case["adapters"], case["rank"], case["out"]
        if 2 * n * r * (width + out) > 2e12:
            return None
        y, x, a, b = (s[q].to(torch.float64) for q in ("base", "x", "a", "b"))
        train = case["op"] == "adapt_train"
        dx, da, db = torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
        which = s["which"].tolist()
        for j in sorted(set(which) - {NONE}):
            rows = torch.tensor([i for i in range(n) if which[i] == j], device="cuda")
            scale = float(s["scales"][j])
            xs = x.index_select(0, rows)
            y[rows] = y[rows] + scale * torch.mm(torch.mm(xs, a[j].t()), b[j].t())
            if train:
                up = s["dy"].index_select(0, rows).to(torch.float64) * scale
                back = torch.mm(up, b[j])
                dx[rows] = torch.mm(back, a[j])
                da[j] = torch.mm(back.t(), xs)
                db[j] = torch.mm(up.t(), torch.mm(xs, a[j].t()))
        return [y, dx, da, db] if train else [y]
    vocab, top = case["vocab"], case["top"]
    if (6 if case["op"] == "score_train" else 2) * n * vocab * width > 1.4e13:
        return None
    x, w = s["x"].double(), s["w"].double()
    entropy, ids = torch.zeros(n, device="cuda", dtype=torch.float64), torch.full((n, top), -1, device="cuda")
    logp, best, dx, dw = entropy.clone(), torch.zeros(n, top, device="cuda", dtype=torch.float64), torch.zeros_like(x), torch.zeros_like(w)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    if case["given"]:
        keep = (s["targets"] >= 0) & (s["targets"] < vocab)
    for rows in keep.nonzero()[:, 0].split(512):
        z = torch.mm(x[rows], w.t())
        log_p = torch.log_softmax(z, dim=1)
        p = log_p.exp()
        entropy[rows] = -(p * log_p).sum(1)
        if case["given"]:
            t = s["targets"][rows].long()
            logp[rows] = log_p[torch.arange(len(rows), device="cuda"), t]
        if top:
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
            ids[rows], best[rows] = order, log_p.gather(1, order)
        if case["op"] == "score_train":
            g, h = s["dlogp"][rows].double()[:, None], s["dentropy"][rows].double()[:, None]
            dz = -p * (g + h * (log_p + entropy[rows][:, None]))
            dz[torch.arange(len(rows), device="cuda"), t] += g[:, 0]
            dx[rows] = torch.mm(dz, w)
            dw += torch.mm(dz.t(), x[rows])
    out = ([logp] if case["given"] else []) + [entropy] + ([ids, best] if top else [])
    return out + ([dx, dw] if case["op"] == "score_train" else [])
