"""The operators over a language model's vocabulary matrices, as cases that can be timed and compared.

Four operators: the embedding lookup with a scale, the gradient of its table, the softmax cross
entropy of a linear output head (per-token losses, the logits never stored), and that loss with
the gradients of the hidden states and of the head's weight.  `own` chooses between the plain form
(elementary torch operations in 32 bits, rounded once at the end) and this package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
IGNORED = -100


def listed():
    """Twelve cases; tokens = rows looked up or scored, vocab x width = the vocabulary matrix."""
    return [
        # decoding: the one new token of a sequence is looked up; latency alone counts
        {"name": "lookup-1-bf16", "op": "lookup", "tokens": 1, "vocab": 32000, "width": 2048, "dtype": "bf16"},
        # a small fp32 model whose rows are no multiple of any vector: unaligned rows
        {"name": "lookup-odd-f32", "op": "lookup", "tokens": 4097, "vocab": 1009, "width": 1001, "dtype": "f32"},
        # a whole batch of a large model: a stream of rows through HBM
        {"name": "lookup-large-bf16", "op": "lookup", "tokens": 65536, "vocab": 131072, "width": 4096, "dtype": "bf16"},
        # one short sequence of a small fp32 model, odd in every size
        {"name": "table-odd-f32", "op": "table", "tokens": 257, "vocab": 4001, "width": 255, "dtype": "f32",
         "accumulate": False},
        # sixteen sequences of 1024 tokens of the 2048-wide model: few rows of the table are met, all are written
        {"name": "table-bf16", "op": "table", "tokens": 16384, "vocab": 32000, "width": 2048, "dtype": "bf16",
         "accumulate": False},
        # a large batch added onto the fp32 gradient that a tied head has left in the same table
        {"name": "table-tied-large", "op": "table", "tokens": 65536, "vocab": 65536, "width": 4096, "dtype": "bf16",
         "accumulate": True},
        # scoring one token: the head's weight is streamed once
        {"name": "loss-1-bf16", "op": "loss", "tokens": 1, "vocab": 32000, "width": 2048, "dtype": "bf16"},
        # evaluating eight sequences of 1024 tokens
        {"name": "loss-bf16", "op": "loss", "tokens": 8192, "vocab": 32000, "width": 2048, "dtype": "bf16"},
        # training a small fp32 model on one odd sequence
        {"name": "train-odd-f32", "op": "train", "tokens": 257, "vocab": 1013, "width": 255, "dtype": "f32"},
        # training with fp32 weights: four sequences of 1024 tokens of a 1024-wide model
        {"name": "train-f32", "op": "train", "tokens": 4096, "vocab": 32000, "width": 1024, "dtype": "f32"},
        # training the 2048-wide model in bf16 on eight sequences of 1024 tokens
        {"name": "train-bf16", "op": "train", "tokens": 8192, "vocab": 32000, "width": 2048, "dtype": "bf16"},
        # the largest: a 4096-wide model with a vocabulary of 131072
        {"name": "train-large-bf16", "op": "train", "tokens": 8192, "vocab": 131072, "width": 4096, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: any length, vocabulary and width, round ones as likely as odd ones."""
    op = rng.choice(["lookup", "table", "loss", "train"])
    case = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    most = 8192 if op in ("loss", "train") else 65536
    while True:
        tokens, vocab, width = _spread(rng, 1, most), _spread(rng, 200, 131072), _spread(rng, 64, 4096)
        if rng.random() < 0.5:   # half of the models are built of round sizes
            width = (width + 63) // 64 * 64
            vocab = (vocab + 63) // 64 * 64
        # no dearer than the largest listed case, and fp32 logits of a plain form that fit beside their gradients
        if vocab * width <= 65536 * 4096 and (op in ("lookup", "table") or tokens * vocab <= 4096 * 131072):
            break
    case.update(tokens=tokens, vocab=vocab, width=width)
    if op == "table":
        case["accumulate"] = rng.random() < 0.5
    return case


def _tokens(gen, count, vocab):
    """Token ids with the skew of text: id k about 1 / (k + 1) as frequent as id 0."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, v, d, dt = case["tokens"], case["vocab"], case["width"], DTYPES[case["dtype"]]
    s = {"case": case, "ids": _tokens(gen, t, v)}
    if case["op"] == "table":
        s["dY"] = torch.empty(t, d, device="cuda").normal_(0, 1e-3, generator=gen).to(dt)
        s["scale"] = math.sqrt(d)
        s["pad"] = 1   # rows of the padding token leave no gradient
        # the gradient's buffer: what a tied head has left in it where it is added to, fp32 then
        gt = torch.float32 if case["accumulate"] else dt
        s["dW"] = torch.empty(v, d, device="cuda", dtype=gt).normal_(0, 1e-3, generator=gen)
        return s
    s["W"] = torch.empty(v, d, device="cuda").normal_(0, d ** -0.5, generator=gen).to(dt)   # 0.022 at 2048
    if case["op"] == "lookup":
        s["scale"] = math.sqrt(d)
        return s
    # normalised hidden states that lean towards their targets' rows as a trained model's do: the
    # target's logit is up to 0.8 log(vocab) above the others, so losses run from about log(vocab) down to
    # a target that has much of the probability
    lean = torch.rand(t, 1, generator=gen, device="cuda") * (0.8 * math.log(v))
    h = torch.randn(t, d, generator=gen, device="cuda")
    s["H"] = (h + lean * s["W"][s["ids"]].float()).to(dt)
    # a few rows in a hundred are padding and count for nothing
    s["targets"] = torch.where(torch.rand(t, generator=gen, device="cuda") < 0.05, IGNORED, s["ids"])
    if t == 1:
        s["targets"] = s["ids"]
    # the mean over the rows that count
    s["grad"] = 1.0 / (s["targets"] != IGNORED).sum().clamp(min=1).float().reshape(1)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


def _plain(s):
    case = s["case"]
    if case["op"] == "lookup":
        return (s["W"][s["ids"]].float() * s["scale"]).to(s["W"].dtype)
    if case["op"] == "table":
        rows = s["dY"].float() * s["scale"]
        rows *= (s["ids"] != s["pad"])[:, None]
        dW = s["dW"]
        if case["accumulate"]:
            return dW.index_add_(0, s["ids"], rows)
        total = torch.zeros(dW.shape, device=dW.device).index_add_(0, s["ids"], rows)
        return dW.copy_(total)
    H, W, counts = s["H"].float(), s["W"].float(), s["targets"] != IGNORED
    rows, picked = torch.arange(H.shape[0], device=H.device), s["targets"].clamp(min=0)
    z = H @ W.t()
    top = z.amax(1)
    target = z[rows, picked]
    z -= top[:, None]
    z.exp_()
    total = z.sum(1)
    loss = torch.where(counts, total.log() + top - target, 0.0)
    if case["op"] == "loss":
        return loss
    z /= total[:, None]
    z[rows, picked] -= 1
    z *= (counts * s["grad"])[:, None]
    return {"loss": loss, "dH": (z @ W).to(s["H"].dtype), "dW": (z.t() @ H).to(s["W"].dtype)}


def _own(s):
    import rank_orthonormalized_optimizer_amd as dion
    case = s["case"]
    if case["op"] == "lookup":
        return dion.embedding_(s["ids"], s["W"], s["scale"])
    if case["op"] == "table":
        return dion.embedding_grad_(s["ids"], s["dY"], s["dW"], s["scale"], padding_id=s["pad"],
                                    accumulate=case["accumulate"])
    loss, lse = dion.linear_cross_entropy_(s["H"], s["W"], s["targets"], ignore_index=IGNORED)
    if case["op"] == "loss":
        return loss
    dH, dW = torch.empty_like(s["H"]), torch.empty_like(s["W"])
    dion.linear_cross_entropy_grad_(s["H"], s["W"], s["targets"], lse, s["grad"], dH, dW, ignore_index=IGNORED)
    return {"loss": loss, "dH": dH, "dW": dW}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    t, v, d, b = case["tokens"], case["vocab"], case["width"], BYTES[case["dtype"]]
    if case["op"] == "lookup":   # a row is read and written for each token
        return {"bytes": 2.0 * t * d * b + 8 * t, "flops": 1.0 * t * d}
    if case["op"] == "table":    # the tokens' rows are read; the table is written, or its met rows read and written
        met = min(t, v)          # at most
        table = 2.0 * met * d * 4 if case["accumulate"] else 1.0 * v * d * b
        return {"bytes": 1.0 * t * d * b + table + 8 * t, "flops": 2.0 * t * d}
    product = 2.0 * t * v * d
    if case["op"] == "loss":     # one product over the vocabulary
        return {"bytes": 1.0 * (t + v) * d * b + 12 * t, "flops": product + 3.0 * t * v}
    # the logits and the two gradients' products
    return {"bytes": 2.0 * (t + v) * d * b + 12 * t, "flops": 3 * product + 6.0 * t * v}


def exact(case, seed):
    """The operators' definitions in 64 bits, the vocabulary taken in blocks with a running maximum and sum."""
    s = _inputs(case, seed)
    v, f64 = case["vocab"], torch.float64
    if case["op"] == "lookup":
        return torch.index_select(s["W"], 0, s["ids"]).to(f64).mul_(s["scale"])
    if case["op"] == "table":
        keep = torch.nonzero(s["ids"] != s["pad"])[:, 0]
        order = keep[torch.argsort(s["ids"][keep], stable=True)]
        ids = s["ids"][order]
        out = s["dW"].to(f64) if case["accumulate"] else torch.zeros(s["dW"].shape, dtype=f64, device="cuda")
        block = max(1, (1 << 26) // case["width"])
        for a in range(0, ids.numel(), block):
            rows = s["dY"][order[a:a + block]].to(f64) * s["scale"]
            out.index_put_((ids[a:a + block],), rows, accumulate=True)
        return out
    H, y = s["H"].to(f64), s["targets"]
    n, block = H.shape[0], max(1, min(v, (1 << 28) // max(1, H.shape[0])))
    top = torch.full((n,), -math.inf, dtype=f64, device="cuda")
    total, at_target = torch.zeros_like(top), torch.zeros_like(top)
    starts = range(0, v, block)
    for a in starts:
        z = torch.mm(H, s["W"][a:a + block].to(f64).t())
        new = torch.maximum(top, z.amax(1))
        total = total * torch.exp(top - new) + torch.exp(z - new[:, None]).sum(1)
        top = new
        inside = torch.nonzero((y >= a) & (y < a + z.shape[1]))[:, 0]
        at_target[inside] = z[inside, y[inside] - a]
    lse = top + torch.log(total)
    counts = (y >= 0).to(f64)
    loss = (lse - at_target) * counts
    if case["op"] == "loss":
        return loss
    share = counts * s["grad"].to(f64)
    dH = torch.zeros_like(H)
    dW = torch.empty(v, H.shape[1], dtype=f64, device="cuda")
    for a in starts:
        w = s["W"][a:a + block].to(f64)
        p = torch.exp(torch.mm(H, w.t()) - lse[:, None])
        inside = torch.nonzero((y >= a) & (y < a + p.shape[1]))[:, 0]
        p[inside, y[inside] - a] -= 1
        p *= share[:, None]
        dH += torch.mm(p, w)
        dW[a:a + block] = torch.mm(p.t(), H)
    return {"loss": loss, "dH": dH, "dW": dW}
