"""The operators of a model's residual blocks, as cases that can be timed and compared.

Five operators: dropout from a counter-based generator whose mask is never stored, the root-mean-square
norm with the residual's addition (and dropout) in front of it and an output in the input's type or in
8 bits with a scale per row, that norm's gradients, the gated feed-forward block, and that block's
training step with all its gradients.  `own` chooses between the plain form (elementary torch operations
in 32 bits, rounded once at the end) and this package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6
SITE = 7   # the number of the layer whose mask it is


def listed():
    """Twelve cases; tokens x width = the activations, hidden = the feed-forward block's inner width, dtype = their
    type (and the weights'), stream = the type of the residual stream, p = the dropout's probability."""
    return [
        # one odd sequence of a small fp32 model: latency counts
        {"name": "dropout-odd-f32", "op": "dropout", "tokens": 257, "width": 255, "dtype": "f32", "p": 0.1, "residual": False},
        # the embeddings' dropout of a whole batch of a large model
        {"name": "dropout-large-bf16", "op": "dropout", "tokens": 65536, "width": 4096, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # decoding: the new token of one sequence, latency alone counts
        {"name": "norm-1-bf16", "op": "norm", "tokens": 1, "width": 2048, "dtype": "bf16", "stream": "bf16", "p": 0.0, "bits": 16},
        # a small fp32 model in training whose rows are no multiple of any vector
        {"name": "norm-odd-f32", "op": "norm", "tokens": 4097, "width": 1001, "dtype": "f32", "stream": "f32", "p": 0.1,
         "bits": 16},
        # sixteen sequences of 1024 tokens of the 2048-wide model, the feed-forward block's input in 8 bits
        {"name": "norm-8bit", "op": "norm", "tokens": 16384, "width": 2048, "dtype": "bf16", "stream": "bf16", "p": 0.1, "bits": 8},
        # the backward pass of the small fp32 model's odd sequence
        {"name": "normgrad-odd-f32", "op": "normgrad", "tokens": 257, "width": 255, "dtype": "f32", "stream": "f32", "p": 0.0},
        # the backward pass of a whole batch of a large model with an fp32 residual stream
        {"name": "normgrad-large", "op": "normgrad", "tokens": 65536, "width": 4096, "dtype": "bf16", "stream": "f32", "p": 0.1},
        # decoding with the 2048-wide model: three matrices are streamed once
        {"name": "ffn-1-bf16", "op": "ffn", "tokens": 1, "width": 2048, "hidden": 5632, "dtype": "bf16", "act": "silu", "bits": 16},
        # evaluating four sequences of 1024 tokens with the 8192-wide model, the input in 8 bits
        {"name": "ffn-large-8bit", "op": "ffn", "tokens": 4096, "width": 8192, "hidden": 28672, "dtype": "bf16", "act": "silu",
         "bits": 8},
        # training the small fp32 model on one odd sequence
        {"name": "train-odd-f32", "op": "train", "tokens": 257, "width": 255, "hidden": 1013, "dtype": "f32", "act": "gelu",
         "bits": 16},
        # training with fp32 weights: four sequences of 1024 tokens of a 1024-wide model
        {"name": "train-f32", "op": "train", "tokens": 4096, "width": 1024, "hidden": 4096, "dtype": "f32", "act": "silu",
         "bits": 16},
        # training the 2048-wide model in bf16 on eight sequences of 1024 tokens
        {"name": "train-bf16", "op": "train", "tokens": 8192, "width": 2048, "hidden": 5632, "dtype": "bf16", "act": "silu",
         "bits": 16},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: any length and width, round ones as likely as odd ones."""
    op = rng.choice(["dropout", "norm", "normgrad", "ffn", "train"])
    case = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    round_sizes = rng.random() < 0.5
    if op in ("ffn", "train"):
        while True:
            tokens, width, hidden = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 64, 28672)
            if round_sizes:
                width, hidden = (width + 63) // 64 * 64, (hidden + 63) // 64 * 64
            # no dearer than the largest listed case of its operator
            most = 4096 * 8192 * 28672 if op == "ffn" else 8192 * 2048 * 5632
            if tokens * width * hidden <= most:
                break
        case.update(tokens=tokens, width=width, hidden=hidden, act=rng.choice(["silu", "gelu"]),
                    bits=8 if case["dtype"] == "bf16" and rng.random() < 0.3 else 16)
        return case
    while True:
        tokens, width = _spread(rng, 1, 65536), _spread(rng, 64, 8192)
        if round_sizes:
            width = (width + 63) // 64 * 64
        if tokens * width <= 65536 * 4096:
            break
    case.update(tokens=tokens, width=width, p=rng.choice([0.1, 0.5]) if op == "dropout" else rng.choice([0.0, 0.1]))
    if op == "dropout":
        case["residual"] = rng.random() < 0.5
    else:
        case["stream"] = rng.choice(["f32", case["dtype"]])
    if op == "norm":
        case["bits"] = rng.choice([8, 16])
    return case


def _normal(gen, shape, std, dtype):
    return torch.empty(shape, device="cuda").normal_(0, std, generator=gen).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, d, dt = case["tokens"], case["width"], DTYPES[case["dtype"]]
    s = {"case": case, "seed": torch.randint(-2 ** 62, 2 ** 62, (1,), generator=gen, device="cuda")}
    if case["op"] == "dropout":
        s["x"] = _normal(gen, (t, d), 1.0, dt)
        s["residual"] = _normal(gen, (t, d), 3.0, dt) if case["residual"] else None
        return s
    if case["op"] in ("norm", "normgrad"):
        st = DTYPES[case["stream"]]
        # a stream that grew over some layers, with the few wide features that trained models have
        wide = 1.0 + 20.0 * (torch.rand(d, generator=gen, device="cuda") < 0.01)
        s["w"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt)
        h = torch.randn(t, d, generator=gen, device="cuda") * (3.0 * wide)
        if case["op"] == "norm":
            s["residual"], s["x"] = h.to(st), _normal(gen, (t, d), 1.0, dt)
            return s
        s["h"] = h.to(st)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dY"] = _normal(gen, (t, d), 1e-3, dt)
        s["dsum"] = _normal(gen, (t, d), 1e-3, st)   # what reaches the stream from the layers above
        return s
    f = case["hidden"]
    x = torch.randn(t, d, generator=gen, device="cuda") * (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda"))
    s["scale"] = None
    if case["bits"] == 8:   # as the norm leaves them: the largest of a row between 224 and 448 times a power of two
        s["scale"] = torch.exp2(torch.ceil(torch.log2(x.abs().amax(1) / 448)))
        s["X"] = (x / s["scale"][:, None]).to(torch.float8_e4m3fn)
    else:
        s["X"] = x.to(dt)
    s["Wg"], s["Wu"] = _normal(gen, (f, d), d ** -0.5, dt), _normal(gen, (f, d), d ** -0.5, dt)
    s["Wd"] = _normal(gen, (d, f), f ** -0.5, dt)
    if case["op"] == "train":
        s["dY"] = _normal(gen, (t, d), 1e-3, dt)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


def _kept(s, count):
    """The mask: the words of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) over the element's number, against p."""
    mask32 = 0xffffffff
    k0, k1 = s["seed"] & mask32, s["seed"] >> 32 & mask32
    i = torch.arange((count + 3) // 4, device="cuda")
    c0, c1, c2, c3 = i & mask32, i >> 32, torch.full_like(i, SITE), torch.zeros_like(i)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & mask32) ^ c1 ^ k0, b & mask32, (a >> 32 & mask32) ^ c3 ^ k1, a & mask32
        k0, k1 = k0 + 0x9E3779B9 & mask32, k1 + 0xBB67AE85 & mask32
    words = torch.stack([c0, c1, c2, c3], 1).reshape(-1)[:count]
    return words >= min(round(s["case"]["p"] * 2 ** 32), mask32)


def _dropped(s, x):
    """x / (1 - p) where the mask keeps it."""
    p = s["case"]["p"]
    return x if p == 0 else torch.where(_kept(s, x.numel()).view(x.shape), x * (1 / (1 - p)), 0.0)


def _act(z, act):
    """The activation and its derivative."""
    if act == "silu":
        r = 1 / (1 + torch.exp(-z))
        return z * r, r * (1 + z * (1 - r))
    c = math.sqrt(2 / math.pi)
    r = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + r), 0.5 * (1 + r) + 0.5 * z * (1 - r * r) * (c * (1 + 3 * 0.044715 * z * z))


def _plain_norm(s):
    case = s["case"]
    real = torch.float64 if case["bits"] == 8 else torch.float32   # values next to a border of the 8-bit numbers
    h = s["residual"].to(real) + _dropped(s, s["x"].to(real))
    rstd = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * s["w"].to(real)
    out = {"h": h.to(s["residual"].dtype), "rstd": rstd.float()}
    if case["bits"] == 16:
        out["y"] = y.to(s["x"].dtype)
        return out
    top = y.abs().amax(1)
    m, e = torch.frexp(top)   # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875)), 1.0)[:, None]
    y /= scale
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))   # e4m3: four significant bits, steps of 2^-9 below 2^-6
    step = torch.ldexp(torch.ones_like(y), e - 4)
    out["y"] = (torch.round(y / step) * step * scale).float()
    out["scale"] = scale[:, 0].float()
    return out


def _plain(s):
    case = s["case"]
    if case["op"] == "dropout":
        y = _dropped(s, s["x"].float())
        return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "normgrad":
        n = s["h"].float() * s["rstd"][:, None]
        dY = s["dY"].float()
        g = dY * s["w"].float()
        dh = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True)) + s["dsum"].float()
        out = {"dh": dh.to(s["h"].dtype), "dw": (dY * n).sum(0).to(s["w"].dtype)}
        if case["p"] > 0:
            out["dx"] = _dropped(s, dh).to(s["dY"].dtype)
        return out
    X = s["X"].float()
    if s["scale"] is not None:
        X = X * s["scale"][:, None]
    Wg, Wu, Wd, dt = s["Wg"].float(), s["Wu"].float(), s["Wd"].float(), s["Wg"].dtype
    a, b = X @ Wg.t(), X @ Wu.t()
    v, slope = _act(a, case["act"])
    u = v * b
    y = (u @ Wd.t()).to(dt)
    if case["op"] == "ffn":
        return y
    dY = s["dY"].float()
    du = dY @ Wd
    da, db = du * b * slope, du * v
    return {"y": y, "dX": (da @ Wg + db @ Wu).to(dt), "dWg": (da.t() @ X).to(dt), "dWu": (db.t() @ X).to(dt),
            "dWd": (dY.t() @ u).to(dt)}


def _own(s):
    import rank_orthonormalized_optimizer_amd as dion
    case = s["case"]
    if case["op"] == "dropout":
        return dion.dropout_(s["x"], case["p"], s["seed"], SITE, residual=s["residual"])
    if case["op"] == "norm":
        if case["bits"] == 16:
            y, h, rstd = dion.rms_norm_(s["x"], s["w"], EPS, residual=s["residual"], p=case["p"], seed=s["seed"], site=SITE)
            return {"h": h, "rstd": rstd, "y": y}
        q, scale, h, rstd = dion.rms_norm_8bit_(s["x"], s["w"], EPS, residual=s["residual"], p=case["p"], seed=s["seed"],
                                                site=SITE)
        return {"h": h, "rstd": rstd, "y": q, "scale": scale}
    if case["op"] == "normgrad":
        dw = torch.empty_like(s["w"])
        dh, dx = dion.rms_norm_grad_(s["dY"], s["h"], s["w"], s["rstd"], dw, dsum=s["dsum"], p=case["p"], seed=s["seed"],
                                     site=SITE)
        out = {"dh": dh, "dw": dw}
        if case["p"] > 0:
            out["dx"] = dx
        return out
    X, scale, act = s["X"], s["scale"], case["act"]
    Wg, Wu, Wd = s["Wg"], s["Wu"], s["Wd"]
    if case["op"] == "ffn":
        return dion.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale)
    gate = torch.empty(X.shape[0], Wg.shape[0], dtype=Wg.dtype, device=Wg.device)
    up = torch.empty_like(gate)
    y = dion.gated_ffn_(X, Wg, Wu, Wd, act=act, scale=scale, gate=gate, up=up)
    dX, dWg, dWu, dWd = torch.empty_like(s["dY"]), torch.empty_like(Wg), torch.empty_like(Wu), torch.empty_like(Wd)
    dion.gated_ffn_grad_(X, Wg, Wu, Wd, s["dY"], gate, up, dX, dWg, dWu, dWd, act=act, scale=scale)
    return {"y": y, "dX": dX, "dWg": dWg, "dWu": dWu, "dWd": dWd}


def run(state):
    out = _own(state) if own else _plain(state)
    if own and state["case"].get("bits") == 8 and state["case"]["op"] == "norm":   # 8 bits as the values they stand for
        out["y"] = out["y"].float() * out["scale"][:, None]
    return out


def work(case):
    t, d, b = case["tokens"], case["width"], BYTES[case["dtype"]]
    n = 1.0 * t * d
    if case["op"] == "dropout":
        return {"bytes": n * b * (3 if case["residual"] else 2), "flops": 2.0 * n}
    if case["op"] == "norm":       # x and the stream in, the stream and the row out
        return {"bytes": n * (b + 2 * BYTES[case["stream"]] + (1 if case["bits"] == 8 else b)), "flops": 6.0 * n}
    if case["op"] == "normgrad":   # dY, the stream and its gradient in, the stream's and the input's gradient out
        return {"bytes": n * (b + 3 * BYTES[case["stream"]] + (b if case["p"] > 0 else 0)), "flops": 12.0 * n}
    f = case["hidden"]
    xb = 1 if case["bits"] == 8 else b
    if case["op"] == "ffn":        # three products
        return {"bytes": n * (xb + b) + 3.0 * d * f * b, "flops": 6.0 * t * d * f + 6.0 * t * f}
    # those and six for the gradients
    return {"bytes": n * (xb + 3 * b) + 6.0 * d * f * b, "flops": 18.0 * t * d * f + 20.0 * t * f}


def _kept64(case, seed, count):
    """The mask again: the generator's 32 x 32 bit products from 16-bit halves."""
    def product(a, m):
        mid = (a & 0xffff) * (m >> 16) + ((a & 0xffff) * (m & 0xffff) >> 16)   # below 2^33
        rest = (a >> 16) * (m & 0xffff) + (mid & 0xffff)
        high = (a >> 16) * (m >> 16) + (mid >> 16) + (rest >> 16)
        return high, (rest & 0xffff) << 16 | (a & 0xffff) * (m & 0xffff) & 0xffff
    key = int(seed.item()) % 2 ** 64
    words = torch.empty((count + 3) // 4, 4, dtype=torch.bool, device="cuda")
    for at in range(0, words.shape[0], 1 << 24):
        rows = torch.arange(at, min(at + (1 << 24), words.shape[0]), device="cuda")
        x = [rows % 2 ** 32, rows // 2 ** 32, torch.full_like(rows, SITE), torch.zeros_like(rows)]
        for r in range(10):
            high0, low0 = product(x[0], 0xD2511F53)
            high2, low2 = product(x[2], 0xCD9E8D57)
            x = [high2 ^ x[1] ^ (key + r * 0x9E3779B9) % 2 ** 32, low2,
                 high0 ^ x[3] ^ ((key >> 32) + r * 0xBB67AE85) % 2 ** 32, low0]
        for j in range(4):
            words[at:at + rows.numel(), j] = x[j] >= min(round(case["p"] * 2 ** 32), 2 ** 32 - 1)
    return words.view(-1)[:count]


def _dropped64(case, s, x):
    if case["p"] == 0:
        return x
    return x * _kept64(case, s["seed"], x.numel()).view(x.shape) / (1 - case["p"])


def exact(case, seed):
    """The operators' definitions in 64 bits, rows in blocks."""
    s, f64 = _inputs(case, seed), torch.float64
    if case["op"] == "dropout":
        y = _dropped64(case, s, s["x"].to(f64))
        return y if s["residual"] is None else y.add_(s["residual"])
    if case["op"] == "norm":
        h = _dropped64(case, s, s["x"].to(f64)).add_(s["residual"])
        rstd = (h.square().sum(1) / case["width"] + EPS).pow(-0.5)
        y = h * torch.outer(rstd, s["w"].to(f64))
        if case["bits"] == 16:
            return {"h": h, "rstd": rstd, "y": y}
        top = y.abs().amax(1)
        step = torch.ceil(torch.log2(top / 448))
        step += (top > 448 * torch.exp2(step)).to(f64) - (top <= 448 * torch.exp2(step - 1)).to(f64)
        scale = torch.where(top > 0, torch.exp2(step), 1.0)
        # the nearest number of three bits behind the leading one, or of 2^-9 below 2^-6; ties to even
        v = y / scale[:, None]
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return {"h": h, "rstd": rstd, "y": torch.round(v / unit) * unit * scale[:, None], "scale": scale}
    if case["op"] == "normgrad":
        w, h, t, d = s["w"].to(f64), s["h"], case["tokens"], case["width"]
        dh, dw = torch.empty(t, d, dtype=f64, device="cuda"), torch.zeros(d, dtype=f64, device="cuda")
        for at in range(0, t, 8192):
            rows = slice(at, at + 8192)
            r = s["rstd"][rows].to(f64)[:, None]
            x, dy = h[rows].to(f64), s["dY"][rows].to(f64)
            dw += (dy * x * r).sum(0)
            dot = (dy * w * x).sum(1, keepdim=True)
            dh[rows] = dy * w * r - x * (dot * r ** 3 / d) + s["dsum"][rows].to(f64)
        out = {"dh": dh, "dw": dw}
        if case["p"] > 0:
            out["dx"] = _dropped64(case, s, dh)
        return out
    X = s["X"].to(f64)
    if s["scale"] is not None:
        X *= s["scale"].to(f64)[:, None]
    Wg, Wu, Wd = (s[k].to(f64) for k in ("Wg", "Wu", "Wd"))
    out = {k: [] for k in ("y", "dX")}
    total = {}
    for at in range(0, case["tokens"], 4096):
        x = X[at:at + 4096]
        a, b = torch.mm(x, Wg.t()), torch.mm(x, Wu.t())
        if case["act"] == "silu":
            r = torch.sigmoid(a)
            v, slope = a * r, r + a * r * (1 - r)
        else:
            r = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))   # (1 + tanh) / 2
            v = a * r
            slope = r + 2 * a * r * (1 - r) * math.sqrt(2 / math.pi) * (1 + 0.134145 * a ** 2)
        out["y"].append(torch.mm(v * b, Wd.t()))
        if case["op"] == "ffn":
            continue
        dY = s["dY"][at:at + 4096].to(f64)
        du = torch.mm(dY, Wd)
        da, db = du * b * slope, du * v
        out["dX"].append(torch.mm(da, Wg) + torch.mm(db, Wu))
        for k, g in (("dWg", torch.mm(da.t(), x)), ("dWu", torch.mm(db.t(), x)), ("dWd", torch.mm(dY.t(), v * b))):
            total[k] = total[k] + g if k in total else g
    y = torch.cat(out["y"])
    return y if case["op"] == "ffn" else {"y": y, "dX": torch.cat(out["dX"]), **total}
