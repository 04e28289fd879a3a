"""Cases and plain forms of the operators at the two ends of a model, where the
vocabulary is: both work on a matrix of one row for each token of it.

* embed: rows of the embedding table looked up by token and scaled; its
  gradient sums the rows of the output's gradient by token, into a whole new
  matrix or onto one that holds earlier microbatches' sums.
* loss: softmax cross entropy of hidden states under the output head, without
  keeping the logits; with "grad" also the gradients of the hidden states and
  of the head, as one training step needs them.

The plain forms are elementary torch operations in float32.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORED = -100


def listed():
    return [
        # latency: the token a generation loop has just made
        {"name": "lookup 1 token", "op": "lookup", "rows": 128256, "cols": 4096, "tokens": 1,
         "table": "bf16", "y": "bf16", "scale": 1.0},
        # a training batch, or a long prompt
        {"name": "lookup 8192 tokens", "op": "lookup", "rows": 128256, "cols": 4096, "tokens": 8192,
         "table": "bf16", "y": "bf16", "scale": 1.0},
        # odd sizes: rows of a float32 table that start at any 4 bytes, scaled, to BF16
        {"name": "lookup odd sizes", "op": "lookup", "rows": 32003, "cols": 1001, "tokens": 5003,
         "table": "f32", "y": "bf16", "scale": 31.64},
        # latency: a small table's gradient
        {"name": "table gradient 300 tokens", "op": "scatter", "rows": 1999, "cols": 513, "tokens": 300,
         "dy": "f32", "dw": "f32", "scale": 1.0, "padding": False, "add": False},
        # a training batch's gradient of the whole table, as the optimiser takes it
        {"name": "table gradient 8192 tokens", "op": "scatter", "rows": 128256, "cols": 4096,
         "tokens": 8192, "dy": "bf16", "dw": "bf16", "scale": 1.0, "padding": False, "add": False},
        # long sequences of a large model, padded, added to earlier microbatches' sums
        {"name": "table gradient added 32768 tokens", "op": "scatter", "rows": 128256, "cols": 8192,
         "tokens": 32768, "dy": "bf16", "dw": "f32", "scale": 1.0, "padding": True, "add": True},
        # latency: one token scored under a small head
        {"name": "loss 1 token small", "op": "loss", "rows": 1999, "cols": 256, "tokens": 1,
         "grad": False, "dx": "bf16", "dw": "bf16", "add": False},
        # a draft's tokens scored: bound by reading the head
        {"name": "loss 16 tokens", "op": "loss", "rows": 128256, "cols": 4096, "tokens": 16,
         "grad": False, "dx": "bf16", "dw": "bf16", "add": False},
        # an evaluation text scored
        {"name": "loss 2048 tokens", "op": "loss", "rows": 128256, "cols": 4096, "tokens": 2048,
         "grad": False, "dx": "bf16", "dw": "bf16", "add": False},
        # a short microbatch's step
        {"name": "loss and gradient 512 tokens", "op": "loss", "rows": 128256, "cols": 4096,
         "tokens": 512, "grad": True, "dx": "bf16", "dw": "bf16", "add": False},
        # odd sizes, the head's gradient in float32 and added to earlier microbatches' sums
        {"name": "loss and gradient odd sizes", "op": "loss", "rows": 32003, "cols": 1000,
         "tokens": 1001, "grad": True, "dx": "bf16", "dw": "f32", "add": True},
        # a training batch, the largest
        {"name": "loss and gradient 8192 tokens", "op": "loss", "rows": 128256, "cols": 4096,
         "tokens": 8192, "grad": True, "dx": "bf16", "dw": "bf16", "add": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "scatter", "loss", "loss"])
    if op == "loss":
        while True:
            rows, tokens, cols = _log(rng, 16, 131072), _log(rng, 1, 8192), 8 * _log(rng, 1, 1024)
            if rows * tokens * cols <= 2 ** 41 and rows * cols <= 2 ** 30:
                break
        dw = rng.choice(["bf16", "bf16", "f32"])
        grad = rng.random() < 0.6
        return {"op": op, "rows": rows, "cols": cols, "tokens": tokens, "grad": grad,
                "dx": rng.choice(["bf16", "bf16", "f32"]), "dw": dw,
                "add": grad and dw == "f32" and rng.random() < 0.6}
    while True:
        rows, tokens, cols = _log(rng, 16, 131072), _log(rng, 1, 32768), _log(rng, 16, 8192)
        if rng.random() < 0.5:
            cols = (cols + 7) // 8 * 8
        if rows * cols <= 2 ** 30:
            break
    scale = rng.choice([1.0, math.sqrt(cols)])
    if op == "lookup":
        return {"op": op, "rows": rows, "cols": cols, "tokens": tokens,
                "table": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "y": rng.choice(["bf16", "bf16", "f16", "f32"]), "scale": scale}
    dw = rng.choice(["bf16", "f32"])
    return {"op": op, "rows": rows, "cols": cols, "tokens": tokens, "dy": rng.choice(["bf16", "f32"]),
            "dw": dw, "scale": scale, "padding": rng.random() < 0.5, "add": dw == "f32" and rng.random() < 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    rows, cols, n = case["rows"], case["cols"], case["tokens"]
    s = {"case": dict(case)}
    # tokens of a text: the k-th commonest comes with a probability of about
    # 1 / (k ln rows); where it stands in the vocabulary has no order
    common = (uniform(n).double() * math.log(rows)).exp().long().clamp(1, rows) - 1
    tokens = (common * 7919 + int(seed) % rows) % rows
    if case["op"] == "lookup":
        s["w"] = (normal(rows, cols) * 0.02).to(TYPES[case["table"]])
        s["tokens"] = tokens
        return s
    if case["op"] == "scatter":
        s["dy"] = (normal(n, cols) * 1e-3).to(TYPES[case["dy"]])
        s["padding"] = None
        if case["padding"]:  # the last quarter of the batch is padding
            s["padding"] = int(tokens[0])
            tokens = torch.where(torch.arange(n, device="cuda") < n - n // 4, tokens, s["padding"])
        s["tokens"] = tokens
        if case["add"]:
            s["dw"] = normal(rows, cols) * 1e-3
        return s
    w = normal(rows, cols).mul_(torch.exp(normal(rows, 1) * 0.2)).mul_(1 / math.sqrt(cols))
    s["w"] = w.to(torch.bfloat16)
    # hidden states that know the next token more or less well, or not at all
    known = (uniform(n, 1) * 16 - 4).clamp(min=0)
    s["x"] = (normal(n, cols) * 1.5 + known * w[tokens]).to(torch.bfloat16)
    # some tokens are not counted (prompts, padding)
    s["targets"] = torch.where(uniform(n) < 0.05, IGNORED, tokens) if n > 1 else tokens
    s["each"] = 1.0 / n
    if case["add"]:
        s["dw"] = normal(rows, cols) * (0.1 / n)
    return s


def _lookup(s):
    case = s["case"]
    if own:
        import entropy_decoding_amd as ed

        if "embedding" not in s:
            s["embedding"] = ed.Embedding(s["w"], scale=case["scale"])
        return s["embedding"](s["tokens"], TYPES[case["y"]])
    return (s["w"][s["tokens"]].float() * case["scale"]).to(TYPES[case["y"]])


def _scatter(s):
    case = s["case"]
    if own:
        import entropy_decoding_amd as ed

        return ed.embedding_gradient(s["tokens"], s["dy"], case["rows"], dtype=TYPES[case["dw"]],
                                     out=s["dw"] if case["add"] else None, accumulate=case["add"],
                                     scale=case["scale"], padding_idx=s["padding"])
    dy = s["dy"].float() * case["scale"]
    if s["padding"] is not None:
        dy = torch.where((s["tokens"] != s["padding"])[:, None], dy, 0.0)
    sums = torch.zeros(case["rows"], case["cols"], device="cuda").index_add_(0, s["tokens"], dy)
    if case["add"]:
        return s["dw"].add_(sums)
    return sums.to(TYPES[case["dw"]])


def _loss(s):
    case = s["case"]
    if own:
        import entropy_decoding_amd as ed

        if "head" not in s:
            s["head"] = ed.VocabLoss([s["w"]])
        losses, lse = s["head"](s["x"], s["targets"])
        if not case["grad"]:
            return {"loss": losses, "lse": lse}
        dx, (dw,) = s["head"].gradient(s["x"], s["targets"], lse, s["each"], dx_dtype=TYPES[case["dx"]],
                                       dw_dtype=TYPES[case["dw"]], accumulate=case["add"],
                                       dws=[s["dw"]] if case["add"] else None, losses=losses)
        return {"loss": losses, "lse": lse, "dx": dx, "dw": dw}
    x, w = s["x"].float(), s["w"].float()
    logits = x @ w.T
    counted = s["targets"] != IGNORED
    at = torch.where(counted, s["targets"], 0)[:, None]
    top = logits.amax(1, keepdim=True)
    told = logits.gather(1, at)[:, 0]
    p = logits.sub_(top).exp_()
    total = p.sum(1)
    lse = total.log() + top[:, 0]
    out = {"loss": torch.where(counted, lse - told, 0.0), "lse": lse}
    if case["grad"]:
        each = counted.float() * s["each"]
        g = p.mul_((each / total)[:, None]).scatter_add_(1, at, -each[:, None])
        out["dx"] = (g @ w).to(TYPES[case["dx"]])
        dw = g.T @ x
        out["dw"] = s["dw"].add_(dw) if case["add"] else dw.to(TYPES[case["dw"]])
    return out


def run(state):
    return {"lookup": _lookup, "scatter": _scatter, "loss": _loss}[state["case"]["op"]](state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        return torch.index_select(s["w"].double(), 0, s["tokens"]) * case["scale"]
    if case["op"] == "scatter":
        # sums of a sorted list are differences of its running sums, by columns
        dy = s["dy"]
        order = s["tokens"].argsort()
        found, count = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        last = count.cumsum(0) - 1
        out = torch.zeros(case["rows"], case["cols"], dtype=torch.float64, device="cuda")
        for c in range(0, case["cols"], 512):
            running = dy[:, c:c + 512].double()[order].cumsum(0)[last]
            running[1:] -= running[:-1].clone()
            out[found, c:c + 512] = running * case["scale"]
        if s["padding"] is not None:
            out[s["padding"]] = 0
        return out + s["dw"].double() if case["add"] else out
    x, w = s["x"].double(), s["w"].double()
    out = {"loss": [], "lse": []}
    dx, dw = [], s["dw"].double() if case["add"] else torch.zeros_like(w)
    for first in range(0, case["tokens"], 2048):
        part = x[first:first + 2048]
        targets = s["targets"][first:first + 2048]
        logits = torch.matmul(part, w.t())
        lse = torch.logsumexp(logits, dim=1)
        counted = (targets >= 0).double()
        at = torch.arange(len(targets), device="cuda"), targets.clamp(min=0)
        out["loss"].append(counted * (lse - logits[at]))
        out["lse"].append(lse)
        if case["grad"]:
            g = torch.exp(logits - lse.view(-1, 1))
            g[at] -= 1
            g *= (counted * s["each"]).view(-1, 1)
            dx.append(torch.matmul(g, w))
            dw += torch.matmul(g.t(), part)
    out = {k: torch.cat(v) for k, v in out.items()}
    if case["grad"]:
        out["dx"], out["dw"] = torch.cat(dx), dw
    return out


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    rows, cols, n = case["rows"], case["cols"], case["tokens"]
    if case.get("padding"):
        n -= n // 4
    # rows that tokens of prepare()'s distribution meet
    met = sum(1 - (1 - math.log1p(1 / k) / math.log(rows)) ** n for k in range(1, rows + 1))
    if case["op"] == "lookup":
        return {"bytes": 8 * n + met * cols * size[case["table"]] + n * cols * size[case["y"]],
                "flops": n * cols}
    if case["op"] == "scatter":
        nbytes = 8 * case["tokens"] + n * cols * size[case["dy"]]
        nbytes += 8 * met * cols if case["add"] else rows * cols * size[case["dw"]]
        return {"bytes": nbytes, "flops": n * cols}
    nbytes = (rows + n) * cols * 2 + 16 * n
    if case["grad"]:
        nbytes += n * cols * size[case["dx"]] + rows * cols * (8 if case["add"] else size[case["dw"]])
    return {"bytes": nbytes, "flops": (6 if case["grad"] else 2) * n * rows * cols}
