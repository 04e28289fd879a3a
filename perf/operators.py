"""Cases and plain forms of the operators that work on a block's uncompressed weights.

Two groups, both over the list of matrices or tensors of one transformer block:

* int8: activations quantised row by row to 8-bit integers (one scale per
  token) times weights held as 8-bit integers (one scale per output channel),
  many matrices a call; with "fresh" the weights come in BF16 and are
  quantised within the pass, as after an update of them.
* adamw: one AdamW step over many tensors, states in 32 bits or in 8 (codes of
  blocks of 256 elements), optionally with the gradients' global norm and clip
  factor, and with the exponent histogram of the new weights that the entropy
  coder wants.

The plain forms are elementary torch operations in float32, the gradient norm
in float64.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 256            # elements of one tensor that share a scale in 8-bit states
TINY = 2.0 ** -100     # a block whose largest |m| is below this is held as zeros
LR, B1, B2, EPS, MAX_NORM = 1e-3, 0.9, 0.95, 1e-8, 1.0

# "rows x cols / index of the activations": the q, k, v projections read one
# input, gate and up another, o and down each their own
BLOCK_8B = "4096x4096/0,1024x4096/0,1024x4096/0,4096x4096/1,14336x4096/2,14336x4096/2,4096x14336/3"
BLOCK_70B = "8192x8192/0,1024x8192/0,1024x8192/0,8192x8192/1,28672x8192/2,28672x8192/2,8192x28672/3"
BLOCK_70B_TP8 = "1024x8192,128x8192,128x8192,8192x1024,3584x8192,3584x8192,8192x3584"


def listed():
    b8 = ",".join(m.split("/")[0] for m in BLOCK_8B.split(","))
    return [
        # latency: one small matrix, one token of a generation loop
        {"name": "int8 1024x1024 1 token", "op": "int8", "mats": "1024x1024/0", "tokens": 1,
         "x": "bf16", "y": "f32", "fresh": False},
        # one token through the matrices of a block: bound by reading the weights
        {"name": "int8 8b block 1 token", "op": "int8", "mats": BLOCK_8B, "tokens": 1,
         "x": "bf16", "y": "bf16", "fresh": False},
        # a small batch of generated tokens
        {"name": "int8 8b block 16 tokens", "op": "int8", "mats": BLOCK_8B, "tokens": 16,
         "x": "bf16", "y": "bf16", "fresh": False},
        # ragged: odd rows, columns and tokens, half-precision activations
        {"name": "int8 odd sizes 77 tokens", "op": "int8", "mats": "1999x1001/0,4097x1001/0,1001x4099/1",
         "tokens": 77, "x": "f16", "y": "f16", "fresh": False},
        # a prompt's chunk
        {"name": "int8 8b block 512 tokens", "op": "int8", "mats": BLOCK_8B, "tokens": 512,
         "x": "bf16", "y": "bf16", "fresh": False},
        # the weights of a block requantised and used: the pass after they changed
        {"name": "int8 8b block fresh weights", "op": "int8", "mats": BLOCK_8B, "tokens": 64,
         "x": "f32", "y": "f32", "fresh": True},
        # a long prompt, the largest products
        {"name": "int8 70b block 4096 tokens", "op": "int8", "mats": BLOCK_70B, "tokens": 4096,
         "x": "bf16", "y": "bf16", "fresh": False},
        # latency: norms, biases and small matrices, all in float32
        {"name": "adamw small tensors f32", "op": "adamw", "tensors":
         "1,7,64,255,256,257,1000,1024,4096,4097,333,8192,5,2048,2049,511,512,513,12289,100,31,3,77,1025",
         "w": "f32", "g": "f32", "master": False, "bits": 32, "clip": True, "counts": False},
        # a block in mixed precision: BF16 weights with float32 masters
        {"name": "adamw 8b block master", "op": "adamw", "tensors": b8, "w": "bf16", "g": "bf16",
         "master": True, "bits": 32, "clip": True, "counts": False},
        # the same with states in 8 bits
        {"name": "adamw 8b block 8-bit", "op": "adamw", "tensors": b8, "w": "bf16", "g": "bf16",
         "master": True, "bits": 8, "clip": True, "counts": False},
        # tensors at odd offsets and of odd lengths, BF16 weights alone, 8-bit states
        {"name": "adamw odd sizes 8-bit", "op": "adamw", "tensors":
         "4097x1001,333,1999x1001,7,1001x4099,65537,1", "w": "bf16", "g": "f32",
         "master": False, "bits": 8, "clip": False, "counts": True},
        # one GPU's share of a large block, updated and counted for the encoder
        {"name": "adamw 70b share with counts", "op": "adamw", "tensors": BLOCK_70B_TP8, "w": "bf16",
         "g": "bf16", "master": False, "bits": 32, "clip": True, "counts": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            n = rng.randint(1, 7)
            xs = sorted(rng.randint(0, n - 1) for _ in range(n))
            cols = {i: _log(rng, 16, 28672) for i in set(xs)}
            mats = [(_log(rng, 16, 28672), cols[i], i) for i in xs]
            tokens = _log(rng, 1, 4096)
            if sum(r * c for r, c, _ in mats) <= 2 ** 28 and sum(r for r, _, _ in mats) * tokens <= 2 ** 28:
                break
        return {"op": "int8", "mats": ",".join("%dx%d/%d" % m for m in mats), "tokens": tokens,
                "x": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "y": rng.choice(["bf16", "bf16", "f16", "f32"]), "fresh": rng.random() < 0.2}
    n = rng.randint(1, 40)
    total = _log(rng, 2000, 100_000_000)
    parts = [rng.expovariate(1.0) for _ in range(n)]
    sizes = [max(1, int(total * p / sum(parts))) for p in parts]
    w = rng.choice(["bf16", "bf16", "f32"])
    return {"op": "adamw", "tensors": ",".join(map(str, sizes)), "w": w,
            "g": rng.choice(["bf16", "f32"]), "master": w == "bf16" and rng.random() < 0.5,
            "bits": rng.choice([32, 8]), "clip": rng.random() < 0.5,
            "counts": w == "bf16" and rng.random() < 0.5}


def _mats(case):
    got = []
    for m in case["mats"].split(","):
        shape, x = m.split("/")
        r, c = shape.split("x")
        got.append((int(r), int(c), int(x)))
    return got


def _sizes(case):
    return [math.prod(int(d) for d in t.split("x")) for t in case["tensors"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if case["op"] == "int8":
        mats = _mats(case)
        s = {"case": dict(case), "shapes": [(r, c) for r, c, _ in mats], "index": [i for _, _, i in mats]}
        s["x"] = {}
        for _, c, i in mats:
            if i not in s["x"]:
                # activations: unit normal with a few channels far larger
                x = normal(case["tokens"], c) * torch.where(uniform(c) < 0.01, 12.0, 1.0)
                s["x"][i] = x.to(TYPES[case["x"]])
        s["w"], s["w_scale"] = [], []
        for r, c, _ in mats:
            w = (normal(r, c) * torch.exp(normal(r, 1) * 0.3) * 0.02).to(torch.bfloat16)
            if not case["fresh"]:
                q, sc = _quantise(w)
                w = torch.zeros(r, (c + 15) // 16 * 16, dtype=torch.int8, device="cuda")
                w[:, :c] = q.to(torch.int8)
                s["w_scale"].append(sc)
            s["w"].append(w)
        return s
    sizes = _sizes(case)
    n, k = sum(sizes), len(sizes)
    s = {"case": dict(case), "sizes": sizes, "t": 10}
    # the tensors lie one behind the other in flat buffers, at any offset
    w = normal(n) * 0.02
    s["w"] = w.to(TYPES[case["w"]])
    if case["master"]:
        s["master"] = w
    s["g"] = (normal(n) * 1e-3 * (1 + 9 * (uniform(n) < 0.01))).to(TYPES[case["g"]])
    s["decay"] = [0.0 if i % 3 == 1 else 0.1 for i in range(k)]  # norms and biases have none
    s["keep"] = torch.tensor([1 - LR * d for d in s["decay"]], device="cuda")
    at = torch.tensor(sizes, device="cuda")
    s["tensor_of"] = torch.repeat_interleave(torch.arange(k, device="cuda", dtype=torch.int32), at,
                                             output_size=n)
    if case["bits"] == 32:
        s["m"] = normal(n) * 3e-4
        s["v"] = (1e-3 * (0.5 + uniform(n))) ** 2
    else:
        blocks = [-(-c // BLOCK) for c in sizes]
        s["blocks"] = blocks
        first = torch.tensor([0] + list(np.cumsum(blocks)[:-1]), device="cuda")
        start = torch.tensor([0] + list(np.cumsum(sizes)[:-1]), device="cuda")
        of = s["tensor_of"].long()
        # where each element lies when every tensor is padded to whole blocks
        s["at"] = first[of] * BLOCK + torch.arange(n, device="cuda") - start[of]
        s["block_of"] = (s["at"] // BLOCK).int()
        s["m"] = (normal(n) * 45).round().clamp(-127, 127).to(torch.int8)
        s["v"] = (100 + 155 * uniform(n)).round().to(torch.uint8)
        s["m_scale"] = (0.5 + uniform(sum(blocks))) * (1e-3 / 127 ** 2)
        s["v_scale"] = (0.5 + uniform(sum(blocks))) * (2e-3 / 255 ** 2)
    return s


def _quantise(x):
    """Codes (as floats) and scales of the rows of x: round(127 x / max|x|)."""
    x = x.to(torch.float64 if x.dtype == torch.float32 else torch.float32)  # 127 x exact
    top = x.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(x * 127 / top), 0.0)
    return q.float(), (top[:, 0].float() / 127)


def _int8(s):
    if own:
        import entropy_decoding_amd as ed

        out = TYPES[s["case"]["y"]]
        xs = [s["x"][i] for i in s["index"]]
        if s["case"]["fresh"]:
            return ed.Int8Linear.from_tensors(s["w"])(xs, out)
        if "layer" not in s:
            s["layer"] = ed.Int8Linear(s["w"], s["w_scale"], s["shapes"])
        return s["layer"](xs, out)
    acts = {i: _quantise(x) for i, x in s["x"].items()}
    ys = []
    for k, (w, i, (_, c)) in enumerate(zip(s["w"], s["index"], s["shapes"])):
        q, sc = _quantise(w) if s["case"]["fresh"] else (w[:, :c].float(), s["w_scale"][k])
        qx, sx = acts[i]
        # the codes' products and sums are whole numbers below 2^24 on this data
        ys.append(((qx @ q.T) * sx[:, None] * sc).to(TYPES[s["case"]["y"]]))
    return ys


def _adamw_own(s):
    import entropy_decoding_amd as ed

    case = s["case"]
    if "opt" not in s:
        part = lambda t, sizes: list(t.split(sizes))  # noqa: E731
        state = {"m": part(s["m"], s["sizes"]), "v": part(s["v"], s["sizes"])}
        if case["bits"] == 8:
            state.update(m_scale=part(s["m_scale"], s["blocks"]), v_scale=part(s["v_scale"], s["blocks"]))
        s["opt"] = ed.AdamW(part(s["w"], s["sizes"]), part(s["g"], s["sizes"]),
                            masters=part(s["master"], s["sizes"]) if case["master"] else None,
                            state_bits=case["bits"], state=state, counts=case["counts"], lr=LR,
                            betas=(B1, B2), eps=EPS, weight_decay=s["decay"], step=s["t"])
        if case["bits"] == 8:
            s["values"] = [torch.empty(sum(s["sizes"]), dtype=torch.bfloat16, device="cuda") for _ in "mv"]
            s["parts"] = [part(t, s["sizes"]) for t in s["values"]]
    opt = s["opt"]
    norm = opt.step(max_norm=MAX_NORM if case["clip"] else None)
    out = {"w": s["w"], "norm": norm}
    if case["master"]:
        out["master"] = s["master"]
    if case["bits"] == 8:
        opt.state_values(*s["parts"])
        out["m"], out["v"] = s["values"]
    else:
        out["m"], out["v"] = s["m"], s["v"]
    if case["counts"]:
        out["counts"] = opt.counts
    return out


def _adamw(s):
    if own:
        return _adamw_own(s)
    case = s["case"]
    s["t"] += 1
    out, norm = {}, None
    g = s["g"].float()
    if case["clip"]:
        norm = s["g"].double().square().sum().sqrt()
        norm = torch.stack([norm, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)]).float()
        g = g * norm[1]
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        b = s["block_of"]
        c = s["m"].float()
        m = s["m_scale"][b] * (c * c.abs())
        c = s["v"].float()
        v = (s["v_scale"][b] * (c * c)).square()
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * (1 - B2) * g
    r = v.sqrt()
    upd = m / (r * (1 / math.sqrt(1 - B2 ** s["t"])) + EPS)
    w = (s["master"] if case["master"] else s["w"].float()) * s["keep"][s["tensor_of"]]
    w = w - upd * (LR / (1 - B1 ** s["t"]))
    if case["master"]:
        out["master"] = s["master"].copy_(w)
    out["w"] = s["w"].copy_(w)
    if case["bits"] == 32:
        out["m"], out["v"] = s["m"].copy_(m), s["v"].copy_(v)
    else:
        out["m"], out["v"] = _hold(s, m, r)
    if case["counts"]:
        e = (out["w"].view(torch.int16).int() >> 7) & 0xFF
        k = len(s["sizes"])
        out["counts"] = torch.bincount(s["tensor_of"] * 256 + e, minlength=256 * k).view(k, 256)
    return dict(out, norm=norm)


def _hold(s, m, r):
    """Stores m and r = sqrt(v) as codes and scales; the values they stand for, m and v."""
    b = s["block_of"]
    padded = m.new_zeros(s["m_scale"].numel(), BLOCK)
    padded.view(-1)[s["at"]] = m.abs()
    top = padded.amax(1)
    sm = torch.where(top < TINY, 0.0, top / 127 ** 2)
    c = (m.abs() * torch.where(sm > 0, 1 / sm, 0.0)[b]).sqrt().round().clamp(max=127)
    c = torch.where(m < 0, -c, c)
    padded.view(-1)[s["at"]] = r
    sv = padded.amax(1) / 255 ** 2
    d = (r * torch.where(sv > 0, 1 / sv, 0.0)[b]).sqrt().round().clamp(max=255)
    d = torch.where(r > 0, d.clamp(min=1), 0.0)
    s["m"].copy_(c), s["v"].copy_(d), s["m_scale"].copy_(sm), s["v_scale"].copy_(sv)
    return (sm[b] * (c * c.abs())).bfloat16(), (sv[b] * (d * d)).square().bfloat16()


def run(state):
    return _int8(state) if state["case"]["op"] == "int8" else _adamw(state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int8":
        def codes(x):
            x = x.double()
            top = x.abs().max(dim=1).values
            return torch.where((top > 0)[:, None], (127 * x / top[:, None]).round(), 0.0), top / 127

        held = {i: codes(x) for i, x in s["x"].items()}
        out = []
        for k, (rows, cols) in enumerate(s["shapes"]):
            if case["fresh"]:
                qw, sw = codes(s["w"][k])
            else:
                qw, sw = s["w"][k].double()[:, :cols], s["w_scale"][k].double()
            qx, sx = held[s["index"][k]]
            out.append(torch.matmul(qx, qw.t()).mul_(sx.view(-1, 1)).mul_(sw.view(1, -1)))
        return out
    t = s["t"] + 1
    g = s["g"].double()
    norm = None
    if case["clip"]:
        length = torch.linalg.vector_norm(g)
        factor = min(1.0, MAX_NORM / (float(length) + 1e-6))
        norm = torch.tensor([float(length), factor], dtype=torch.float64)
        g = g * factor
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        sm, sv = (s[k].double()[s["block_of"]] for k in ("m_scale", "v_scale"))
        m = sm * s["m"].double() * s["m"].double().abs()
        v = (sv * s["v"].double() ** 2) ** 2
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g ** 2
    step = (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)) ** 0.5 + EPS)
    lam = torch.tensor(s["decay"], dtype=torch.float64, device="cuda")[s["tensor_of"]]
    w = s["master"].double() if case["master"] else s["w"].double()
    w = w - LR * lam * w - LR * step
    out = {"w": w, "norm": norm}
    if case["master"]:
        out["master"] = w
    if case["counts"]:
        out["counts"] = None
    if case["bits"] == 32:
        out["m"], out["v"] = m, v
        return out
    index, blocks = s["at"] // BLOCK, s["m_scale"].numel()
    for name, value, most in (("m", m, 127), ("v", v.sqrt(), 255)):
        top = torch.zeros(blocks, dtype=torch.float64, device="cuda")
        top.index_reduce_(0, index, value.abs(), "amax")
        code = ((value.abs() / top[index]).sqrt() * most).round()
        if name == "v":
            code = torch.where(value > 0, code.clamp(min=1), code)
        held = value.sign() * top[index] * (code / most) ** 2
        out[name] = held if name == "m" else held * held
    return out


def work(case):
    if case["op"] == "int8":
        mats, t = _mats(case), case["tokens"]
        size = {"bf16": 2, "f16": 2, "f32": 4}
        xs = {i: c for _, c, i in mats}
        nbytes = sum(r * c * (2 if case["fresh"] else 1) + (0 if case["fresh"] else 4 * r) for r, c, _ in mats)
        nbytes += t * sum(xs.values()) * size[case["x"]] + t * sum(r for r, _, _ in mats) * size[case["y"]]
        return {"bytes": nbytes, "flops": 2 * t * sum(r * c for r, c, _ in mats)}
    sizes = _sizes(case)
    n = sum(sizes)
    w, g = (2 if case[k] == "bf16" else 4 for k in ("w", "g"))
    each = g + w + (8 if case["master"] else w)  # masters are read and written, the weights then only written
    nbytes = n * each
    if case["bits"] == 32:
        nbytes += 16 * n
    else:  # codes and scales read and written, and the values they stand for written
        nbytes += 4 * n + 16 * sum(-(-c // BLOCK) for c in sizes) + 4 * n
    if case["counts"]:
        nbytes += 8 * 256 * len(sizes)
    return {"bytes": nbytes, "flops": (20 if case["bits"] == 32 else 45) * n}
