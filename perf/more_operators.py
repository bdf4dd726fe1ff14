"""Workloads of the first and the inner layers of the model whose parameters the
library updates: the token embedding with its gradient, and linear layers whose
products run in microscaled 4-bit floating point (MXFP4).

MXFP4 holds blocks of 32 consecutive values as 4-bit floats (sign, two bits of
exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times one power of two
per block.  For a block with the largest magnitude a the power is
2^(floor(log2 a) - 2), and values are rounded to nearest, ties to even, larger
ones than 6 to 6.  With given random bytes r they are rounded up with
probability: from t = n + f steps to n + 1 where 256 f > r + 0.5, and the power
is doubled where a would be above 6, so that no value is cut off.

A linear layer is y = Q(x) Q(w)^T, its gradients dx = Q(dy) Q(w^T)^T and
dw = Q(dy^T) Q(x^T)^T, with blocks along the axis that each product sums over.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
SCALE = 8.0        # on embedded rows, and on their gradient
BLOCK = 32


def listed():
    return [
        # the last token of sixteen requests being answered: all latency
        {"name": "lookup-decode", "op": "lookup", "tokens": 16, "vocab": 32768, "width": 4096,
         "table": "bf16", "out": "bf16", "pad": 0.0, "skew": 0.0},
        # a training batch of 8 x 4096 tokens, from fp32 masters
        {"name": "lookup-train", "op": "lookup", "tokens": 32768, "vocab": 32768, "width": 4096,
         "table": "f32", "out": "bf16", "pad": 0.0, "skew": 0.0},
        # a small model: 1024 windows of four tokens, vocabulary 256, into a slice of a 16-bit gradient bucket
        {"name": "embedding-grad-small", "op": "embedding_grad", "tokens": 4096, "vocab": 256, "width": 128,
         "grad": "bf16", "into": "bf16", "pad": 0.0, "skew": 0.0, "accumulate": False},
        # the training batch: every row of the table's fp32 gradient is written
        {"name": "embedding-grad-train", "op": "embedding_grad", "tokens": 32768, "vocab": 32768, "width": 4096,
         "grad": "bf16", "into": "f32", "pad": 0.0, "skew": 0.0, "accumulate": False},
        # a later microbatch of a padded batch, added to the gradient: odd sizes, a third of the batch padding,
        # a third one token
        {"name": "embedding-grad-padded", "op": "embedding_grad", "tokens": 10007, "vocab": 49999, "width": 1531,
         "grad": "f16", "into": "f32", "pad": 0.33, "skew": 0.33, "accumulate": True},
        # odd fp32 gradients rounded with random bytes, both ways
        {"name": "quantise-odd", "op": "quantise", "batch": 3, "rows": 257, "cols": 1531, "type": "f32",
         "noise": True},
        # a dense model's MLP matrix after its update, for the products of forward and backward pass
        {"name": "quantise-weights", "op": "quantise", "batch": 1, "rows": 4096, "cols": 16384, "type": "f32",
         "noise": False},
        # one token through the down projection: the weights are read once
        {"name": "linear-token", "op": "linear", "batch": 1, "m": 1, "n": 4096, "k": 16384, "type": "bf16"},
        # 64 experts with 48 tokens each
        {"name": "linear-experts", "op": "linear", "batch": 64, "m": 48, "n": 2048, "k": 7168, "type": "bf16"},
        # a training batch through the up projection
        {"name": "linear-train", "op": "linear", "batch": 1, "m": 8192, "n": 16384, "k": 4096, "type": "bf16"},
        # odd sizes throughout
        {"name": "linear-grad-odd", "op": "linear_grad", "batch": 1, "m": 1000, "n": 777, "k": 513, "type": "f16"},
        # the gradients of the training batch, the weights' added to fp32 main gradients
        {"name": "linear-grad-train", "op": "linear_grad", "batch": 1, "m": 8192, "n": 16384, "k": 4096,
         "type": "bf16"},
    ]


def between(rng, low, high):
    """A whole number spread over the logarithm of its range."""
    return int(round(2.0 ** rng.uniform(math.log2(low), math.log2(high))))


def draw(rng):
    op = rng.choice(["lookup", "embedding_grad", "quantise", "linear", "linear", "linear_grad"])
    if op in ("lookup", "embedding_grad"):
        width = between(rng, 16, 8192)
        case = {"op": op, "tokens": min(between(rng, 1, 65536), (1 << 27) // width),
                "vocab": min(between(rng, 64, 131072), (1 << 27) // width), "width": width,
                "pad": rng.choice([0.0, 0.0, rng.uniform(0.0, 0.6)]),
                "skew": rng.choice([0.0, rng.uniform(0.0, 0.4)])}
        if op == "lookup":
            case.update(table=rng.choice(list(TYPES)), out=rng.choice(["bf16", "f16", "f32"]))
        else:
            case.update(grad=rng.choice(list(TYPES)), into=rng.choice(list(TYPES)), accumulate=rng.random() < 0.5)
        return case
    batch = rng.choice([1, 1, 1, between(rng, 2, 64)])
    if op == "quantise":
        total = 2.0 ** rng.uniform(10.0, 26.0) / batch
        cols = max(1, min(20000, int(total ** rng.uniform(0.3, 0.7))))
        return {"op": op, "batch": batch, "rows": max(1, int(total / cols)), "cols": cols,
                "type": rng.choice(list(TYPES)), "noise": rng.random() < 0.5}
    n, k = between(rng, 48, 16384), between(rng, 48, 16384)
    batch = max(1, min(batch, (1 << 29) // (n * k)))
    m = between(rng, 1, 8192) if op == "linear" else between(rng, 64, 8192)
    m = max(1, min(m, int(2.0 ** 39 / (batch * n * k))))
    if rng.random() < 0.5:                             # whole blocks, as most layers are
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    return {"op": op, "batch": batch, "m": m, "n": n, "k": k, "type": rng.choice(["bf16", "bf16", "f16", "f32"])}


# ---------------------------------------------------------------------------
# the plain form of the quantisation: the values that codes and powers stand for
# ---------------------------------------------------------------------------
def power_of_two(exponent):
    """2^exponent in fp32, exactly."""
    return ((exponent.int() + 127) << 23).view(torch.float32)


def rounded(x, noise=None):
    """Q(x) in fp32, with blocks along the last axis."""
    shape = x.shape
    x = x.float()
    short = -shape[-1] % BLOCK
    if short:
        x = torch.nn.functional.pad(x, (0, short))
        noise = None if noise is None else torch.nn.functional.pad(noise, (0, short))
    x = x.reshape(*shape[:-1], -1, BLOCK)
    largest = x.abs().amax(-1, keepdim=True)
    power = power_of_two((torch.frexp(largest)[1] - 3).clamp(min=-126))
    if noise is not None:
        power = torch.where(largest > 6 * power, 2 * power, power)
    t = x.abs() / power
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    t = t / step
    if noise is None:
        t = torch.round(t)
    else:
        whole = torch.floor(t)
        t = whole + ((t - whole) * 256 > noise.reshape(x.shape).float() + 0.5).float()
    t = (t * step).clamp(max=6.0) * power
    t = torch.where(x < 0, -t, t).reshape(*shape[:-1], -1)
    return t[..., :shape[-1]]


def tokens_of(case, gen):
    """Token numbers whose frequency falls with their rank, shuffled over the
    vocabulary; -1 is padding."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp(0, vocab - 1)
    tokens = torch.randperm(vocab, generator=gen, device="cuda")[rank]
    if case["skew"]:
        tokens[torch.rand(n, generator=gen, device="cuda") < case["skew"]] = vocab // 3
    if case["pad"]:
        tokens[torch.rand(n, generator=gen, device="cuda") < case["pad"]] = -1
    return tokens


def values(gen, shape, spread, kind):
    """Normal values whose columns differ in spread, as activations do."""
    x = torch.empty(shape, device="cuda").normal_(0.0, spread, generator=gen)
    return x.mul_(torch.empty(shape[-1], device="cuda").log_normal_(0.0, 0.5, generator=gen)).to(TYPES[kind])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "lookup":
        s["tokens"] = tokens_of(case, gen)
        s["table"] = values(gen, (case["vocab"], case["width"]), 0.02, case["table"])
        return s
    if case["op"] == "embedding_grad":
        s["tokens"] = tokens_of(case, gen)
        s["grad"] = values(gen, (case["tokens"], case["width"]), 0.002, case["grad"])
        s["into"] = torch.zeros(case["vocab"], case["width"], device="cuda", dtype=TYPES[case["into"]])
        if case["accumulate"]:
            s["into"].normal_(0.0, 0.002, generator=gen)
        return s
    if case["op"] == "quantise":
        shape = (case["batch"], case["rows"], case["cols"])
        s["x"] = values(gen, shape, 0.02, case["type"])
        s["noise"] = torch.randint(256, shape, generator=gen, device="cuda", dtype=torch.uint8) if case["noise"] \
            else None
        return s
    b, m, n, k = (case[name] for name in "batch m n k".split())
    x = values(gen, (b, m, k), 1.0, case["type"])
    w = torch.empty(b, n, k, device="cuda").normal_(0.0, k ** -0.5, generator=gen)
    if case["op"] == "linear":
        s["x"] = x
        if own:
            import gram_newton_schulz_amd as gns
            s["w"] = gns.mxfp4_quantize(w)              # once, after the weights' update
        else:
            s["w"] = rounded(w).to(torch.bfloat16)      # (its values are exact in 16 bits)
        return s
    # what the forward pass leaves for the backward pass, the incoming gradient, and the main gradient
    s["dy"] = values(gen, (b, m, n), 0.01, case["type"])
    s["dw"] = torch.empty(b, n, k, device="cuda").normal_(0.0, 0.01, generator=gen)
    if own:
        import gram_newton_schulz_amd as gns
        s["xt"], s["wt"] = gns.mxfp4_quantize(x, transposed=True), gns.mxfp4_quantize(w, transposed=True)
    else:
        s["xt"], s["wt"] = (rounded(t.mT).to(torch.bfloat16) for t in (x, w))
    return s


def run_own(s):
    import gram_newton_schulz_amd as gns
    case = s["case"]
    if case["op"] == "lookup":
        return gns.embedding(s["tokens"], s["table"], scale=SCALE, dtype=TYPES[case["out"]])
    if case["op"] == "embedding_grad":
        return gns.embedding_grad(s["tokens"], s["grad"], s["into"], scale=SCALE, accumulate=case["accumulate"])
    if case["op"] == "quantise":
        rows, columns = gns.mxfp4_quantize_both(s["x"], noise=s["noise"])
        return {"rows": gns.mxfp4_dequantize(rows), "columns": gns.mxfp4_dequantize(columns)}
    if case["op"] == "linear":
        return gns.mxfp4_matmul(s["x"], s["w"], dtype=TYPES[case["type"]])
    rows, columns = gns.mxfp4_quantize_both(s["dy"])
    return {"dx": gns.mxfp4_matmul(rows, s["wt"], dtype=TYPES[case["type"]]),
            "dw": gns.mxfp4_matmul(columns, s["xt"], out=s["dw"], accumulate=True)}


def run(s):
    if own:
        return run_own(s)
    case = s["case"]
    if case["op"] == "lookup":
        got = s["table"][s["tokens"].clamp(min=0)].float() * SCALE
        return torch.where((s["tokens"] >= 0)[:, None], got, 0.0).to(TYPES[case["out"]])
    if case["op"] == "embedding_grad":
        real = s["tokens"] >= 0
        sums = torch.zeros(s["into"].shape, device="cuda")
        sums.index_add_(0, s["tokens"].clamp(min=0), torch.where(real[:, None], s["grad"].float(), 0.0))
        sums *= SCALE
        if case["accumulate"]:
            sums += s["into"]
        return s["into"].copy_(sums)
    if case["op"] == "quantise":
        noise = s["noise"]
        columns = rounded(s["x"].mT, None if noise is None else noise.mT)
        return {"rows": rounded(s["x"], noise).to(torch.bfloat16), "columns": columns.to(torch.bfloat16)}
    if case["op"] == "linear":
        return torch.matmul(rounded(s["x"]), s["w"].float().mT).to(TYPES[case["type"]])
    dx = torch.matmul(rounded(s["dy"]), s["wt"].float().mT)
    s["dw"] += torch.matmul(rounded(s["dy"].mT), s["xt"].float().mT)
    return {"dx": dx.to(TYPES[case["type"]]), "dw": s["dw"]}


def packed(batch, rows, cols):
    """Bytes of a matrix in MXFP4."""
    return batch * rows * (cols / 2 + (cols + BLOCK - 1) // BLOCK)


def work(case):
    if case["op"] == "lookup":
        n, width = case["tokens"], case["width"]
        distinct = min(n, case["vocab"])
        return {"bytes": 8 * n + distinct * width * SIZE[case["table"]] + n * width * SIZE[case["out"]],
                "flops": n * width}
    if case["op"] == "embedding_grad":
        n, width, vocab = case["tokens"], case["width"], case["vocab"]
        real = n * (1.0 - case["pad"])
        # added to the gradient, only the rows of tokens that occur are read and written
        table = 2 * min(real, vocab) if case["accumulate"] else vocab
        return {"bytes": 8 * n + real * width * SIZE[case["grad"]] + table * width * SIZE[case["into"]],
                "flops": real * width}
    if case["op"] == "quantise":
        b, r, c = case["batch"], case["rows"], case["cols"]
        each = b * r * c
        return {"bytes": each * (SIZE[case["type"]] + (1 if case["noise"] else 0) + 2 * 2) + packed(b, r, c) +
                packed(b, c, r), "flops": 4 * each}
    b, m, n, k = (case[name] for name in "batch m n k".split())
    size = SIZE[case["type"]]
    if case["op"] == "linear":
        return {"bytes": b * m * (k + n) * size + packed(b, n, k), "flops": 2.0 * b * m * n * k}
    return {"bytes": b * m * (n + k) * size + packed(b, k, n) + packed(b, k, m) + 8 * b * n * k,
            "flops": 4.0 * b * m * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def nearest(x, noise=None):
    """Q(x) along the last axis, from the definition: the two neighbours of
    every value on the grid, and which of them it goes to."""
    grid = torch.tensor(GRID + (8.0,), dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[-1], BLOCK):
        block = x[..., at:at + BLOCK].double()
        a = block.abs().amax(-1, keepdim=True)
        bits = torch.where(a > 0, a, 1.0).view(torch.int64)            # a >= 0: its exponent is what is above its
        power = (((bits >> 52) - 2) << 52).view(torch.float64)         # 52 bits of mantissa
        if noise is not None:
            power = torch.where(a > 6 * power, 2 * power, power)
        t = block.abs() / power
        low = (torch.searchsorted(grid, t.contiguous(), right=True) - 1).clamp(max=7)
        f = (t - grid[low]) / (grid[low + 1] - grid[low])
        if noise is None:
            up = (f > 0.5) | ((f == 0.5) & (low % 2 == 1))
        else:
            up = 256 * f > noise[..., at:at + BLOCK].double() + 0.5
        out[..., at:at + BLOCK] = torch.copysign(grid[(low + up.long()).clamp(max=7)] * power, block)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        got = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        real = s["tokens"] >= 0
        got[real] = s["table"].double()[s["tokens"][real]] * SCALE
        return got
    if case["op"] == "embedding_grad":
        real = s["tokens"] >= 0
        got = s["into"].double() / SCALE if case["accumulate"] else torch.zeros_like(s["into"], dtype=torch.float64)
        return got.index_add_(0, s["tokens"][real], s["grad"][real].double()).mul_(SCALE)
    if case["op"] == "quantise":
        noise = s["noise"]
        return {"rows": nearest(s["x"], noise),
                "columns": nearest(s["x"].mT, None if noise is None else noise.mT)}
    # the inputs again, as prepare() draws them
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, m, n, k = (case[name] for name in "batch m n k".split())
    x = values(gen, (b, m, k), 1.0, case["type"])
    w = torch.empty(b, n, k, device="cuda").normal_(0.0, k ** -0.5, generator=gen)
    if case["op"] == "linear":
        return torch.matmul(nearest(x), nearest(w).mT)
    return {"dx": torch.matmul(nearest(s["dy"]), nearest(w.mT).mT),
            "dw": s["dw"].double() + torch.matmul(nearest(s["dy"].mT), nearest(x.mT).mT)}
