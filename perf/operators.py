"""Workloads of the optimiser-side operators over many tensors: the global
gradient norm, clipping by it, and the AdamW update that takes the clip
coefficient.

A case's tensors are views of one flat buffer per role, as gradient buckets
and flattened optimiser states are kept: "aligned" starts every tensor on a
256-byte boundary, "packed" starts it right behind the one before it (odd
offsets), and "columns" makes the tensors column slices of one fused matrix.
The buffers are what run() returns, so every element of every tensor comes
back; the gaps between aligned tensors hold zeros.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS_CLIP = 1e-6
ADAM = {"lr": 1e-3, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}


def listed():
    return [
        # the norm weights and biases of a small model: the smallest call, all latency
        {"name": "norm-vectors", "op": "norm", "count": 24, "rows": 1, "cols": 1024, "ragged": False,
         "layout": "aligned", "grad": "f32", "ord": "2", "per_tensor": False},
        # twelve layers' worth of 1024x4096 matrices with every tensor's own norm for the log
        {"name": "norm-per-tensor", "op": "norm", "count": 36, "rows": 1024, "cols": 4096, "ragged": False,
         "layout": "aligned", "grad": "bf16", "ord": "2", "per_tensor": True},
        # the largest absolute gradient of odd-sized tensors packed into one fp16 bucket
        {"name": "norm-max-packed", "op": "norm", "count": 90, "rows": 257, "cols": 1531, "ragged": True,
         "layout": "packed", "grad": "f16", "ord": "inf", "per_tensor": False},
        # a dense model's MLP gradients, 8 x 4096x16384
        {"name": "norm-dense-mlp", "op": "norm", "count": 8, "rows": 4096, "cols": 16384, "ragged": False,
         "layout": "aligned", "grad": "bf16", "ord": "2", "per_tensor": False},
        # a stack of 64 expert gradients 2048x7168 whose norm is below the bound, clipped in place
        {"name": "clip-experts-below", "op": "clip", "count": 64, "rows": 2048, "cols": 7168, "ragged": False,
         "layout": "aligned", "grad": "bf16", "out": "", "bound": 2.0, "scaled": False},
        # 16-bit gradients unscaled and clipped into fp32 main gradients
        {"name": "clip-main-grads", "op": "clip", "count": 16, "rows": 1024, "cols": 4096, "ragged": False,
         "layout": "aligned", "grad": "f16", "out": "f32", "bound": 0.25, "scaled": True},
        # query, key and value gradients as odd column slices of one fused matrix, clipped into a 16-bit buffer
        {"name": "clip-columns", "op": "clip", "count": 3, "rows": 513, "cols": 777, "ragged": False,
         "layout": "columns", "grad": "bf16", "out": "bf16", "bound": 0.5, "scaled": False},
        # norm weights and biases of a small model: the smallest update
        {"name": "adamw-vectors", "op": "adamw", "count": 48, "rows": 1, "cols": 1024, "ragged": False,
         "layout": "aligned", "grad": "f32", "copy": "", "bound": 0.0},
        # embedding and output head in mixed precision: 16-bit gradients, fp32 master weights, 16-bit copy, clipped
        {"name": "adamw-embedding", "op": "adamw", "count": 2, "rows": 32768, "cols": 4096, "ragged": False,
         "layout": "aligned", "grad": "bf16", "copy": "bf16", "bound": 0.5},
        # a few hundred odd-sized tensors packed into flat buffers, fp32 gradients, clipped
        {"name": "adamw-packed", "op": "adamw", "count": 200, "rows": 61, "cols": 1283, "ragged": True,
         "layout": "packed", "grad": "f32", "copy": "", "bound": 0.5},
    ]


def draw(rng):
    op = rng.choice(["norm", "clip", "adamw"])
    most = {"norm": 29.0, "clip": 28.0, "adamw": 27.0}[op]
    total = 2.0 ** rng.uniform(13.0, most)
    count = min(int(2.0 ** rng.uniform(0.0, 9.0)), max(1, int(total / 256)))
    each = total / count
    cols = max(1, min(20000, int(each / 2.0 ** rng.uniform(0.0, 12.0))))
    rows = max(1, int(each / cols))
    case = {"op": op, "count": count, "rows": rows, "cols": cols, "ragged": rng.random() < 0.5,
            "layout": rng.choice(["aligned", "aligned", "packed", "columns"]),
            "grad": rng.choice(["f32", "bf16", "f16"])}
    if case["layout"] == "columns":
        case["ragged"] = False
    if op == "norm":
        case.update(ord=rng.choice(["2", "2", "inf"]), per_tensor=rng.random() < 0.5)
    elif op == "clip":
        case.update(out=rng.choice(["", "f32", case["grad"]]), bound=rng.choice([0.25, 0.5, 2.0]))
        case["scaled"] = case["out"] != "" and rng.random() < 0.5
    else:
        case.update(copy=rng.choice(["", "bf16", "f16"]), bound=rng.choice([0.0, 0.5, 2.0]))
    return case


def shapes(case):
    rows, cols = case["rows"], case["cols"]
    if not case["ragged"]:
        return [(rows, cols)] * case["count"]
    return [(rows - i * 37 % (rows // 2 + 1), cols - i * 53 % (cols // 2 + 1)) for i in range(case["count"])]


def elements(case):
    return sum(r * c for r, c in shapes(case))


def places(case):
    """(offset, shape, strides) of every tensor in its flat buffer, and the buffer's length."""
    at, got = 0, []
    if case["layout"] == "columns":
        pitch = case["cols"] * case["count"]
        return [(i * case["cols"], (case["rows"], case["cols"]), (pitch, 1)) for i in range(case["count"])], \
            pitch * case["rows"]
    for r, c in shapes(case):
        got.append((at, (r, c), (c, 1)))
        at += r * c
        if case["layout"] == "aligned":
            at = (at + 127) // 128 * 128
    return got, at


def views(case, flat):
    return [flat.as_strided(shape, strides, flat.storage_offset() + at) for at, shape, strides in places(case)[0]]


def gradients(case, seed, gen):
    """A flat buffer of gradients: every tensor's entries normal with a spread of its own."""
    flat = torch.zeros(places(case)[1], dtype=TYPES[case["grad"]], device="cuda")
    for i, g in enumerate(views(case, flat)):
        g.normal_(0.0, 0.002 * (1 + (i * 7 + seed) % 5), generator=gen)
    return flat


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    flat = gradients(case, seed, gen)
    s = {"case": case, "grad": flat, "grads": views(case, flat), "step": 0, "inv_scale": None, "max_norm": math.inf}
    if case.get("scaled"):
        flat.mul_(256.0)
        s["inv_scale"] = torch.tensor(1.0 / 256.0, device="cuda")
    if case.get("bound"):
        # a bound that is this share of the norm the gradients are expected to have
        spread = [0.002 * (1 + (i * 7 + seed) % 5) for i in range(case["count"])]
        s["max_norm"] = case["bound"] * math.sqrt(sum(r * c * d * d for (r, c), d in zip(shapes(case), spread)))
    if case["op"] == "clip" and case["out"]:
        s["out"] = torch.zeros(flat.numel(), dtype=TYPES[case["out"]], device="cuda")
    if case["op"] == "adamw":
        for name, spread in (("param", 0.02), ("exp_avg", 0.004), ("exp_avg_sq", 0.002)):
            s[name] = torch.zeros(flat.numel(), device="cuda")
            for t in views(case, s[name]):
                t.normal_(0.0, spread, generator=gen)
        s["exp_avg_sq"].square_()
        s["step"] = 10
        if case["copy"]:
            s["copy"] = s["param"].to(TYPES[case["copy"]])
    if own:
        import gram_newton_schulz_amd as gns
        # the lists of tensors that a training loop builds once
        if case["op"] == "adamw":
            s["list"] = gns.adamw_list(views(case, s["param"]), s["grads"], views(case, s["exp_avg"]),
                                       views(case, s["exp_avg_sq"]),
                                       copies=views(case, s["copy"]) if case["copy"] else None)
        else:
            s["list"] = gns.tensor_list(s["grads"], out=views(case, s["out"]) if "out" in s else None)
    return s


def run_own(s):
    import gram_newton_schulz_amd as gns
    case = s["case"]
    if case["op"] == "norm":
        got = gns.grad_norm(s["list"], ord=float(case["ord"]), per_tensor=case["per_tensor"])
        return {"norm": got.norm, "tensor_norms": got.tensor_norms}
    if case["op"] == "clip":
        got = gns.clip_grad_norm_(s["list"], s["max_norm"], eps=EPS_CLIP, inv_scale=s["inv_scale"])
        return {"norm": got.norm, "grad": s.get("out", s["grad"])}
    s["step"] += 1
    out = {}
    clip = None
    if case["bound"]:
        got = gns.grad_norm(s["list"], max_norm=s["max_norm"], eps=EPS_CLIP)
        out["norm"], clip = got.norm, got.clip
    gns.adamw_step(s["list"], s["step"], grad_scale=clip, **ADAM)
    out.update({k: s[k] for k in ("param", "exp_avg", "exp_avg_sq", "copy") if k in s})
    return out


def plain_norm(s):
    """Norm of the (unscaled) gradients and the factor that unscales and clips them."""
    x = s["grad"].float()
    norm = (x * x).sum().sqrt()
    inv = 1.0 if s["inv_scale"] is None else s["inv_scale"]
    norm = norm * inv
    return x, norm, inv * torch.clamp(s["max_norm"] / (norm + EPS_CLIP), max=1.0)


def run(s):
    if own:
        return run_own(s)
    case = s["case"]
    if case["op"] == "norm":
        x = s["grad"].float()
        each = None
        if case["ord"] == "inf":
            norm = x.abs().max()
            if case["per_tensor"]:
                each = torch.stack([g.abs().max() for g in views(case, x)])
        elif case["per_tensor"]:
            each = torch.stack([(g * g).sum() for g in views(case, x)])
            norm, each = each.sum().sqrt(), each.sqrt()
        else:
            norm = (x * x).sum().sqrt()
        return {"norm": norm, "tensor_norms": each}
    if case["op"] == "clip":
        x, norm, clip = plain_norm(s)
        return {"norm": norm, "grad": s.get("out", s["grad"]).copy_(x * clip)}
    s["step"] += 1
    (b1, b2), t = ADAM["betas"], s["step"]
    out = {}
    if case["bound"]:
        g, out["norm"], clip = plain_norm(s)
        g = g * clip
    else:
        g = s["grad"].float()
    s["exp_avg"].mul_(b1).add_(g * (1 - b1))
    s["exp_avg_sq"].mul_(b2).add_(g * g * (1 - b2))
    denom = s["exp_avg_sq"].sqrt() / math.sqrt(1 - b2 ** t) + ADAM["eps"]
    s["param"].mul_(1 - ADAM["lr"] * ADAM["weight_decay"]).sub_(s["exp_avg"] / denom * (ADAM["lr"] / (1 - b1 ** t)))
    if case["copy"]:
        s["copy"].copy_(s["param"])
    out.update({k: s[k] for k in ("param", "exp_avg", "exp_avg_sq", "copy") if k in s})
    return out


def work(case):
    n = elements(case)
    read = n * SIZE[case["grad"]]
    if case["op"] == "norm":
        return {"bytes": read + 4 + (4 * case["count"] if case["per_tensor"] else 0), "flops": 2 * n}
    if case["op"] == "clip":
        # in place and below the bound nothing changes
        write = n * SIZE[case["out"] or case["grad"]] if case["out"] or case["bound"] < 1 or case["scaled"] else 0
        return {"bytes": read + write, "flops": (3 if write else 2) * n}
    write = n * (12 + (SIZE[case["copy"]] if case["copy"] else 0))
    return {"bytes": read + 12 * n + write, "flops": (17 if case["bound"] else 14) * n}


def exact(case, seed):
    """The definitions in 64 bits, tensor by tensor where run() goes over the flat buffers."""
    s = prepare(dict(case), seed)
    g = s["grad"].double()
    inv = 1.0 if s["inv_scale"] is None else float(s["inv_scale"])
    if case["op"] == "norm" and case["ord"] == "inf":
        each = [float(t.abs().max()) for t in views(case, g)]
        norm = max(each)
    else:
        each = [math.sqrt(float(torch.dot(t.reshape(-1), t.reshape(-1)))) * inv for t in views(case, g)]
        norm = math.sqrt(math.fsum(e * e for e in each))
    if case["op"] == "norm":
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "tensor_norms": torch.tensor(each, dtype=torch.float64) if case["per_tensor"] else None}
    g *= inv * min(1.0, s["max_norm"] / (norm + EPS_CLIP))
    if case["op"] == "clip":
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grad": g}
    (b1, b2), t = ADAM["betas"], s["step"] + 1
    m = s["exp_avg"].double() * b1 + (1 - b1) * g
    v = s["exp_avg_sq"].double() * b2 + (1 - b2) * g.square()
    del g
    p = s["param"].double() * (1 - ADAM["lr"] * ADAM["weight_decay"])
    p -= ADAM["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + ADAM["eps"])
    got = {"param": p, "exp_avg": m, "exp_avg_sq": v}
    if case["copy"]:
        got["copy"] = p
    if case["bound"]:
        got["norm"] = torch.tensor(norm, dtype=torch.float64)
    return got
