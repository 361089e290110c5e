"""Measured cases of the gradient-norm and clipping operators: the global norm
over many tensors, clipping (in place, or into tensors of another type), and
the AdamW and Muon steps that take the clip factor as they read the gradients.

With `own` false, run() computes an operator from elementary torch operations
in 32 bits on the flat buffers behind the tensor lists; with `own` true it
makes the library calls a training program makes on the lists.

Definitions (g_i the gradients, all sums over every element of every tensor):
  norm   = scale * sqrt(sum g^2)
  factor = scale * min(1, max_norm / (norm + 1e-6))
  clip   out = g * factor
  AdamW  on g' = g * factor:  p <- p (1 - lr wd); u <- b1 u + (1 - b1) g';
         v <- b2 v + (1 - b2) g'^2;
         p <- p - lr (u / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
  Muon   on g' = g * factor:  m <- beta m + g'; x = bf16((g' + beta m) /
         (||g' + beta m||_F + 1e-7)); ns times: a = bf16(x x^T),
         b = bf16(cb a + cc a a), x = bf16(ca x + b x); w <- w - lr x
"""
import math
import random

import torch

own = False

WIDTH, LAYERS = 768, 12          # GPT-2 124M
WIDTH_XL, LAYERS_XL = 1600, 48   # the GPT-2-XL shape
VOCAB, CONTEXT = 50257, 1024
BETA1, BETA2, EPS, DECAY, LR_ADAMW, STEP = 0.9, 0.95, 1e-8, 0.1, 6e-4, 1000
LR_MUON, BETA, NS_STEPS, COEFFS = 2e-4, 0.95, 5, (3.4445, -4.7750, 2.0315)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # Gradient norm of one block's 1-D parameters: a call whose time is its latency.
        dict(name="norm-block-1d", op="norm", set="block-1d", grads="fp32", std=1e-3, max_norm=1.0, scale=1.0),
        # The norm every training step of GPT-2 124M logs and clips by: 148 tensors, fp32.
        dict(name="norm-gpt2-fp32", op="norm", set="gpt2", grads="fp32", std=1e-3, max_norm=1.0, scale=1.0),
        # The same at the XL shape with bf16 gradients: 580 tensors, 3.1 GB.
        dict(name="norm-xl-bf16", op="norm", set="xl", grads="bf16", std=1e-3, max_norm=1.0, scale=1.0),
        # Shards cut at odd places, 16-bit and fp32 gradients in one call: odd sizes, unaligned views.
        dict(name="norm-ragged-mixed", op="norm", set="ragged", count=61, total=5_000_011, grads="mixed", std=1e-2,
             max_norm=1.0, scale=0.25),
        # A stable run's usual step: the norm is below the limit, so the gradients stay as they are.
        dict(name="clip-gpt2-below", op="clip", set="gpt2", grads="fp32", outs="in place", std=2e-5, max_norm=1.0,
             scale=1.0),
        # bf16 gradients of four micro-batches averaged and clipped into fp32 main gradients.
        dict(name="clip-gpt2-bf16-fp32", op="clip", set="gpt2", grads="bf16", outs="fp32", std=1e-3, max_norm=1.0,
             scale=0.25),
        # fp16 gradients under a loss scale of 1024, unscaled and clipped, odd shards of mid size.
        dict(name="clip-ragged-fp16", op="clip", set="ragged", count=37, total=1_000_003, grads="fp16", outs="fp32",
             std=1.0, max_norm=0.5, scale=2.0 ** -10),
        # AdamW over one block's 1-D parameters after clipping: latency again.
        dict(name="adamw-block-1d", op="adamw", set="block-1d", grads="fp32", std=1e-3, max_norm=0.05, scale=1.0),
        # Norm and step over the GPT-2 parameters AdamW takes (embeddings and 1-D): 100 tensors, 39.5 M elements.
        dict(name="adamw-gpt2-rest", op="adamw", set="gpt2-rest", grads="fp32", std=1e-3, max_norm=1.0, scale=1.0),
        # Norm and step over a whole XL-shaped model with bf16 gradients: the largest call.
        dict(name="adamw-xl-bf16", op="adamw", set="xl", grads="bf16", std=1e-3, max_norm=1.0, scale=1.0),
        # Norm and Muon step of one small matrix: the smallest Muon call.
        dict(name="muon-256x512", op="muon", set="matrices", shapes="256x512", grads="fp32", std=1e-3, max_norm=0.1,
             scale=1.0),
        # Norm and Muon step of one GPT-2 124M block's four matrices.
        dict(name="muon-gpt2-block", op="muon", set="matrices", grads="fp32", std=1e-3, max_norm=1.0, scale=1.0,
             shapes="x".join(map(str, (WIDTH, 3 * WIDTH))) + f",{WIDTH}x{WIDTH},{WIDTH}x{4 * WIDTH},{4 * WIDTH}x{WIDTH}"),
    ]


def draw(rng):
    """Tensor lists of 1 to 200 tensors, 2^10 to 2^27 elements in all, aligned
    or odd, of each type, below and above the limit; 1 to 4 matrices."""
    op = rng.choice(["norm", "norm", "clip", "clip", "adamw", "adamw", "muon"])
    case = dict(op=op, scale=rng.choice([1.0, 0.25, 0.125]))
    if op == "muon":
        dims = [(int(2 ** rng.uniform(7, 11)), int(2 ** rng.uniform(7, 11))) for _ in range(rng.randint(1, 4))]
        numel = sum(r * c for r, c in dims)
        case.update(set="matrices", shapes=",".join(f"{r}x{c}" for r, c in dims), grads="fp32")
    else:
        numel = int(2 ** rng.uniform(10, 27))
        count = int(2 ** rng.uniform(0, math.log2(200)))
        case.update(set=rng.choice(["ragged", "ragged", "padded"]), count=count, total=max(numel, 512 * count),
                    grads=rng.choice(["fp32", "bf16", "fp16"] + (["mixed"] if op == "norm" else [])))
        if op == "clip":
            case["outs"] = rng.choice(["fp32", case["grads"]])
    case["std"] = 2.0 ** rng.uniform(-6, -2)
    # the limit between a sixteenth and four times the norm that such gradients have
    case["max_norm"] = case["std"] * math.sqrt(numel) * case["scale"] * 2.0 ** rng.uniform(-4, 2)
    return case


def _layers(width, layers):
    vectors = [width, width, 3 * width, width, width, width, 4 * width, width]
    matrices = [3 * width * width, width * width, 4 * width * width, 4 * width * width]
    return vectors * layers, matrices * layers


def sizes(case):
    """(element counts of the tensors, how many leading ones are decayed)."""
    kind = case["set"]
    if kind == "block-1d":
        return _layers(WIDTH, 1)[0], 0
    if kind in ("gpt2", "gpt2-rest", "xl"):
        width, layers = (WIDTH_XL, LAYERS_XL) if kind == "xl" else (WIDTH, LAYERS)
        vectors, matrices = _layers(width, layers)
        decayed = [VOCAB * width, CONTEXT * width] + (matrices if kind != "gpt2-rest" else [])
        return decayed + vectors + [width, width], len(decayed)
    if kind == "matrices":
        return [math.prod(map(int, s.split("x"))) for s in case["shapes"].split(",")], 0
    # random cuts of the total: odd shards, or shards padded to 64 elements
    r = random.Random(case["count"] * 1_000_003 + case["total"])
    cuts = sorted(r.randint(0, case["total"]) for _ in range(case["count"] - 1))
    counts = [b - a for a, b in zip([0] + cuts, cuts + [case["total"]])]
    if kind == "padded":
        counts = [-(-max(c, 1) // 64) * 64 for c in counts]
    return counts, case["count"] // 2


# ------------------------------------------------------------------ inputs --

def _views(flat, counts):
    return list(torch.split(flat, counts))


def prepare(case, seed):
    counts, decayed = sizes(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = random.Random(seed)
    normal = lambda n, std: torch.randn(n, generator=gen, device="cuda").mul_(std)  # noqa: E731
    kinds = ["fp32", "bf16", "fp16"] if case["grads"] == "mixed" else [case["grads"]]
    state = dict(case=case, flats=[], grads=[], decayed=sum(counts[:decayed]))
    for k, kind in enumerate(kinds):
        mine = counts[k::len(kinds)]
        flat = normal(sum(mine), case["std"])
        if len(mine) > 1:  # tensors of different layers differ in size
            for view in _views(flat, mine):
                view.mul_(2.0 ** pick.uniform(-1, 1))
        flat = flat.to(DTYPES[kind])
        state["flats"].append(flat)
        state["grads"] += _views(flat, mine)
    total = sum(counts)
    if case["op"] == "clip" and case["outs"] != "in place":
        state["out"] = torch.empty(total, dtype=DTYPES[case["outs"]], device="cuda")
        state["outs"] = _views(state["out"], counts)
    if case["op"] in ("adamw", "muon"):
        state["p"] = normal(total, 0.02)
        state["m"] = normal(total, 0.1 * case["std"])
    if case["op"] == "adamw":
        state["v"] = normal(total, case["std"]).square_()
        for k in "pmv":
            state["list_" + k] = _views(state[k], counts)
        state["wd"] = [DECAY] * decayed + [0.0] * (len(counts) - decayed)
    if case["op"] == "muon":
        shapes = [tuple(map(int, s.split("x"))) for s in case["shapes"].split(",")]
        state["update"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
        for k, flat in (("p", state["p"]), ("m", state["m"]), ("update", state["update"])):
            state["list_" + k] = [t.view(s) for t, s in zip(_views(flat, counts), shapes)]
        state["grads"] = [t.view(s) for t, s in zip(state["grads"], shapes)]
    return state


# --------------------------------------------------------------- the passes --

def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import optimizer_muon_step_amd as mu
    case = state["case"]
    if case["op"] == "clip":
        record = mu.muon_grad_clip(state["grads"], case["max_norm"], scale=case["scale"], outs=state.get("outs"))
        return {"record": record, "grads": state.get("out", state["flats"][0])}
    record = mu.muon_grad_norm(state["grads"], case["max_norm"], scale=case["scale"])
    if case["op"] == "adamw":
        mu.muon_adamw_step(state["list_p"], state["grads"], state["list_m"], state["list_v"], LR_ADAMW, (BETA1, BETA2),
                           EPS, state["wd"], step=STEP, clip=record)
        return {"record": record, "p": state["p"], "m": state["m"], "v": state["v"]}
    if case["op"] == "muon":
        mu.muon_step(state["list_p"], state["grads"], state["list_m"], LR_MUON, BETA, NS_STEPS, COEFFS,
                     updates=state["list_update"], clip=record)
        return {"record": record, "p": state["p"], "m": state["m"], "update": state["update"]}
    return {"record": record}


def _record(flats, max_norm, scale):
    norm = sum(f.float().square().sum() for f in flats).sqrt() * scale
    return torch.stack([norm, scale * (max_norm / (norm + 1e-6)).clamp(max=1.0)])


def _plain(state):
    case = state["case"]
    record = _record(state["flats"], case["max_norm"], case["scale"])
    if case["op"] == "norm":
        return {"record": record}
    flat = state["flats"][0]
    if case["op"] == "clip":
        if case["outs"] == "in place":
            return {"record": record, "grads": flat.mul_(record[1])}
        return {"record": record, "grads": state["out"].copy_(flat.float() * record[1])}
    g = flat.float() * record[1]
    if case["op"] == "adamw":
        p, m, v = state["p"], state["m"], state["v"]
        p[:state["decayed"]].mul_(1 - LR_ADAMW * DECAY)
        m.mul_(BETA1).add_(g * (1 - BETA1))
        v.mul_(BETA2).add_(g.square_().mul_(1 - BETA2))
        root = (v / (1 - BETA2 ** STEP)).sqrt_().add_(EPS)
        p.sub_((m * (LR_ADAMW / (1 - BETA1 ** STEP))).div_(root))
        return {"record": record, "p": p, "m": m, "v": v}
    m = state["m"].mul_(BETA).add_(g)
    look = _views(g + BETA * m, [t.numel() for t in state["list_p"]])
    state["update"].copy_(torch.cat([_orthogonal(u.view(t.shape), torch.float32).reshape(-1)
                                     for u, t in zip(look, state["list_p"])]))
    state["p"].sub_(LR_MUON * state["update"].float())
    return {"record": record, "p": state["p"], "m": m, "update": state["update"]}


def _orthogonal(u, wide):
    """Newton-Schulz of one matrix: bf16 storage points, products in `wide`."""
    bf16 = lambda t: t.to(torch.bfloat16).to(wide)  # noqa: E731
    a, b, c = COEFFS
    x = bf16(u / (u.square().sum().sqrt() + 1e-7))
    x = x.T.contiguous() if u.shape[0] > u.shape[1] else x
    for _ in range(NS_STEPS):
        gram = bf16(x @ x.T.contiguous())
        poly = bf16(b * gram + c * (gram @ gram))
        x = bf16(a * x + poly @ x)
    return x.T if u.shape[0] > u.shape[1] else x


def exact(case, seed):
    """The definitions in 64 bits (Muon with its bf16 storage points; the bf16
    update itself has no one value: which way a sum next to a rounding border
    goes decides its last bits)."""
    state = prepare(case, seed)
    total = sum((f.double().square().sum() for f in state["flats"]), torch.zeros((), dtype=torch.float64, device="cuda"))
    norm = total.sqrt() * case["scale"]
    factor = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0) * case["scale"]
    record = torch.stack([norm, factor])
    if case["op"] == "norm":
        return {"record": record}
    g = state["flats"][0].double() * factor
    if case["op"] == "clip":
        return {"record": record, "grads": g}
    m, p = state["m"].double(), state["p"].double()
    if case["op"] == "adamw":
        del state["flats"], state["grads"]
        m = m.mul_(BETA1).add_(g, alpha=1 - BETA1)
        v = state["v"].double().mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
        del g
        p[:state["decayed"]] *= 1 - LR_ADAMW * DECAY
        p.addcdiv_(m / (1 - BETA1 ** STEP), (v / (1 - BETA2 ** STEP)).sqrt_() + EPS, value=-LR_ADAMW)
        return {"record": record, "p": p, "m": m, "v": v}
    m = BETA * m + g
    look = _views(g + BETA * m, [t.numel() for t in state["list_p"]])
    update = torch.cat([_orthogonal(u.view(t.shape), torch.float64).reshape(-1) for u, t in zip(look, state["list_p"])])
    return {"record": record, "p": p - LR_MUON * update, "m": m, "update": None}


def work(case):
    counts, _ = sizes(case)
    n = sum(counts)
    kinds = ["fp32", "bf16", "fp16"] if case["grads"] == "mixed" else [case["grads"]]
    read = sum(BYTES[kind] * sum(counts[k::len(kinds)]) for k, kind in enumerate(kinds))
    if case["op"] == "norm":
        return {"bytes": read + 8, "flops": 2 * n}
    if case["op"] == "clip":  # below the limit and in place there is nothing to write
        return {"bytes": read + (0 if case["outs"] == "in place" else BYTES[case["outs"]] * n), "flops": 3 * n}
    if case["op"] == "adamw":
        return {"bytes": read + 24 * n, "flops": 18 * n}
    flops = 0
    for s in case["shapes"].split(","):
        a, b = sorted(map(int, s.split("x")))
        # the Gram and the square are symmetric: half of each is enough
        flops += NS_STEPS * (a * a * b + a * a * a + 2 * a * a * b)
    return {"bytes": read + 18 * n, "flops": flops + 8 * n}
