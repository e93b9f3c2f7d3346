"""Workloads of a training step's products with fused ends: the gated feed-forward
block, the cross entropy of a linear layer's logits, and gradient clipping.

Three operators, each in its plain form (elementary torch operations in 32 bits)
and, with ``own`` set, through the library's entry points:

  gated_ffn             y = (act(x Wg^T) * (x Wu^T)) Wd^T, and its gradients
  linear_cross_entropy  mean over the tokens of logsumexp(x W^T) - (x W^T)[target],
                        and its gradients; tokens with target -100 do not count
  clip_grad_norm        the norm of many tensors taken as one vector, and the
                        tensors scaled so that it is at most max_norm
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100
EPS = 1e-6


def listed():
    return [
        # one token of a served model: bound by one read of the three weights
        {"name": "ffn_serve_1x4096x11008", "op": "gated_ffn", "m": 1, "k": 4096, "f": 11008, "n": 4096, "dtype": "bf16", "act": "silu", "train": False},
        # a decode batch of an odd size
        {"name": "ffn_serve_100x4096x11008", "op": "gated_ffn", "m": 100, "k": 4096, "f": 11008, "n": 4096, "dtype": "bf16", "act": "silu", "train": False},
        # a training step of a small block: latency of a chain of small products
        {"name": "ffn_train_512x1024x2816", "op": "gated_ffn", "m": 512, "k": 1024, "f": 2816, "n": 1024, "dtype": "bf16", "act": "silu", "train": True},
        # packed sequences of an odd length, odd widths, half precision, the other activation
        {"name": "ffn_train_f16_2047x2050x5461", "op": "gated_ffn", "m": 2047, "k": 2050, "f": 5461, "n": 2050, "dtype": "f16", "act": "gelu", "train": True},
        # a training step of a large block
        {"name": "ffn_train_4096x4096x11008", "op": "gated_ffn", "m": 4096, "k": 4096, "f": 11008, "n": 4096, "dtype": "bf16", "act": "silu", "train": True},
        # a short batch of a small model, half precision, odd vocabulary, most tokens ignored (a prompt before the answer)
        {"name": "loss_f16_200x768x50257", "op": "linear_cross_entropy", "m": 200, "k": 768, "v": 50257, "dtype": "f16", "ignored": 0.7, "train": True},
        # evaluation: the loss of each token, no gradients
        {"name": "loss_eval_2048x2048x32000", "op": "linear_cross_entropy", "m": 2048, "k": 2048, "v": 32000, "dtype": "bf16", "ignored": 0.0, "train": False},
        # a training step over a middle-sized vocabulary, odd number of tokens
        {"name": "loss_4095x4096x32000", "op": "linear_cross_entropy", "m": 4095, "k": 4096, "v": 32000, "dtype": "bf16", "ignored": 0.1, "train": True},
        # a training step over a large one, whose logits alone would take 2 GB in 16 bits
        {"name": "loss_8192x4096x128256", "op": "linear_cross_entropy", "m": 8192, "k": 4096, "v": 128256, "dtype": "bf16", "ignored": 0.1, "train": True},
        # gradients of a small model in float32: latency of many small tensors
        {"name": "clip_f32_2x256x704", "op": "clip_grad_norm", "layers": 2, "hidden": 256, "inner": 704, "dtype": "f32", "clips": True},
        # odd sizes, matrices in half precision beside float32 vectors; the norm is below its limit
        {"name": "clip_f16_6x1023x2729", "op": "clip_grad_norm", "layers": 6, "hidden": 1023, "inner": 2729, "dtype": "f16", "clips": False},
        # gradients of some large layers: memory traffic
        {"name": "clip_bf16_8x4096x11008", "op": "clip_grad_norm", "layers": 8, "hidden": 4096, "inner": 11008, "dtype": "bf16", "clips": True},
    ]


def draw(rng):
    def size(lo, hi, odd=0.4):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if rng.random() < odd:
            return max(lo, min(hi, v))
        step = 64 if v >= 256 else 16 if v >= 32 else 1
        return max(lo, min(hi, v // step * step))

    op = rng.choice(["gated_ffn", "gated_ffn", "linear_cross_entropy", "linear_cross_entropy", "clip_grad_norm"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "gated_ffn":
        train = rng.random() < 0.6
        m, k, f = size(16, 4096) if train else size(1, 1024), size(64, 4096), size(128, 11008)
        return {"op": op, "m": m, "k": k, "f": f, "n": k if rng.random() < 0.8 else size(64, 4096), "dtype": dtype,
                "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]), "train": train}
    if op == "linear_cross_entropy":
        return {"op": op, "m": size(1, 8192), "k": size(64, 4096), "v": size(100, 128256), "dtype": dtype,
                "ignored": rng.choice([0.0, 0.1, 0.7]), "train": rng.random() < 0.7}
    hidden = size(64, 4096)
    return {"op": op, "layers": rng.randint(1, 8), "hidden": hidden, "inner": max(64, hidden * rng.randint(20, 40) // 15) if hidden < 4000 else 11008,
            "dtype": rng.choice(["bf16", "f16", "f32"]) if hidden < 2048 else dtype, "clips": rng.random() < 0.7}


# ---- inputs ------------------------------------------------------------------

def _shapes(case):
    """Gradients of a model: attention's projections, the block's, two vectors a layer, an embedding."""
    h, f = case["hidden"], case["inner"]
    layer = [(h, h), (h, h), (f, h), (f, h), (h, f), (h,), (h,)]
    return layer * case["layers"] + [(4 * h + 1, h)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    op = case["op"]
    if op == "clip_grad_norm":
        grads, squares = [], 0.0
        for i, shape in enumerate(_shapes(case)):
            dtype = TYPES[case["dtype"]] if len(shape) == 2 else torch.float32
            scale = 1e-3 * 1.5 ** (i % 7)  # kinds of weights have gradients of their own size
            t = (normal(*shape) * scale).to(dtype)
            squares += t.numel() * scale * scale
            grads.append(t)
        limit = math.sqrt(squares) * (0.3 if case["clips"] else 3.0)
        return {**case, "grads": grads, "max_norm": limit, "out": [torch.empty_like(t) for t in grads]}
    dtype, train = TYPES[case["dtype"]], case["train"]
    m, k = case["m"], case["k"]
    # rows of the last norm's output: about one in size, a few columns larger than the rest
    x = normal(m, k) * (1 + 3 * (torch.rand((1, k), generator=g, device="cuda") < 0.01))
    if op == "gated_ffn":
        f, n = case["f"], case["n"]
        state = {"x": x, "wg": normal(f, k) / math.sqrt(k), "wu": normal(f, k) / math.sqrt(k), "wd": normal(n, f) / math.sqrt(f)}
        state = {name: t.to(dtype).requires_grad_(train) for name, t in state.items()}
        if train:  # the gradient of a scaled loss
            state["dy"] = (normal(m, n) * torch.exp(0.5 * normal(m, 1)) * 0.1).to(dtype)
        return {**case, **state}
    v = case["v"]
    w = normal(v, k) / math.sqrt(k)
    # a model that has learnt something: the target's row points the way of its token in half of the cases
    target = torch.randint(0, v, (m,), generator=g, device="cuda")
    if m:
        lean = (torch.rand((m, 1), generator=g, device="cuda") < 0.5) * 0.08
        x = x + lean * w[target] * math.sqrt(k)
    target = torch.where(torch.rand((m,), generator=g, device="cuda") < case["ignored"], IGNORE, target)
    target[0] = 0  # one token counts in every batch
    state = {"x": x.to(dtype).requires_grad_(train), "w": w.to(dtype).requires_grad_(train), "target": target}
    if train:  # loss scaling, as half precision needs it
        state["dloss"] = torch.full((), 1024.0, device="cuda")
    return {**case, **state}


# ---- plain forms ---------------------------------------------------------------

def _activation(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return torch.where(g > 0, g, 0), (g > 0).to(g.dtype)


def _plain_ffn(state):
    dtype = TYPES[state["dtype"]]
    x, wg, wu, wd = (state[name].float() for name in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _activation(g, state["act"])
    h = a * u
    y = (h @ wd.t()).to(dtype)
    if not state["train"]:
        return {"y": y}
    dy = state["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return {"y": y, "dx": (dg @ wg + du @ wu).to(dtype), "dwg": (dg.t() @ x).to(dtype), "dwu": (du.t() @ x).to(dtype),
            "dwd": (dy.t() @ h).to(dtype)}


def _plain_loss(state):
    dtype = TYPES[state["dtype"]]
    x, w, target = state["x"].float(), state["w"].float(), state["target"]
    z = x @ w.t()
    most = z.amax(1, keepdim=True)
    e = torch.exp(z - most)
    total = e.sum(1, keepdim=True)
    counts = target != IGNORE
    at = torch.where(counts, target, 0)[:, None]
    each = torch.where(counts, (torch.log(total) + most - z.gather(1, at))[:, 0], 0)
    if not state["train"]:
        return {"loss": each}
    count = counts.sum()
    dz = e / total
    dz.scatter_add_(1, at, torch.full_like(total, -1.0))
    dz *= torch.where(counts, state["dloss"] / count, 0)[:, None]
    return {"loss": each.sum() / count, "dx": (dz @ w).to(dtype), "dw": (dz.t() @ x).to(dtype)}


def _plain_clip(state):
    norm = torch.sqrt(torch.stack([torch.sum(torch.square(t.float())) for t in state["grads"]]).sum())
    scale = torch.clamp(state["max_norm"] / (norm + EPS), max=1.0)
    return {"norm": norm, "clipped": [(t.float() * scale).to(t.dtype) for t in state["grads"]]}


def run(state):
    op = state["op"]
    if not own:
        with torch.no_grad():
            return {"gated_ffn": _plain_ffn, "linear_cross_entropy": _plain_loss, "clip_grad_norm": _plain_clip}[op](state)
    from tiled_software_pipelined_amd import lib
    if op == "clip_grad_norm":
        norm = lib.clip_grad_norm(state["grads"], state["max_norm"], eps=EPS, out=state["out"])
        return {"norm": norm, "clipped": state["out"]}
    if op == "gated_ffn":
        leaves = [state[name] for name in ("x", "wg", "wu", "wd")]
        y = lib.gated_ffn(*leaves, activation=state["act"])
        if not state["train"]:
            return {"y": y}
        return {"y": y.detach(), **dict(zip(("dx", "dwg", "dwu", "dwd"), torch.autograd.grad(y, leaves, state["dy"])))}
    x, w = state["x"], state["w"]
    if not state["train"]:
        return {"loss": lib.linear_cross_entropy(x, w, state["target"], reduction="none")}
    loss = lib.linear_cross_entropy(x, w, state["target"])
    dx, dw = torch.autograd.grad(loss, (x, w), state["dloss"])
    return {"loss": loss.detach(), "dx": dx, "dw": dw}


def work(case):
    op = case["op"]
    if op == "clip_grad_norm":
        counts = [math.prod(s) for s in _shapes(case)]
        sizes = [TYPES[case["dtype"]].itemsize if len(s) == 2 else 4 for s in _shapes(case)]
        return {"bytes": 2 * sum(n * b for n, b in zip(counts, sizes)) + 4, "flops": 3 * sum(counts)}
    m, k = case["m"], case["k"]
    if op == "gated_ffn":
        f, n = case["f"], case["n"]
        flops, data = 2 * m * f * (2 * k + n), 2 * (m * (k + n) + f * (2 * k + n))
        return {"bytes": data * (2 if case["train"] else 1), "flops": flops * (3 if case["train"] else 1)}
    v = case["v"]
    data = 2 * (m + v) * k
    return {"bytes": data * (2 if case["train"] else 1) + 12 * m, "flops": 2 * m * v * k * (3 if case["train"] else 1)}


# ---- the definition in 64 bits -----------------------------------------------

def _exact_ffn(state):
    x, wg, wu, wd = (state[name].detach().to(torch.float64) for name in ("x", "wg", "wu", "wd"))
    gate, up = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
    act = state["act"]
    if act == "silu":
        value = gate * torch.sigmoid(gate)
        slope = torch.sigmoid(gate) + value * torch.sigmoid(-gate)
    elif act == "gelu":
        normal = torch.special.ndtr(gate)
        value, slope = gate * normal, normal + gate * torch.exp(-gate ** 2 / 2) / math.sqrt(2 * math.pi)
    elif act == "gelu_tanh":
        # 1 + tanh(a) = 2 sigmoid(2 a)
        inner = math.sqrt(8 / math.pi) * (gate + 0.044715 * gate ** 3)
        share = torch.sigmoid(inner)
        value = gate * share
        slope = share + gate * share * torch.sigmoid(-inner) * math.sqrt(8 / math.pi) * (1 + 0.134145 * gate ** 2)
    else:
        value, slope = gate.clamp(min=0), torch.heaviside(gate, torch.zeros((), dtype=torch.float64, device=gate.device))
    out = {"y": torch.matmul(value * up, wd.T)}
    if state["train"]:
        dy = state["dy"].to(torch.float64)
        out["dwd"] = torch.matmul(dy.T, value * up)
        back = torch.matmul(dy, wd)
        into_gate, into_up = back * up * slope, back * value
        out["dx"] = torch.matmul(into_gate, wg) + torch.matmul(into_up, wu)
        out["dwg"], out["dwu"] = torch.matmul(into_gate.T, x), torch.matmul(into_up.T, x)
    return out


def _exact_loss(state):
    x, w, target = state["x"].detach().to(torch.float64), state["w"].detach().to(torch.float64), state["target"]
    rows = torch.arange(target.numel(), device=target.device)
    live = rows[target != IGNORE]
    each = torch.zeros(target.shape, dtype=torch.float64, device=target.device)
    dx, dw, total = torch.zeros_like(x), torch.zeros_like(w), live.numel()
    for part in live.split(1024):  # the logits of some tokens at a time
        logits = torch.matmul(x[part], w.T)
        lse = torch.logsumexp(logits, 1)
        here = target[part]
        each[part] = lse - logits[torch.arange(len(part), device=part.device), here]
        if state["train"]:
            share = torch.exp(logits - lse[:, None])
            share[torch.arange(len(part), device=part.device), here] -= 1
            share *= state["dloss"].to(torch.float64) / total
            dx[part] = torch.matmul(share, w)
            dw += torch.matmul(share.T, x[part])
    return {"loss": each.sum() / total, "dx": dx, "dw": dw} if state["train"] else {"loss": each}


def exact(case, seed):
    state = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "gated_ffn":
            return _exact_ffn(state)
        if case["op"] == "linear_cross_entropy":
            return _exact_loss(state)
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in state["grads"]))
        factor = min(1.0, state["max_norm"] / (norm + EPS))
        return {"norm": norm, "clipped": [t.to(torch.float64) * factor for t in state["grads"]]}
