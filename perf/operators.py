"""Workloads of the 8-bit floating point products and of the orthogonalised update.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and, with ``own`` set, through the library's entry points:

  quantize_fp8   X -> 8-bit values with a power-of-two scale for each 128 of a
                 row (or each 128 x 128 block), and the same of X transposed
  gemm_fp8       C = A B^T of two quantised operands, C in bfloat16
  linear_fp8     y = x w^T with both operands quantised, and its gradients
  orthogonalize  Newton-Schulz products that bring a matrix's singular values
                 near one (the update of the Muon optimiser)

A quantised operand is the pair (Q, S): Q (rows, cols) in an 8-bit float type,
S (ceil(cols / 128), rows) in float8_e8m0fnu; element (r, c) stands for
Q[r, c] * S[c // 128, r].
"""
import math

import torch

own = False

BLOCK = 128
#: the largest value of each 8-bit type: mantissa and exponent of its highest binade
TOP = {"e4m3": (1.75, 8), "e5m2": (1.75, 15)}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
IN = {"bf16": torch.bfloat16, "f32": torch.float32}
#: x <- a x + (b A + c A^2) x with A = x x^T, the usual five steps
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5


def listed():
    return [
        # activations of a decode batch, once per layer: latency
        {"name": "quantize_rows_16x4096", "op": "quantize_fp8", "rows": 16, "cols": 4096, "dtype": "bf16", "fmt": "e4m3", "block": "row", "transpose": False},
        # activations of a training step: the rows feed the forward product, the transposed image the weight gradient
        {"name": "quantize_both_8192x4096", "op": "quantize_fp8", "rows": 8192, "cols": 4096, "dtype": "bf16", "fmt": "e4m3", "block": "row", "transpose": True},
        # a float32 master weight with odd sizes, one scale for each square block
        {"name": "quantize_square_4095x4104", "op": "quantize_fp8", "rows": 4095, "cols": 4104, "dtype": "f32", "fmt": "e4m3", "block": "square", "transpose": True},
        # one token against a weight: bound by one read of the weight
        {"name": "gemm_1x4096x4096", "op": "gemm_fp8", "m": 1, "n": 4096, "k": 4096, "fmt_a": "e4m3", "fmt_b": "e4m3"},
        # a decode batch of an odd size
        {"name": "gemm_100x4096x4096", "op": "gemm_fp8", "m": 100, "n": 4096, "k": 4096, "fmt_a": "e4m3", "fmt_b": "e4m3"},
        # the square product the library's other types are measured on
        {"name": "gemm_4096x4096x4096", "op": "gemm_fp8", "m": 4096, "n": 4096, "k": 4096, "fmt_a": "e4m3", "fmt_b": "e4m3"},
        # the ragged one, a gradient in e5m2 against a weight
        {"name": "gemm_e5m2_4095x4097x4104", "op": "gemm_fp8", "m": 4095, "n": 4097, "k": 4104, "fmt_a": "e5m2", "fmt_b": "e4m3"},
        # a training step of a small layer: forward, gradient of the input and of the weight
        {"name": "linear_512x1024x1024", "op": "linear_fp8", "m": 512, "n": 1024, "k": 1024},
        # the same of a large one
        {"name": "linear_4096x4096x4096", "op": "linear_fp8", "m": 4096, "n": 4096, "k": 4096},
        # the update of a small weight matrix: latency of a chain of products
        {"name": "orthogonalize_256x256", "op": "orthogonalize", "batch": 1, "rows": 256, "cols": 256, "dtype": "bf16"},
        # a stack of projections with more rows than columns, odd sizes, float32 momentum
        {"name": "orthogonalize_4x2050x513", "op": "orthogonalize", "batch": 4, "rows": 2050, "cols": 513, "dtype": "f32"},
        # a large weight matrix
        {"name": "orthogonalize_4096x4096", "op": "orthogonalize", "batch": 1, "rows": 4096, "cols": 4096, "dtype": "bf16"},
    ]


def draw(rng):
    def size(lo, hi, odd=0.4):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if rng.random() < odd:
            return max(lo, min(hi, v))
        step = 64 if v >= 256 else 16 if v >= 32 else 1
        return max(lo, min(hi, v // step * step))

    op = rng.choice(["quantize_fp8", "gemm_fp8", "gemm_fp8", "linear_fp8", "orthogonalize", "orthogonalize"])
    if op == "quantize_fp8":
        rows, cols = size(1, 8192), size(64, 8192)
        while rows * cols > 1 << 25:
            rows //= 2
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "block": rng.choice(["row", "row", "square"]), "transpose": rng.random() < 0.6}
    if op == "gemm_fp8":
        m, n, k = size(1, 8192), size(16, 8192), size(64, 8192)
        while m * n * k > 4096 ** 3:
            m, n = max(1, m // 2), n * 3 // 4
        return {"op": op, "m": m, "n": n, "k": k, "fmt_a": rng.choice(["e4m3", "e4m3", "e5m2"]), "fmt_b": rng.choice(["e4m3", "e4m3", "e4m3", "e5m2"])}
    if op == "linear_fp8":
        return {"op": op, "m": size(1, 4096), "n": size(32, 4096), "k": size(64, 4096)}
    rows, cols = size(16, 4096), size(16, 4096)
    most = max(1, min(8, (1 << 23) // (rows * cols)))
    return {"op": op, "batch": rng.randint(1, most), "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"])}


# ---- inputs ------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, g):
    """Rows of different size, a few columns far larger than the rest, one row in 64 all zero (padding)."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn((rows, 1), generator=g, device="cuda"))
    x *= 1 + 30 * (torch.rand((1, cols), generator=g, device="cuda") < 0.005)
    if rows > 1:
        x *= torch.rand((rows, 1), generator=g, device="cuda") >= 1 / 64
    return x


def _weight(rows, cols, g):
    return torch.randn((rows, cols), generator=g, device="cuda") * 0.02


def _gradient(rows, cols, g):
    return torch.randn((rows, cols), generator=g, device="cuda") * torch.exp(1.5 * torch.randn((rows, 1), generator=g, device="cuda")) * 1e-5


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "quantize_fp8":
        make = _weight if case["block"] == "square" else _activations
        return {**case, "x": make(case["rows"], case["cols"], g).to(IN[case["dtype"]])}
    if op == "gemm_fp8":
        a = (_gradient if case["fmt_a"] == "e5m2" else _activations)(case["m"], case["k"], g).bfloat16()
        b = (_gradient if case["fmt_b"] == "e5m2" else _weight)(case["n"], case["k"], g).bfloat16()
        qa, sa = _quantize(a, case["fmt_a"], "row")
        qb, sb = _quantize(b, case["fmt_b"], "row" if case["fmt_b"] == "e5m2" else "square")
        return {**case, "a": qa, "sa": sa, "b": qb, "sb": sb}
    if op == "linear_fp8":
        x = _activations(case["m"], case["k"], g).bfloat16().requires_grad_()
        w = _weight(case["n"], case["k"], g).bfloat16().requires_grad_()
        return {**case, "x": x, "w": w, "dy": _gradient(case["m"], case["n"], g).bfloat16()}
    # a momentum of gradients: a sum of outer products with decaying weights, over a floor of noise
    b, r, c = case["batch"], case["rows"], case["cols"]
    rank = max(4, min(r, c) // 4)
    u = torch.randn((b, r, rank), generator=g, device="cuda") / torch.arange(1, rank + 1, device="cuda").sqrt()
    v = torch.randn((b, rank, c), generator=g, device="cuda")
    x = (u @ v + 0.5 * torch.randn((b, r, c), generator=g, device="cuda")) * 1e-3
    return {**case, "x": (x if b > 1 else x[0]).to(IN[case["dtype"]])}


# ---- plain forms ---------------------------------------------------------------

def _blocks(v, size):
    """v's last axis in groups of `size`, filled up with zeros."""
    short = -v.shape[-1] % size
    return torch.nn.functional.pad(v, (0, short)).unflatten(-1, (-1, size))


def _exponent(amax, fmt):
    """The least e with amax <= largest value * 2^e, 0 for a block of zeros."""
    mant, top = TOP[fmt]
    m, e = torch.frexp(amax)  # amax = 2 m * 2^(e - 1), 1 <= 2 m < 2
    e = e - 1 - top + (2 * m > mant)
    return torch.where(amax > 0, e.clamp(-127, 127), 0).to(torch.int32)


def _power(e):
    """2^e in 32 bits, from its bits: exp2 need not be exact."""
    return ((e + 127) << 23).view(torch.float32)


def _quantize(x, fmt, block):
    """(Q, S) of the rows of x."""
    rows, cols = x.shape
    v = _blocks(x.float(), BLOCK)
    amax = v.abs().amax(-1)
    if block == "square":
        amax = _blocks(amax.t(), BLOCK).amax(-1).repeat_interleave(BLOCK, -1)[:, :rows].t()
    e = _exponent(amax, fmt)
    half = torch.div(e, 2, rounding_mode="floor")  # 2^-e as two factors that are normal numbers
    q = v * _power(-half)[..., None] * _power(half - e)[..., None]
    q = q.flatten(-2)[:, :cols].to(FP8[fmt])
    s = torch.zeros((e.shape[1], -(-rows // 16) * 16), dtype=torch.uint8, device=x.device)
    s[:, :rows] = (e + 127).t().to(torch.uint8)
    return q.contiguous(), s.view(torch.float8_e8m0fnu)[:, :rows]


def _values(q, s):
    """What (Q, S) stands for, in 32 bits."""
    return q.float() * s.float().t().repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def _orthogonalize(x):
    a, b, c = COEFFICIENTS
    v = x.float()
    tall = v.shape[-2] > v.shape[-1]
    v = v.mT if tall else v
    v = v / (torch.sqrt(torch.sum(v * v, (-2, -1), keepdim=True)) + 1e-7)
    for _ in range(STEPS):
        p = v @ v.mT
        v = a * v + (b * p + c * (p @ p)) @ v
    return (v.mT if tall else v).bfloat16().contiguous()


def run(state):
    op = state["op"]
    if op == "quantize_fp8":
        if own:
            from tiled_software_pipelined_amd import lib
            got = lib.quantize_fp8(state["x"], dtype=FP8[state["fmt"]], block=state["block"], transpose=state["transpose"])
        else:
            got = _quantize(state["x"], state["fmt"], state["block"])
            if state["transpose"]:
                got += _quantize(state["x"].t(), state["fmt"], state["block"])
        return dict(zip(("q", "s", "qt", "st"), got))
    if op == "gemm_fp8":
        if own:
            from tiled_software_pipelined_amd import lib
            return lib.gemm_fp8(state["a"], state["sa"], state["b"], state["sb"])
        return (_values(state["a"], state["sa"]) @ _values(state["b"], state["sb"]).t()).bfloat16()
    if op == "linear_fp8":
        x, w, dy = state["x"], state["w"], state["dy"]
        if own:
            from tiled_software_pipelined_amd import lib
            y = lib.linear_fp8(x, w)
            dx, dw = torch.autograd.grad(y, (x, w), dy)
            return {"y": y.detach(), "dx": dx, "dw": dw}
        with torch.no_grad():
            wv = _values(*_quantize(w, "e4m3", "square"))
            y = _values(*_quantize(x, "e4m3", "row")) @ wv.t()
            dx = _values(*_quantize(dy, "e4m3", "row")) @ wv
            dw = _values(*_quantize(dy.t(), "e4m3", "row")) @ _values(*_quantize(x.t(), "e4m3", "row")).t()
            return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw.bfloat16()}
    if own:
        from tiled_software_pipelined_amd import lib
        return lib.orthogonalize(state["x"], steps=STEPS, coefficients=COEFFICIENTS)
    return _orthogonalize(state["x"])


def work(case):
    op = case["op"]
    if op == "quantize_fp8":
        n = case["rows"] * case["cols"]
        images = 2 if case["transpose"] else 1
        return {"bytes": n * (IN[case["dtype"]].itemsize + images) + images * n / BLOCK, "flops": 2 * images * n}
    if op == "orthogonalize":
        m, n = sorted((case["rows"], case["cols"]))
        # two of the three products of a step are symmetric: half of each is enough
        return {"bytes": case["batch"] * m * n * (IN[case["dtype"]].itemsize + 2), "flops": case["batch"] * STEPS * (3 * m * m * n + m ** 3)}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "gemm_fp8":
        return {"bytes": (m + n) * k * (1 + 1 / BLOCK) + 2 * m * n, "flops": 2 * m * n * k}
    return {"bytes": 4 * (m * k + n * k + m * n), "flops": 6 * m * n * k}


# ---- the definition in 64 bits -----------------------------------------------

def _two_to(e):
    """2^e in 64 bits for whole numbers e, exactly."""
    return ((e.to(torch.int64) + 1023) * 2 ** 52).view(torch.float64)


def _grid(y, fmt):
    """y rounded to the nearest value of the 8-bit type, ties to even."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** (low - 20)))).clamp(min=low)
    e = torch.where(_two_to(e + 1) <= y.abs(), e + 1, e)
    step = _two_to(e - bits)
    return torch.round(y / step) * step


def _exact_quantize(x, fmt, block):
    """(values of Q, values of S, what they stand for) in 64 bits."""
    rows, cols = x.shape
    groups = -(-cols // BLOCK)
    v = torch.zeros((rows, groups * BLOCK), dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    most = v.reshape(rows, groups, BLOCK).abs().max(2).values
    if block == "square":
        for r in range(0, rows, BLOCK):
            most[r:r + BLOCK] = most[r:r + BLOCK].max(0, keepdim=True).values
    top = TOP[fmt][0] * 2.0 ** TOP[fmt][1]
    e = torch.ceil(torch.log2(most.clamp(min=2.0 ** -200) / top))
    e = torch.where(_two_to(e - 1) * top >= most, e - 1, e)  # where the logarithm was rounded up
    e = torch.where(_two_to(e) * top < most, e + 1, e).clamp(-127, 127)
    s = torch.where(most > 0, _two_to(e), torch.ones_like(e))
    wide = torch.repeat_interleave(s, BLOCK, dim=1)[:, :cols]
    q = _grid(v[:, :cols] / wide, fmt)
    return q, s.t(), q * wide


def _exact_values(q, s):
    e = s.view(torch.uint8).to(torch.float64) - 127
    v = q.to(torch.float64)
    for kb in range(e.shape[0]):
        v[:, kb * BLOCK:(kb + 1) * BLOCK] *= _two_to(e[kb])[:, None]
    return v


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize_fp8":
        x = state["x"]
        out = dict(zip(("q", "s"), _exact_quantize(x, case["fmt"], case["block"])))
        if case["transpose"]:
            out.update(zip(("qt", "st"), _exact_quantize(x.t(), case["fmt"], case["block"])))
        return out
    if op == "gemm_fp8":
        return torch.matmul(_exact_values(state["a"], state["sa"]), _exact_values(state["b"], state["sb"]).t())
    if op == "linear_fp8":
        x, w, dy = (state[k].detach() for k in ("x", "w", "dy"))
        wv = _exact_quantize(w, "e4m3", "square")[2]
        xv, xt = _exact_quantize(x, "e4m3", "row")[2], _exact_quantize(x.t(), "e4m3", "row")[2]
        gv, gt = _exact_quantize(dy, "e4m3", "row")[2], _exact_quantize(dy.t(), "e4m3", "row")[2]
        return {"y": torch.matmul(xv, wv.t()), "dx": torch.matmul(gv, wv), "dw": torch.matmul(gt, xt.t())}
    found = []
    for one in state["x"].reshape(case["batch"], case["rows"], case["cols"]):
        v = one.to(torch.float64)
        v = v / (torch.linalg.vector_norm(v) + 1e-7)
        wide = case["rows"] <= case["cols"]
        a, b, c = COEFFICIENTS
        for _ in range(STEPS):  # the Gram matrix on the shorter side
            gram = torch.matmul(v, v.t()) if wide else torch.matmul(v.t(), v)
            poly = b * gram + c * torch.matmul(gram, gram)
            v = a * v + (torch.matmul(poly, v) if wide else torch.matmul(v, poly))
        found.append(v)
    return torch.stack(found).reshape(state["x"].shape)
