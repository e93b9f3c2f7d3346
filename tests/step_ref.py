"""Plain forms in 64 bits of the feed-forward block, the cross entropy of a
linear layer and gradient clipping, with bounds of what the kernels' roundings
may add up to.

u is half a step of the 16-bit type relative to a value (2^-8 for bfloat16, 2^-11
for float16), TINY half a step below its normal numbers.  A float sum of n products is off by at most n 2^-24 of the
sum of their magnitudes.  First-order terms are added up; 2 % covers the rest.
"""
import math

import torch

F32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
SLACK = 1.02


def act(g, name):
    """act(g), act'(g) and a bound of |act''|."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), 0.5
    if name == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), 0.8
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g), 0.9
    return torch.relu(g), (g > 0).double(), 0.0


def mm(a, b):
    return a @ b.contiguous()


def product(a, b, ea, u, tiny):
    """a @ b in 64 bits and the bound of its float sum, rounded once, where a is off by ea."""
    c, size = mm(a, b), mm(a.abs(), b.abs())
    return c, SLACK * (mm(ea, b.abs()) + (a.shape[1] + 2) * F32 * size + u * c.abs()) + tiny


def ffn(x, wg, wu, wd, name, dy=None):
    """{output: (value, bound)}"""
    t = x.dtype
    u, tiny = U[t], TINY[t]
    x, wg, wu, wd = (v.double() for v in (x, wg, wu, wd))
    K, F, N = x.shape[1], wd.shape[1], wd.shape[0]
    g, up = mm(x, wg.t()), mm(x, wu.t())
    eg, eu = ((K + 2) * F32 * mm(x.abs(), w.abs().t()) for w in (wg, wu))
    a, d, d2 = act(g, name)
    # the activation itself: a few units of float's last place, relative and of g
    # where relu's argument is within its error of zero, either slope
    jump = (g.abs() <= eg).double() * (name == "relu")
    ea = (d.abs() + jump) * eg + 2.0 ** -20 * (a.abs() + 2.0 ** -3 * g.abs() * (d.abs() + 1e-3))
    h = a * up
    eh = u * h.abs() + ea * up.abs() + a.abs() * eu + tiny
    out = {"y": product(h, wd.t(), eh, u, tiny)}
    if dy is None:
        return out
    dy = dy.double()
    dh = mm(dy, wd)
    edh = (N + 2) * F32 * mm(dy.abs(), wd.abs())
    ea = (d.abs() + jump) * eg + d2 * eg * eg + 2.0 ** -20 * (a.abs() + g.abs())
    ed = d2 * eg + jump + 2.0 ** -20 * (1 + g.abs())
    dg, du = dh * up * d, dh * a
    # act'(g) u, act(g) and h are kept, each rounded once from float, and dg and du rounded again
    eb = u * (up * d).abs() + eu * d.abs() + (up.abs() + eu) * ed + tiny
    ea = u * a.abs() + ea + tiny
    edg = u * dg.abs() + edh * ((up * d).abs() + eb) + dh.abs() * eb + tiny
    edu = u * du.abs() + edh * (a.abs() + ea) + dh.abs() * ea + tiny
    c1, b1 = product(dg, wg, edg, u, tiny)
    c2, b2 = product(du, wu, edu, u, tiny)
    out["dx"] = c1 + c2, b1 + b2 + SLACK * F * F32 * (mm(dg.abs(), wg.abs()) + mm(du.abs(), wu.abs()))
    out["dw_gate"] = product(dg.t(), x, edg.t(), u, tiny)
    out["dw_up"] = product(du.t(), x, edu.t(), u, tiny)
    c, b = product(h.t(), dy, eh.t(), u, tiny)
    out["dw_down"] = c.t(), b.t()
    return out


def xent(x, w, target, ignore=-100, reduction="mean", dloss=None, kept=None):
    """{output: (value, bound)}; dloss: one number, or one for each row; kept: whether the powers are kept for
    the backward pass (None: as the library does by itself)."""
    t = x.dtype
    u, tiny = U[t], TINY[t]
    x, w = x.double(), w.double()
    (M, K), V = x.shape, w.shape[0]
    z = mm(x, w.t())
    ez = (K + 2) * F32 * mm(x.abs(), w.abs().t())
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    counts = target != ignore
    at = torch.where(counts, target, 0)[:, None]
    # a lane adds 64 powers, 32 threads a row's pieces, one the 32 sums
    far = (p * (z - z.amax(1, keepdim=True)).abs()).sum(1)
    elog = (100 + V / 2048) * F32 + (8 + far) * 2 * F32 + 4 * F32 * lse.abs()
    elogsum = (p * ez).sum(1) + elog
    each = torch.where(counts, lse - z.gather(1, at)[:, 0], 0)
    eeach = torch.where(counts, elogsum + ez.gather(1, at)[:, 0] + 2 * F32 * each.abs(), 0)
    n = counts.sum().double()
    if reduction == "none":
        out = {"loss": (each, SLACK * eeach)}
    else:
        by = n if reduction == "mean" else 1.0
        out = {"loss": (each.sum() / by, SLACK * (eeach.sum() / by + 2 * F32 * (each.sum() / by).abs()))}
    if dloss is None:
        return out
    dloss = torch.as_tensor(dloss, dtype=torch.float64, device=x.device)
    coef = torch.where(counts, dloss / n if reduction == "mean" else dloss, 0.0)[:, None]
    dz = p.scatter_add(1, at, -torch.ones_like(lse)[:, None]) * coef
    edz = coef.abs() * p * (ez + elogsum[:, None] + (8 + (z - lse[:, None]).abs()) * 2 * F32) + (u + 6 * F32) * dz.abs()
    # dz is rounded after its scale brought the largest factor to 2^14; a
    # probability below float's normal numbers (2^-126) may be taken as zero
    edz = edz + tiny * 2.0 ** -14 * coef.abs().max() + 2.0 ** -126 * coef.abs()
    if kept if kept is not None else K >= 512:
        # p comes as exp(max - lse) times the kept exp(z - max), 2^15 times as much of which was rounded: half a step
        # more, relative or of the type's least (the exponents add up to z - lse's); the target's p is made in float
        edz = edz + (1 - torch.zeros_like(p).scatter_(1, at, 1.0)) * coef.abs() * (p * (u + 16 * F32) + tiny * 2.0 ** -15)
    out["dx"] = product(dz, w, edz, u, tiny)
    out["dw"] = product(dz.t(), x, edz.t(), u, tiny)
    return out


def check(got, want, names=None):
    """Every element of every output inside its bound."""
    for name, (value, bound) in want.items():
        if names is not None and name not in names:
            continue
        g = got[name].detach().double()
        assert g.shape == value.shape, name
        off = (g - value).abs()
        ok = off <= bound
        if not bool(ok.all()):
            i = int((off - bound).argmax())
            raise AssertionError("%s: %d of %d outside; worst off by %.3g, bound %.3g, value %.3g" % (
                name, int((~ok).sum()), ok.numel(), float(off.flatten()[i]), float(bound.flatten()[i]), float(value.flatten()[i])))
