"""orthogonalize on the CPU: the iteration in 64 bits, and the same with every
rounding that the kernels make (sums in 64 bits, where theirs are in 32)."""
import torch

USUAL = (3.4445, -4.7750, 2.0315)
ONE = 4096.0  # what stands for 1 in the kernels' matrices


def _steps(steps, coefficients):
    return list(coefficients) if hasattr(coefficients[0], "__len__") else [coefficients] * steps


def _start(G, eps):
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.t().contiguous() if tall else X
    return X / (X.square().sum().sqrt() + eps), tall


def exact(G, steps=5, coefficients=USUAL, eps=1e-7):
    """The definition in 64 bits, of one matrix."""
    X, tall = _start(G, eps)
    for a, b, c in _steps(steps, coefficients):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if tall else X


def half(x):
    """To float, then to half precision, to nearest."""
    return x.float().half().double()


def emulate(G, steps=5, coefficients=USUAL, eps=1e-7):
    """What the kernels compute of one matrix, before its rounding to bfloat16."""
    X, tall = _start(G, eps)
    X = (X * ONE).float().double()
    small = X.shape[0] <= 64
    for a, b, c in _steps(steps, coefficients):
        hi = half(X)
        lo = half(X - hi)
        A = (hi @ hi.t() + (hi @ lo.t() + lo @ hi.t() if small else 0)) / ONE ** 2
        d = A.diagonal().clone()
        A = half((A - A.diagonal().diag()) * ONE) / ONE
        square = A @ A
        e = b * d + c * (d * d + square.diagonal())
        B = b * A + c * ((d[:, None] + d) * A + square)
        B = half((B - B.diagonal().diag()) * ONE) / ONE
        low = a + e * (small | (square.diagonal() <= 1.5 * d * d))
        X = ((a + e)[:, None] * hi + low[:, None] * lo + B @ (hi + lo if small else hi)).float().double()
    X = X / ONE
    return X.t() if tall else X


def low_rank(m, n):
    """Matrices of rank one, two and about that, m x n."""
    g = torch.Generator().manual_seed(m * 1000 + n)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"one": draw(m, 1) * draw(1, n), "two": draw(m, 2) @ draw(2, n), "equal rows": draw(1, n).expand(m, n),
            "rows and a column": draw(1, n) + 0.01 * draw(m, 1), "ones and noise": 1 + 1e-3 * draw(m, n),
            "ramp": torch.arange(float(m))[:, None] + torch.arange(1.0, n + 1)}
