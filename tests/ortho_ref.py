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


def dithered(x, which):
    """To half precision: away from zero where the 13 bits that a float has beyond
    it reach past a threshold of the element's place, else towards zero."""
    C, R, D = {"X": (0xD1B54A33, 0x8CB92BA7, 0xABC98389), "A": (0x9E3779B1, 0x68E31DA4, 0x68E31DA4),
               "B": (0xB5297A4D, 0x1B56C4E9, 0x1B56C4E9)}[which]
    m, n = torch.arange(x.shape[0])[:, None], torch.arange(x.shape[1])
    t = (m * n * C + m * R + n * D & 0xFFFFFFFF) >> 19
    bits = (x.float().view(torch.int32).long() & 0xFFFFFFFF) + t
    bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits)
    v = bits.to(torch.int32).view(torch.float32).double()
    step = torch.exp2(torch.frexp(v)[1].clamp(min=-13) - 11.0)  # 11 bits, and 2^-24 at least
    return torch.trunc(v / step) * step


def emulate(G, steps=5, coefficients=USUAL, eps=1e-7):
    """What the kernels compute of one matrix, before its rounding to bfloat16."""
    X, tall = _start(G, eps)
    X = (X * ONE).float().double()
    small = X.shape[0] <= 64
    for a, b, c in _steps(steps, coefficients):
        hi = dithered(X, "X")
        lo = half(X - hi)
        A = (hi @ hi.t() + (hi @ lo.t() + lo @ hi.t() if small else 0)) / ONE ** 2
        d = A.diagonal().clone()
        A = dithered((A - A.diagonal().diag()) * ONE, "A") / ONE
        square = A @ A
        e = b * d + c * (d * d + square.diagonal())
        B = b * A + c * ((d[:, None] + d) * A + square)
        B = dithered((B - B.diagonal().diag()) * ONE, "B") / ONE
        low = a + e * (small | (square.diagonal() <= d * d))
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


def repeated():
    """Matrices with many equal elements, whose roundings are equal too."""
    ones, eye = torch.ones, torch.eye
    g = torch.Generator().manual_seed(3)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    signs = lambda *s: torch.sign(draw(*s))  # noqa: E731
    hadamard = torch.tensor([[1.0 - 2 * (bin(i & j).count("1") % 2) for j in range(32)] for i in range(32)])
    return {
        "ones 64x1000": ones(64, 1000), "ones 101x118": ones(101, 118), "ones 300x257": ones(300, 257),
        "4 blocks 50x125": torch.kron(eye(4), ones(50, 125)), "4 blocks 100x25": torch.kron(eye(4), ones(100, 25)),
        "4 blocks 26x467": torch.kron(eye(4), ones(26, 467)), "3 blocks 20x70": torch.kron(eye(3), ones(20, 70)), "signs 200x300": signs(200, 1) * signs(1, 300),
        "blocks 4x4 of 40x60": torch.kron(draw(4, 4), ones(40, 60)), "blocks 5x2 of 61x100": torch.kron(draw(5, 2), ones(61, 100)),
        "hadamard 32x8 of 4x9": torch.kron(hadamard[:, :8], ones(4, 9)), "ternary 130x90": torch.sign(draw(130, 90)) * (draw(130, 90) > 0),
        "rows twice": draw(50, 300).repeat_interleave(2, 0), "identity and ones": eye(100) + 0.1,
        "ones 2x2": ones(2, 2), "ones 9x33": ones(9, 33), "4 blocks 1x69": torch.kron(eye(4), ones(1, 69)),
    }
