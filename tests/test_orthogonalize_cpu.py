"""CPU: argument checks of orthogonalize, and its workspace size."""
import ctypes

import pytest
import torch

import ortho_ref

tl = pytest.importorskip("tiled_software_pipelined_amd.lib")
P = ctypes.c_void_p
USUAL = (3.4445, -4.7750, 2.0315)


def call(batch=1, rows=4, cols=6, dtype=0, G=P(256), ldg=None, stride_g=None, O=P(256), ldo=None, stride_o=None, steps=5,
         coef=None, eps=1e-7, ws=P(256), ws_bytes=1 << 40):
    coef = USUAL * max(steps, 1) if coef is None else coef
    ldg, ldo = cols if ldg is None else ldg, cols if ldo is None else ldo
    stride_g, stride_o = rows * ldg if stride_g is None else stride_g, rows * ldo if stride_o is None else stride_o
    c = (ctypes.c_double * len(coef))(*coef) if coef != () else None
    return tl._lib.tgemm_orthogonalize(batch, rows, cols, dtype, G, ldg, stride_g, O, ldo, stride_o, steps, c, eps, ws,
                                       ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(rows=-1), -1), (dict(cols=(1 << 20) + 1), -1), (dict(batch=(1 << 16) + 1), -1),
    (dict(dtype=2), -1), (dict(ldg=2 ** 62), -1), (dict(batch=2, stride_o=2 ** 62), -1), (dict(ldg=5), -1), (dict(ldo=5), -1), (dict(batch=2, stride_g=23), -1),
    (dict(batch=2, stride_o=23), -1), (dict(steps=0), -1), (dict(steps=65), -1), (dict(eps=-1e-9), -1),
    (dict(eps=float("nan")), -1), (dict(coef=()), -2), (dict(steps=1, coef=(float("nan"), 0, 0)), -1),
    (dict(steps=1, coef=(1, float("inf"), 0)), -1), (dict(steps=2, coef=(4, 0, 0) * 2), -1),
    (dict(steps=2, coef=(1, 14.5, 0) * 2), -1), (dict(steps=1, coef=(1, 14.5, 0)), -1),
    (dict(G=None), -2), (dict(O=None), -2), (dict(ws=None), -2), (dict(G=P(258)), -3), (dict(dtype=1, G=P(257)), -3),
    (dict(O=P(257)), -3), (dict(ws=P(128)), -3), (dict(ws_bytes=1000), -1),
])
def test_refuses(kw, code):
    assert call(**kw) == code and tl.last_error()


@pytest.mark.parametrize("kw", [dict(batch=0), dict(rows=0), dict(cols=0)])
def test_nothing_to_do_needs_no_device(kw):
    assert call(**kw, G=None, O=None, ws=None) == 0 and tl.last_error() == ""


def test_workspace():
    w = tl._lib.tgemm_orthogonalize_workspace_bytes
    assert w(0, 4, 4) == w(1, 0, 4) == w(1, 4, 0) == 0
    assert w(1, -1, 4) == w(1, 1 << 21, 4) == w(1 << 17, 4, 4) == -1
    # X as two halves and its transpose twice, A and B, for padded sizes
    assert w(1, 4096, 4096) >= 2 * (4 * 4096 * 4096 + 2 * 4096 * 4096)
    assert w(3, 100, 200) == w(3, 200, 100) >= 3 * 2 * (4 * 100 * 200 + 2 * 100 * 100)


def test_binding_refuses():
    with pytest.raises(ValueError, match="GPU"):
        tl.orthogonalize(torch.zeros(4, 4))


def test_matrices_of_a_tensor():
    t = torch.zeros(4, 3, 10, 8)
    assert tl._matrices(t) == ((12, 10, 8), 8, 80)
    assert tl._matrices(t[0, 0]) == ((1, 10, 8), 8, 80)
    assert tl._matrices(t[..., :5]) == ((12, 10, 5), 8, 80)
    assert tl._matrices(t[:, 1]) == ((4, 10, 8), 8, 240)
    assert tl._matrices(t[:1, :, :1]) == ((3, 1, 8), 8, 80)
    assert tl._matrices(t[:, :2]) is None          # uneven steps
    assert tl._matrices(t.mT) is None              # columns first
    assert tl._matrices(t[0, 0].expand(3, 10, 8)) is None
    assert tl._matrices(t[0, 0, 0].expand(10, 8)) is None
    assert tl._matrices(t[:0])[0] == (0, 10, 8)


def reach(coef):
    """What each step's coefficients can make of singular values in [0, 1], on a
    fine grid: the largest before the last step, and of |b s^2 + c s^4|."""
    import numpy as np
    top, most, poly = 1.0, 1.0, 0.0
    for k, (a, b, c) in enumerate(coef):
        s = np.linspace(0.0, top, 20001)
        q = b * s ** 2 + c * s ** 4
        poly = max(poly, float(abs(q).max()))
        top = float(abs((a + q) * s).max())
        if k + 1 < len(coef):
            most = max(most, top)
        if most > 3.5 or poly > 14.0:
            break
    return most, poly


def test_range_of_coefficients():
    import random
    r = random.Random(5)
    seen = set()
    for _ in range(600):
        n = r.randint(1, 6)
        coef = [(r.uniform(-4, 4), r.choice([0.0, r.uniform(-8, 8)]), r.choice([0.0, r.uniform(-6, 6)])) for _ in range(n)]
        if r.random() < 0.3:
            coef = [USUAL] * n
            coef[r.randrange(n)] = tuple(v * r.uniform(0.8, 1.3) for v in USUAL)
        most, poly = reach(coef)
        if min(abs(most - 3.5) / 3.5, abs(poly - 14.0) / 14.0) < 1e-4:
            continue
        fits = most <= 3.5 and poly <= 14.0
        assert (call(batch=0, steps=n, coef=[v for t in coef for v in t]) == 0) == fits, (coef, most, poly)
        seen.add((fits, n))
    assert len(seen) > 8
    # values whose powers leave the range of double
    for t in ((1e200, 0.0, 0.0), (1e308, -1e308, 1e308), (0.0, 1e308, -1e308), (-1e300, 1e-300, 0.0), (0.0, 0.0, 1e308)):
        assert call(batch=0, steps=4, coef=t * 4) == -1
        assert call(batch=0, steps=4, coef=(1.0, 0.0, 0.0) * 2 + t * 2) == -1
    for t in ((0.0, 0.0, 0.0), (1e-300, 0.0, 0.0), (1.0, 1e-300, -1e-300)):
        assert call(batch=0, steps=4, coef=t * 4) == 0


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on the GPU, where nothing is launched."""
    is_cuda = property(lambda self: True)


def test_steps_that_a_32_bit_count_does_not_hold(monkeypatch):
    # 2^32 + 5 would run as 5 steps, 5 - 2^32 as 5 with coefficients for none
    calls = []
    monkeypatch.setattr(tl, "_call", lambda device, fn, *args: calls.append(args))
    G = torch.zeros(4, 6).as_subclass(OnGpu)
    for steps in (2 ** 32 + 5, 5 - 2 ** 32, -(2 ** 40), 2 ** 63, 0, 65, -1, 2.5, float("nan")):
        with pytest.raises(tl.TgemmError):
            tl.orthogonalize(G, steps=steps)
    assert not calls
    for steps, co, want in ((5, USUAL, USUAL * 5), (1, [USUAL], USUAL), (3, [(1, 0, 0)] * 3, (1, 0, 0) * 3),
                            (3, (1, 0, 0), (1, 0, 0) * 3), (2.0, USUAL, USUAL * 2)):
        tl.orthogonalize(G, steps=steps, coefficients=co)
        assert calls[-1][10] == steps and tuple(calls[-1][11]) == tuple(want)


def emulated_error(G):
    want = ortho_ref.exact(G)
    return float((ortho_ref.emulate(G) - want).norm() / want.norm())


# what the header states of the error before the result's own rounding, and the
# tests on the GPU rest on: 1.3e-3 of the norm for random matrices, 4.5e-3 for any
@pytest.mark.parametrize("m,n", [(2, 3), (16, 16), (31, 33), (63, 200), (65, 64), (100, 1000), (128, 384), (257, 129)])
def test_emulated_error_of_random_matrices(m, n):
    for seed in range(3):
        G = torch.randn((m, n), generator=torch.Generator().manual_seed(m + n + seed))
        assert emulated_error(G) <= 1.3e-3
        assert emulated_error(G.bfloat16()) <= 1.3e-3


@pytest.mark.parametrize("m,n", [(2, 4), (3, 21), (5, 193), (17, 4), (40, 1000), (64, 65), (65, 70), (100, 128), (70, 1000),
                                 (200, 90), (129, 300)])
def test_emulated_error_of_low_rank(m, n):
    for kind, G in ortho_ref.low_rank(m, n).items():
        assert emulated_error(G) <= 4.5e-3, kind


@pytest.mark.parametrize("kind", sorted(ortho_ref.repeated()))
def test_emulated_error_of_repeated_elements(kind):
    assert emulated_error(ortho_ref.repeated()[kind]) <= 4.5e-3


def test_launches_that_no_grid_holds_are_refused():
    w = tl._lib.tgemm_orthogonalize_workspace_bytes
    # 2^16 matrices of 256 pieces for the norm: 2^32 threads
    for batch, rows, cols in ((1 << 16, 256, 1025), (1 << 16, 1 << 16, 1), (1 << 16, 1 << 20, 1 << 20)):
        assert w(batch, rows, cols) == -1
        assert call(batch=batch, rows=rows, cols=cols, ws_bytes=1 << 62) == -1 and tl.last_error()
    assert w((1 << 16) - 1, 256, 1025) > 0 and w(1 << 16, 255, 1025) > 0
