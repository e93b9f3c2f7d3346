"""CPU: argument checks of the 8-bit block-scaled operators, their choice of
kernel, and the reference's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_ref as ref

tl = pytest.importorskip("tiled_software_pipelined_amd.lib")
P = ctypes.c_void_p


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_reference_rounding_matches_the_type(fmt, dtype):
    bits = torch.arange(256, dtype=torch.uint8).view(dtype).double().numpy()
    t = ref.TABLE[fmt]
    assert np.array_equal(bits[: len(t)], t) and np.array_equal(bits[128:128 + len(t)], -t)
    g = np.random.default_rng(1)
    y = np.concatenate([g.standard_normal(4000) * 10.0 ** g.integers(-5, 2, 4000), (t[:-1] + t[1:]) / 2, -t, t])
    y = np.clip(y, -t[-1], t[-1]).astype(np.float32)
    got = torch.from_numpy(y).to(dtype).double().numpy()
    assert np.array_equal(ref.round8(y.astype(np.float64), fmt), got)


def test_reference_scales():
    x = np.zeros((3, 130))
    x[0, 0], x[0, 129], x[1, 5] = 448.0, 448.5, 2.0 ** -140
    _, e = ref.quantize(x, "e4m3")
    assert e.shape == (2, 3) and e[0, 0] == 0 and e[1, 0] == 1 and e[0, 1] == -127 and (e[:, 2] == 0).all()
    _, e = ref.quantize(np.array([[57344.0]]), "e5m2")
    assert e[0, 0] == 0


def q(rows, cols, dtype=0, X=P(64), ldx=None, fmt=0, block=0, Q=P(64), ldq=None, S=P(64), lds=None, Qt=None, ldqt=0,
      St=None, ldst=0):
    return tl._lib.tgemm_fp8_quantize(rows, cols, dtype, X, cols if ldx is None else ldx, fmt, block, Q,
                                      cols if ldq is None else ldq, S, rows if lds is None else lds, Qt, ldqt, St,
                                      ldst, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1, cols=4), -1), (dict(rows=4, cols=2 ** 31), -1), (dict(rows=4, cols=4, dtype=2), -1),
    (dict(rows=4, cols=4, dtype=9), -1), (dict(rows=4, cols=4, fmt=2), -1), (dict(rows=4, cols=4, block=2), -1),
    (dict(rows=4, cols=4, ldx=3), -1), (dict(rows=4, cols=4, ldq=3), -1), (dict(rows=4, cols=4, lds=3), -1),
    (dict(rows=4, cols=4, Qt=P(64), St=P(64), ldqt=3, ldst=4), -1),
    (dict(rows=4, cols=4, Qt=P(64), St=P(64), ldqt=4, ldst=3), -1),
    (dict(rows=4, cols=4, ldx=2 ** 41), -1), (dict(rows=4, cols=4, lds=2 ** 62), -1),
    (dict(rows=4, cols=4, X=None), -2), (dict(rows=4, cols=4, Q=None), -2), (dict(rows=4, cols=4, S=None), -2),
    (dict(rows=4, cols=4, Qt=P(64), ldqt=4, ldst=4), -2), (dict(rows=4, cols=4, St=P(64), ldqt=4, ldst=4), -2),
    (dict(rows=4, cols=4, X=P(66)), -3), (dict(rows=4, cols=4, dtype=1, X=P(65)), -3),
])
def test_quantize_refuses(kw, code):
    assert q(**kw) == code and tl.last_error()


@pytest.mark.parametrize("rows,cols", [(0, 4), (4, 0), (0, 0)])
def test_quantize_of_nothing_needs_no_device(rows, cols):
    assert q(rows, cols, X=None, Q=None, S=None) == 0 and tl.last_error() == ""


def g(M, N, K, fa=0, A=P(64), lda=None, SA=P(64), ldsa=None, fb=0, B=P(64), ldb=None, SB=P(64), ldsb=None, C=P(64),
      ldc=None):
    d = lambda v, w: w if v is None else v  # noqa: E731
    return tl._lib.tgemm_fp8_gemm(M, N, K, fa, A, d(lda, K), SA, d(ldsa, (M + 3) // 4 * 4), fb, B, d(ldb, K), SB,
                                  d(ldsb, (N + 3) // 4 * 4), C, d(ldc, N), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1, N=4, K=4), -1), (dict(M=4, N=2 ** 31, K=4), -1), (dict(M=4, N=4, K=2 ** 31 - 1), -1),
    (dict(M=4, N=4, K=4, fa=2), -1), (dict(M=4, N=4, K=4, fb=-1), -1), (dict(M=4, N=4, K=4, lda=3), -1),
    (dict(M=4, N=4, K=4, ldb=3), -1), (dict(M=8, N=4, K=4, ldsa=4), -1), (dict(M=4, N=8, K=4, ldsb=4), -1),
    (dict(M=4, N=4, K=4, lda=2 ** 62), -1), (dict(M=4, N=4, K=4, ldc=2 ** 41), -1),
    (dict(M=4, N=4, K=4, ldc=3), -1), (dict(M=4, N=4, K=4, A=None), -2), (dict(M=4, N=4, K=4, B=None), -2),
    (dict(M=4, N=4, K=4, SA=None), -2), (dict(M=4, N=4, K=4, SB=None), -2), (dict(M=4, N=4, K=4, C=None), -2),
    (dict(M=4, N=4, K=0, C=None), -2), (dict(M=4, N=4, K=4, C=P(65)), -3), (dict(M=4, N=4, K=4, ldsa=6), -3),
    (dict(M=4, N=4, K=4, ldsb=7), -3), (dict(M=4, N=4, K=4, SA=P(66)), -3), (dict(M=4, N=4, K=4, SB=P(65)), -3),
])
def test_gemm_refuses(kw, code):
    assert g(**kw) == code and tl.last_error()


@pytest.mark.parametrize("M,N", [(0, 4), (4, 0)])
def test_gemm_of_nothing_needs_no_device(M, N):
    assert g(M, N, 4, A=None, B=None, SA=None, SB=None, C=None) == 0 and tl.last_error() == ""


def test_kernel_choice():
    k = tl.gemm_fp8_kernel
    assert k(0, 4, 4) == k(4, 0, 4) == k(-1, 4, 4) == k(4, 4, 4, piece=1) == k(4, 4, 4, piece=-1) == ""
    name = lambda *a, **kw: k(*a, **kw).split("_")[0]  # noqa: E731
    assert [name(m, 4096, 4096) for m in (1, 16, 17, 32)] == ["rows16", "rows16", "rows32", "rows32"]
    assert [name(4096, n, 4096) for n in (1, 16, 17, 32)] == ["rows16", "rows16", "rows32", "rows32"]
    assert name(100, 4096, 4096) == name(512, 4096, 4096) == "t64x64x128"
    assert k(1024, 4096, 4096) == "t128x128x128_w2x4_s4_slice" and k(2048, 4096, 4096) == "t128x128x128_w2x2_s2_slice"
    assert name(4096, 4096, 4096) == "t256x256x128"
    # whole tiles, then the last columns or rows
    for m, n in ((4095, 4097), (4097, 4096), (4100, 4096)):
        assert name(m, n, 4104) == "t256x256x128" and name(m, n, 4104, piece=1).startswith("rows")
    # rows too long for a tiled kernel's 32-bit offsets
    assert name(4096, 4096, 64, lda=2 ** 31).startswith("rows") and name(4096, 4096, 64, ldb=2 ** 31).startswith("rows")


def test_binding_refuses_before_any_launch():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        tl.quantize_fp8(x)
    with pytest.raises(TypeError, match="8-bit"):
        tl.quantize_fp8(x, dtype=torch.int8)
    with pytest.raises(ValueError, match="block"):
        tl.quantize_fp8(x, block="column")
    e = torch.zeros(4, 128).to(torch.float8_e4m3fn)
    s = torch.zeros(1, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        tl.gemm_fp8(e, s, e, s)
    with pytest.raises(ValueError, match="GPU"):
        tl.linear_fp8(x, x)
    with pytest.raises(TypeError, match="8-bit"):
        tl.linear_fp8(x, x, grad_dtype=torch.float16)


def test_scale_table_checks():
    dev = torch.device("cpu")
    s = torch.zeros(2, 16, dtype=torch.uint8)
    assert tl._scales(s, 16, 256, dev, "S") == 16
    assert tl._scales(s[:, :5], 5, 256, dev, "S") == 16
    assert tl._scales(s[:1, :5], 5, 7, dev, "S") == 8
    assert tl._scales(s.view(torch.float8_e8m0fnu), 16, 256, dev, "S") == 16
    assert tl._scales(s[:0], 16, 0, dev, "S") == 16
    for bad, rows, cols in ((s, 16, 128), (s, 15, 256), (s[:, 1:5], 4, 256), (torch.zeros(2, 6, dtype=torch.uint8), 6, 256),
                            (torch.zeros(2, 5, dtype=torch.uint8), 5, 256), (s[:, ::2], 8, 256),
                            (torch.zeros(1, 5, dtype=torch.uint8), 5, 100),
                            (torch.zeros(1, 16, dtype=torch.uint8).expand(2, 16), 16, 256)):
        with pytest.raises(ValueError):
            tl._scales(bad, rows, cols, dev, "S")
    with pytest.raises(TypeError):
        tl._scales(s.float(), 16, 256, dev, "S")


def lin(forward, M=4, N=6, K=8, **kw):
    a = dict(xd=1, x=P(256), ldx=K, wd=1, w=P(256), ldw=K, y=P(256), ldy=N, keep=3, saved=P(256), scratch=P(256), gd=1,
             g=P(256), ldg=N, fmt=0, dx=P(256), lddx=K, dw=P(256), lddw=K)
    a.update(kw)
    if forward:
        return tl._lib.tgemm_fp8_linear_forward(M, N, K, a["xd"], a["x"], a["ldx"], a["wd"], a["w"], a["ldw"], a["y"], a["ldy"],
                                                a["keep"], a["saved"], a["scratch"], None)
    return tl._lib.tgemm_fp8_linear_backward(M, N, K, a["gd"], a["g"], a["ldg"], a["fmt"], a["keep"], a["saved"], a["dx"],
                                             a["lddx"], a["dw"], a["lddw"], a["scratch"], None)


@pytest.mark.parametrize("forward,kw,code", [
    (True, dict(M=-1), -1), (True, dict(N=2 ** 31), -1), (True, dict(M=2 ** 30, N=2 ** 30), -1),
    (True, dict(ldx=2 ** 41), -1), (True, dict(keep=4), -1), (True, dict(xd=2), -1),
    (True, dict(wd=5), -1), (True, dict(ldx=7), -1), (True, dict(ldw=7), -1), (True, dict(ldy=5), -1),
    (True, dict(x=None), -2), (True, dict(w=None), -2), (True, dict(y=None), -2), (True, dict(saved=None), -2),
    (True, dict(scratch=None), -2), (True, dict(x=P(257)), -3), (True, dict(xd=0, x=P(258)), -3), (True, dict(y=P(257)), -3),
    (True, dict(saved=P(16)), -3), (True, dict(scratch=P(16)), -3),
    (False, dict(M=-1), -1), (False, dict(keep=-1), -1), (False, dict(gd=2), -1), (False, dict(fmt=2), -1),
    (False, dict(ldg=5), -1), (False, dict(lddx=7), -1), (False, dict(lddw=7), -1), (False, dict(g=None), -2),
    (False, dict(dx=None), -2), (False, dict(dw=None), -2), (False, dict(saved=None), -2), (False, dict(scratch=None), -2),
    (False, dict(g=P(257)), -3), (False, dict(saved=P(16)), -3), (False, dict(scratch=P(16)), -3),
])
def test_linear_refuses(forward, kw, code):
    assert lin(forward, **kw) == code and tl.last_error()


def test_linear_bytes():
    b = tl._linear_bytes
    assert b(0, 0, 0, 3) == (1, 1, 1)
    # an image: one byte an element, rows of whole 128 bytes; its table: rows of 16;
    # each on a 256-byte boundary
    def image(rows, cols):
        up = lambda v, n: -(-v // n) * n  # noqa: E731
        return up(rows * up(cols, 128), 256) + up(up(rows, 16) * -(-cols // 128), 256)
    M, N, K = 100, 200, 300
    assert b(M, N, K, 0) == (1, image(M, K) + image(N, K), image(M, N))
    assert b(M, N, K, 3) == (image(K, N) + image(K, M), image(M, K) + image(N, K), image(M, N) + image(N, M))
    assert b(M, N, K, 1)[0] == image(K, N) and b(M, N, K, 2)[0] == image(K, M)
    assert tl._lib.tgemm_fp8_linear_bytes(1, 1, 1, 0, None) == -2
    with pytest.raises(tl.TgemmError):
        b(1, 1, 1, 4)
    assert lin(True, M=0, N=0, K=0, keep=0, saved=None, scratch=None, x=None, w=None, y=None) == 0
    assert lin(False, M=0, N=0, K=0, keep=0, saved=None, scratch=None, g=None) == 0


def test_package_offers_the_operators():
    import tiled_software_pipelined_amd as package
    for name in package.__all__:
        assert getattr(package, name) is getattr(tl, name)
    assert not hasattr(package, "no_such_name")


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on the GPU, where nothing is launched."""
    is_cuda = property(lambda self: True)


@pytest.mark.parametrize("dual", ["x", "w", "both"])
@pytest.mark.parametrize("grad", [True, False])
def test_linear_refuses_forward_mode(monkeypatch, dual, grad):
    # a dual tensor has no requires_grad: its tangent must not be dropped in silence
    monkeypatch.setattr(tl, "_linear_forward",
                        lambda x, w, keep: (torch.zeros(x.shape[0], w.shape[0]), torch.zeros(1)))
    x, w = torch.ones(4, 8).as_subclass(OnGpu), torch.ones(6, 8).as_subclass(OnGpu)
    assert tl.linear_fp8(x, w).shape == (4, 6)
    ad = torch.autograd.forward_ad
    with ad.dual_level(), torch.set_grad_enabled(grad):
        assert tl.linear_fp8(x, w).shape == (4, 6)  # no tangent: as outside
        xd = ad.make_dual(x, torch.ones(4, 8)) if dual != "w" else x
        wd = ad.make_dual(w, torch.ones(6, 8)) if dual != "x" else w
        with pytest.raises(NotImplementedError):
            tl.linear_fp8(xd, wd)
    assert tl.linear_fp8(x, w).shape == (4, 6)


def test_kernel_choice_few_rows_and_many_columns():
    # bound by one read of B: the kernel measured fastest (microseconds of the
    # fastest and of the next)
    k = tl.gemm_fp8_kernel
    for M, N, K, name in ((1, 11008, 4096, "rows16"),    # 11.9, 13.2
                          (1, 28672, 8192, "rows16"),    # 43, 46
                          (1, 50257, 4096, "rows16"),    # 42, 48
                          (1, 50257, 8192, "rows16"),    # 73, 84
                          (1, 128256, 1024, "t64x64"),   # 27, 30
                          (16, 28672, 4096, "t64x64"),   # 28, 30
                          (16, 128256, 4096, "t64x64"),  # 102, 120
                          (33, 128256, 4096, "t64x64"),  # 106, 123
                          (64, 4096, 1024, "t64x64"),    # 5.3, 6.4
                          (32, 8192, 1024, "t64x64"),    # 5.6, 6.7
                          (100, 28672, 4096, "t128x128x128_w2x4")):  # 31, 39
        assert k(M, N, K).startswith(name), (M, N, K)
        assert k(N, M, K).startswith(name), (N, M, K)
