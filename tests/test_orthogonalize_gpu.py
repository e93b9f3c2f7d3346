"""GPU: orthogonalize against the iteration in 64 bits.

Tolerances.  The result is rounded to bfloat16 once: half a step is 2^-8 of a
value, and 0.42 2^-8 of the norm over many values (a rounding's error is
uniform within a step).  Before that, X is held to 22 bits and products take
half precision operands.  For matrices of random elements an emulation of
these roundings in 64 bits stays below 1.3e-3 of the norm.

Chosen spectra can do worse, and have a bound of their own.  With q(s) = b s^2
+ c s^4, a step multiplies a singular direction by a + q and adds q times the
rounding of half precision X, up to 2^-11 of an element, 0.42 2^-11 of the
norm: relative to the step's result at most |q| / |a + q| of that.  For the
usual coefficients and every s that five steps reach (up to 1.21) |q| <= 2.81
and a + q >= 0.638 (at s^2 = 1.175), a ratio of 4.4.  Where all of the norm
sits in a few equal singular values the steps' parts add up, 5 * 4.4 * 0.42 *
2^-11 = 4.5e-3 of the norm; the roundings of A and B are an order smaller
there.  For one element, 12 times the root mean square of either error.

A matrix far smaller than eps: half precision's subnormal step is 2^-24, and
stands for 2^-36 of X (held times 2^12), so hi + lo is off by up to 2^-37 at
each step, which later steps multiply by a: at most (3.4445^5 - 1) / 2.4445
2^-37 < 2e-9 for an element, FLOOR below.

These derivations take roundings to nearest.  X's high half, A' and B' are now
rounded by thresholds of an element's place, off by up to a whole step and, over
many elements, by 1.41 times as much; X is held to 21 bits.  What that makes of
matrices like those below is emulated rounding by rounding (ortho_ref, and its
tests on the CPU): up to 1.2e-3 of the norm for random ones, and below 4.5e-3
for the others, so the bounds stay.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

tl = None
USUAL = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global tl
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tiled_software_pipelined_amd import lib
    tl = lib
    yield


def want(G, steps=5, coefficients=USUAL, eps=1e-7):
    X = G.detach().cuda().double()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT.contiguous() if tall else X
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for k in range(steps):
        a, b, c = coefficients[k] if hasattr(coefficients[0], "__len__") else coefficients
        A = X @ X.mT.contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT.contiguous() if tall else X


RANDOM, CHOSEN = 1.3e-3, 4.5e-3  # error before the rounding, see above
FLOOR = 2e-9


def check(got, ref, before=RANDOM):
    assert got.dtype == torch.bfloat16 and got.shape == ref.shape
    err = got.double() - ref
    assert bool(torch.isfinite(got).all())
    dims = (-2, -1)
    norm = ref.square().sum(dims).sqrt()
    off, count = err.square().sum(dims).sqrt(), ref.shape[-1] * ref.shape[-2]
    assert bool((off <= (0.42 * 2.0 ** -8 + before) * norm + FLOOR * count ** 0.5).all()), (off / norm).max()
    rms = ref.square().mean(dims, keepdim=True).sqrt()
    assert bool((err.abs() <= 2.0 ** -8 * ref.abs() + 12 * before * rms + FLOOR).all())


def randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (16, 16), (31, 33), (63, 200), (64, 64), (65, 64), (100, 1000), (1000, 100),
          (128, 384), (257, 129), (256, 256), (300, 301), (513, 700), (1, 5000), (5000, 3), (1030, 520)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_shapes(rows, cols, dtype):
    G = randn(rows, cols, seed=rows + cols, dtype=dtype)
    check(tl.orthogonalize(G), want(G))


# sizes that reach the larger tiles of either kind of product, batches too
@pytest.mark.parametrize("batch,rows,cols", [(1, 1500, 1400), (1, 1100, 4200), (6, 530, 1100), (1, 3500, 3600),
                                             (2, 2600, 2500), (40, 200, 190), (300, 40, 70), (3, 129, 2000),
                                             (1, 4300, 4400)])
def test_large_and_batched(batch, rows, cols):
    G = randn(batch, rows, cols, seed=rows, dtype=torch.bfloat16)
    check(tl.orthogonalize(G), want(G))


# few rows and a long axis: the first product is shared by several workgroups,
# whose last one takes fewer columns
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 4096), (1, 64, 4096), (1, 5000, 130), (3, 70, 4500), (2, 200, 8200),
                                             (5, 64, 6000), (1, 129, 40000), (1, 3, 300001)])
def test_few_rows(batch, rows, cols):
    import ctypes
    G = randn(batch, rows, cols, seed=cols, dtype=torch.bfloat16)
    got = tl.orthogonalize(G)
    check(got, want(G))
    # the same every time, and whatever the workspace held
    need = tl._lib.tgemm_orthogonalize_workspace_bytes(batch, rows, cols)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    out, co = torch.zeros_like(got), (ctypes.c_double * 15)(*USUAL * 5)
    for _ in range(8):
        assert tl._lib.tgemm_orthogonalize(batch, rows, cols, tl.BF16, G.data_ptr(), cols, rows * cols, out.data_ptr(),
                                           cols, rows * cols, 5, co, 1e-7, (ws.data_ptr() + 255) // 256 * 256, need,
                                           torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(out, got)


def test_few_rows_at_once_and_replayed():
    xs = randn(100, 5000, seed=21), randn(2, 4200, 60, seed=22)
    ref = [tl.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(tl.orthogonalize(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref[i % 2]) for i, g in enumerate(got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        held = tl.orthogonalize(xs[0])
    for r in range(4):
        xs[0].add_(0.5 * torch.randn_like(xs[0]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, tl.orthogonalize(xs[0])), r


def spectrum(kind, m, n):
    u = torch.linalg.qr(randn(m, m, seed=1).double().cpu())[0]
    v = torch.linalg.qr(randn(n, m, seed=2).double().cpu())[0]
    i = torch.arange(m, dtype=torch.float64)
    s = {"flat": torch.ones(m), "inverse": 1 / (1 + i), "decaying": torch.exp(-i / (m / 12)),
         "one": torch.where(i == 0, 1.0, 1e-3), "few": torch.where(i < 16, 1.0, 1e-3),
         "deficient": torch.where(i < m // 4, 1.0, 0.0)}[kind].double()
    return ((u * s) @ v.t()).float().cuda()


@pytest.mark.parametrize("kind", ["flat", "inverse", "decaying", "one", "few", "deficient"])
@pytest.mark.parametrize("m,n", [(96, 96), (200, 500)])
def test_spectra(kind, m, n):
    G = spectrum(kind, m, n)
    check(tl.orthogonalize(G), want(G), CHOSEN)
    check(tl.orthogonalize(G.t()), want(G.t()), CHOSEN)


def test_singular_values_come_near_one():
    # the usual coefficients bring what is above 1/300 of the norm into 0.6 .. 1.3
    s = torch.linalg.svdvals(tl.orthogonalize(randn(200, 400, seed=3)).float().cpu())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("scale", [1e-30, 1e-15, 1e15, 1e30])
def test_scale_of_the_input(scale):
    G = randn(70, 90, seed=4) * scale
    for eps in (1e-7, 0.0, 1e-38):
        check(tl.orthogonalize(G, eps=eps), want(G, eps=eps))


def test_zeros_and_rows_of_zeros():
    assert (tl.orthogonalize(torch.zeros(40, 60, device="cuda")) == 0).all()
    G = randn(60, 80, seed=5)
    G[7:20] = 0
    G[:, 33] = 0
    got = tl.orthogonalize(G)
    check(got, want(G))
    assert (got[7:20] == 0).all() and (got[:, 33] == 0).all()
    # a zero matrix beside others
    G = randn(3, 60, 80, seed=6)
    G[1] = 0
    got = tl.orthogonalize(G)
    assert (got[1] == 0).all()
    check(got[::2], want(G[::2]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_a_number_stays_in_its_matrix(bad):
    G = randn(3, 50, 70, seed=7)
    clean = tl.orthogonalize(G)
    G[1, 3, 4] = bad
    got = tl.orthogonalize(G)
    assert got[1].isnan().all() and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def test_coefficients_and_steps():
    G = randn(90, 150, seed=8)
    for steps, co in ((1, USUAL), (2, USUAL), (8, USUAL), (6, (1.5, -0.5, 0.0)), (64, (1.875, -1.25, 0.375)),
                      (3, [(3.5, -6.0, 3.0), (2.5, -3.0, 1.2), (1.5, -0.5, 0.0)]), (1, (0.0, 1.0, -1.0)),
                      (2, [(1.0, 0.0, 0.0), (100.0, 0.0, 0.0)])):
        check(tl.orthogonalize(G, steps=steps, coefficients=co), want(G, steps, co))


def test_strides_and_out():
    big = randn(2, 5, 70, 110, seed=9, dtype=torch.bfloat16)
    G = big[:, 1, 3:60, 7:100]
    ref = want(G)
    got = tl.orthogonalize(G)
    check(got, ref)
    assert torch.equal(tl.orthogonalize(G.contiguous()), got)
    assert torch.equal(tl.orthogonalize(big[:, 1].mT), tl.orthogonalize(big[:, 1].mT.contiguous()))
    assert torch.equal(tl.orthogonalize(G[0].expand(3, 57, 93)), got[:1].expand(3, 57, 93))
    assert torch.equal(tl.orthogonalize(big[0, :2]), tl.orthogonalize(big)[0, :2])
    # into a larger tensor, nothing beside it written
    for shape in ((57, 93), (93, 57)):
        g = G[0] if shape[0] == 57 else G[0].t()
        out = torch.full((4, shape[0] + 3, shape[1] + 5), -3.0, dtype=torch.bfloat16, device="cuda")
        view = out[1, 2:2 + shape[0], 3:3 + shape[1]]
        assert tl.orthogonalize(g, out=view) is view
        assert torch.equal(view, tl.orthogonalize(g))
        view.fill_(-3.0)
        assert (out == -3.0).all()
    # in place
    g = G.contiguous()
    tl.orthogonalize(g, out=g)
    assert torch.equal(g, got)


def test_transpose_of_a_matrix_gives_the_transpose():
    G = randn(130, 210, seed=10)
    assert torch.equal(tl.orthogonalize(G.t()), tl.orthogonalize(G).t())


def test_empty_and_refusals():
    for shape in ((0, 5, 6), (5, 0), (0, 5)):
        assert tl.orthogonalize(torch.zeros(shape, device="cuda")).shape == shape
    G = randn(20, 30)
    for kw in (dict(G=G.double()), dict(G=G[0]), dict(G=G.cpu()), dict(coefficients=[USUAL] * 4),
               dict(coefficients=(1.0, 2.0)), dict(out=torch.empty(20, 30, device="cuda")),
               dict(out=torch.empty(30, 20, dtype=torch.bfloat16, device="cuda")),
               dict(out=torch.empty(30, 20, dtype=torch.bfloat16, device="cuda").t())):
        with pytest.raises((ValueError, TypeError)):
            tl.orthogonalize(**{**dict(G=G), **kw})
    for kw in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(coefficients=(9.0, 0.0, 0.0)),
               dict(coefficients=(float("nan"), 0.0, 0.0))):
        with pytest.raises(tl.TgemmError):
            tl.orthogonalize(G, **kw)


def test_small_workspace_is_refused_before_anything_runs():
    import ctypes
    G = randn(64, 64)
    out = torch.full((64, 64), -3.0, dtype=torch.bfloat16, device="cuda")
    need = tl._lib.tgemm_orthogonalize_workspace_bytes(1, 64, 64)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    base = (ws.data_ptr() + 255) // 256 * 256
    co = (ctypes.c_double * 15)(*USUAL * 5)
    args = [1, 64, 64, tl.F32, G.data_ptr(), 64, 0, out.data_ptr(), 64, 0, 5, co, 1e-7, base]
    s = torch.cuda.current_stream().cuda_stream
    assert tl._lib.tgemm_orthogonalize(*args, need - 1, s) == -1
    torch.cuda.synchronize()
    assert (out == -3.0).all()
    assert tl._lib.tgemm_orthogonalize(*args, need, s) == 0
    assert torch.equal(out, tl.orthogonalize(G))


def test_streams_and_graphs():
    G, H = randn(150, 200, seed=11, dtype=torch.bfloat16), randn(2, 300, 60, seed=12)
    ref = tl.orthogonalize(G), tl.orthogonalize(H)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for _ in range(3):  # two calls at once
        for s, x in zip(streams, (G, H)):
            with torch.cuda.stream(s):
                got.append(tl.orthogonalize(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref[i % 2]) for i, g in enumerate(got))
    graphs = []
    for x in (G, H):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            held = tl.orthogonalize(x)
        graphs.append((graph, held, x))
    for r in range(4):
        for graph, held, x in graphs:
            x.add_(0.5 * torch.randn_like(x))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(held, tl.orthogonalize(x)), r


# ---- the operators together ---------------------------------------------------

def test_a_training_step_of_one_layer():
    """Forward and backward through linear_fp8, momentum, the orthogonalised
    update, and the updated weight's product: each part against its reference."""
    import numpy as np
    import fp8_ref as ref8
    M, N, K = 200, 130, 260
    x = randn(M, K, seed=13, dtype=torch.bfloat16)
    w = (randn(N, K, seed=14) * 0.05).bfloat16().requires_grad_()
    gy = randn(M, N, seed=15, dtype=torch.bfloat16) * 1e-3
    momentum = randn(N, K, seed=16) * 1e-3
    y = tl.linear_fp8(x, w)
    y.backward(gy)
    momentum.mul_(0.95).add_(w.grad)
    update = tl.orthogonalize(momentum)
    check(update, want(momentum))
    with torch.no_grad():
        w.add_(update, alpha=-0.02)
    y2 = tl.linear_fp8(x, w.detach())
    h = lambda t: t.detach().float().double().cpu().numpy()  # noqa: E731
    xv, wv = ref8.values(*ref8.quantize(h(x))), ref8.values(*ref8.quantize(h(w), block="square"))
    p, mag = ref8.product(xv, wv)
    assert (np.abs(h(y2) - p) <= ref8.gemm_bound(p, mag, K)).all()
    gt, xt = ref8.values(*ref8.quantize(h(gy).T.copy())), ref8.values(*ref8.quantize(h(x).T.copy()))
    p, mag = ref8.product(gt, xt)
    assert (np.abs(h(w.grad) - p) <= ref8.gemm_bound(p, mag, M)).all()


# ---- matrices whose roundings do not average out ---------------------------------

def check_emulated(G):
    """Within what the roundings make of it: the result's own (half a step is 2^-8
    of a value, all of them off the same way where elements are equal), and float
    sums where the emulation's are in double.  Those, some 2^-22 off, turn a half
    precision rounding (2^-10 of a value, one element in 2^11 near enough to its
    threshold) at most: 2^-10 2^-5.5 of the norm, and times 6 for what each of five
    steps makes of it, below 7e-4."""
    import ortho_ref
    got = tl.orthogonalize(G.cuda())
    check(got, want(G), CHOSEN)
    emulated = ortho_ref.emulate(G)
    off = float((got.cpu().double() - emulated).norm() / emulated.norm())
    assert off <= 2.0 ** -8 + 7e-4, off


@pytest.mark.parametrize("m,n", [(2, 4), (3, 21), (5, 193), (17, 4), (40, 1000), (64, 65), (60, 9000), (65, 70),
                                 (100, 128), (70, 1000), (200, 90), (129, 300), (300, 280)])
def test_low_rank(m, n):
    import ortho_ref
    for G in ortho_ref.low_rank(m, n).values():
        check_emulated(G)


def test_repeated_elements():
    import ortho_ref
    for kind, G in ortho_ref.repeated().items():
        print(kind, flush=True)
        check_emulated(G)
        check_emulated(G.t())


def test_not_a_number_of_any_pattern():
    # all mantissa bits set: adding a threshold to the pattern leaves the NaNs
    for dtype, pattern, ints in ((torch.float32, 0x7FFFFFFF, torch.int32), (torch.float32, -1, torch.int32),
                                 (torch.bfloat16, 0x7FFF, torch.int16), (torch.float16, -1, torch.int16)):
        for m, n in ((50, 70), (70, 90), (300, 280)):
            G = randn(2, m, n, seed=m, dtype=dtype)
            clean = tl.orthogonalize(G)
            G.view(ints)[1, m // 2, n // 3] = pattern
            for steps in (1, 5):
                got = tl.orthogonalize(G, steps=steps)
                assert bool(got[1].isnan().all()), (dtype, pattern, m, steps)
            assert torch.equal(got[0], clean[0])


def test_few_steps_of_small_matrices():
    for m, n in ((1, 1), (40, 70), (64, 64), (3, 5000), (64, 4200), (70, 90)):
        G = randn(m, n, seed=m + n)
        for steps in (1, 2, 3):
            got, ref = tl.orthogonalize(G, steps=steps), want(G, steps)
            if m * n > 1:
                check(got, ref)
            else:
                # 0.42 of half a step is for many values; one is off by up to all of
                # it (three steps make 1.1136 of one element, between 1.1094 and
                # 1.1172: off by 0.0036 rounded to nearest, 0.42 2^-8 of it is 0.0018)
                assert float((got.double() - ref).abs()) <= (2.0 ** -8 + RANDOM) * float(ref.abs())


def test_small_matrices_at_once_and_replayed():
    # up to 64 rows, the first product shared by several workgroups or not
    xs = randn(64, 4200, seed=31), randn(3, 40, 90, seed=32)
    ref = [tl.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(tl.orthogonalize(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref[i % 2]) for i, g in enumerate(got))
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            graphs.append((graph, tl.orthogonalize(x), x))
    for r in range(4):
        for graph, held, x in graphs:
            x.add_(0.5 * torch.randn_like(x))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(held, tl.orthogonalize(x)), r
