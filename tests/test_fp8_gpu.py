"""GPU: the 8-bit block-scaled operators against 64-bit references.

Quantised values and scales have to be equal bit for bit.  Products are held
to fp8_ref.gemm_bound per element, and over all elements to one bfloat16
rounding (2^-8 of the norm), which a lost slice of K would exceed.
"""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

tl = None
FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global tl
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tiled_software_pipelined_amd import lib
    tl = lib
    yield


def draw(rows, cols, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(spread * torch.randn((rows, 1), generator=g))
    x *= torch.exp(spread * torch.randn((1, cols), generator=g))
    return x.to(dtype)


def host(t):
    return t.detach().cpu().float().double().numpy()


def exps(s):
    return s.contiguous().view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def check_image(x, fmt, block, q, s):
    vq, ve = ref.quantize(x, fmt, block)
    assert np.array_equal(host(q), vq, equal_nan=True)
    assert np.array_equal(exps(s), ve)


# ---- quantize_fp8 ----------------------------------------------------------------

SIZES = [(1, 1), (1, 128), (3, 7), (16, 4096), (17, 129), (127, 127), (128, 128), (129, 257), (200, 1000), (1, 5000),
         (300, 8), (640, 384)]


@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(rows, cols, fmt, block):
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x = draw(rows, cols, rows * 1000 + cols, dtype, spread=1.0)
        v = host(x)
        q, s = tl.quantize_fp8(x.cuda(), dtype=FMT[fmt], block=block)
        check_image(v, fmt, block, q, s)
        q, s, qt, st = tl.quantize_fp8(x.cuda(), dtype=FMT[fmt], block=block, transpose=True)
        check_image(v, fmt, block, q, s)
        check_image(np.ascontiguousarray(v.T), fmt, block, qt, st)
        if block == "square":
            assert torch.equal(qt.view(torch.uint8), q.view(torch.uint8).t())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_borders(fmt):
    # largest values on and next to the border of a scale, ties, zeros, the
    # smallest and largest floats, subnormals
    top = ref.TABLE[fmt][-1]
    rows = []
    for k in (-140, -127, -126, -3, 0, 5, 100):
        for m in (1.0, 1.0 + 2.0 ** -20, 1.0 - 2.0 ** -20, 0.5):
            big = np.float64(np.float32(top * m * 2.0 ** k))
            t = ref.TABLE[fmt]
            mids = np.concatenate([(t[:-1] + t[1:]) / 2, t])[:100] * 2.0 ** k
            rows.append(np.concatenate([[big], np.minimum(mids, abs(big)), np.zeros(128 - 1 - len(mids))]))
    rows.append(np.zeros(128))
    rows.append(np.full(128, 2.0 ** -149))
    rows.append(np.full(128, float(np.finfo(np.float32).max)))
    x = torch.from_numpy(np.array(rows)).float()
    q, s, qt, st = tl.quantize_fp8(x.cuda(), dtype=FMT[fmt], transpose=True)
    check_image(host(x), fmt, "row", q, s)
    check_image(np.ascontiguousarray(host(x).T), fmt, "row", qt, st)


@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_nan_and_infinity_stay_where_they_are(fmt, block):
    x = draw(150, 300, 5, spread=0.5)
    x[3, 7], x[140, 299], x[4, 7], x[5, 8] = float("nan"), float("inf"), float("-inf"), -float("nan")
    x[9, :] = float("nan")
    x[:, 256:] = torch.where(torch.arange(150)[:, None] == 20, float("inf"), x[:, 256:])
    q, s, qt, st = tl.quantize_fp8(x.cuda(), dtype=FMT[fmt], block=block, transpose=True)
    check_image(host(x), fmt, block, q, s)
    check_image(np.ascontiguousarray(host(x).T), fmt, block, qt, st)


def test_quantize_strided_and_unaligned_input():
    big = draw(70, 400, 9, torch.bfloat16, 1.0).cuda()
    x = big[2:67, 3:331]
    q, s, qt, st = tl.quantize_fp8(x, transpose=True)
    check_image(host(x), "e4m3", "row", q, s)
    check_image(np.ascontiguousarray(host(x).T), "e4m3", "row", qt, st)


def test_quantize_writes_only_its_images():
    rows, cols, off = 131, 261, 5
    x = draw(rows, cols, 11, torch.bfloat16, 1.0).cuda()
    ldq, lds, ldqt, ldst = cols + 9, rows + 3, rows + 7, cols + 2
    nb, nt = -(-cols // 128), -(-rows // 128)
    bufs = [torch.full((off + n,), 0xA5, dtype=torch.uint8, device="cuda")
            for n in (rows * ldq, nb * lds, cols * ldqt, nt * ldst)]
    q, s, qt, st = (b[off:] for b in bufs)
    assert tl._lib.tgemm_fp8_quantize(rows, cols, tl.BF16, x.data_ptr(), cols, 0, 0, q.data_ptr(), ldq, s.data_ptr(), lds,
                                      qt.data_ptr(), ldqt, st.data_ptr(), ldst,
                                      torch.cuda.current_stream().cuda_stream) == 0
    want = tl.quantize_fp8(x, transpose=True)
    for buf, view, ld, n, w in zip(bufs, (q, s, qt, st), (ldq, lds, ldqt, ldst), (cols, rows, rows, cols), want):
        m = view.view(-1, ld)
        assert torch.equal(m[:, :n], w.view(torch.uint8))
        assert (m[:, n:] == 0xA5).all() and (buf[:off] == 0xA5).all()


def test_quantize_of_nothing():
    for shape in ((0, 128), (128, 0), (0, 0)):
        q, s, qt, st = tl.quantize_fp8(torch.zeros(shape, device="cuda"), transpose=True)
        assert q.shape == shape and qt.shape == shape[::-1]
        assert s.shape == (-(-shape[1] // 128), shape[0]) and st.shape == (-(-shape[0] // 128), shape[1])


# ---- gemm_fp8 ----------------------------------------------------------------------

def operand(rows, cols, seed, fmt="e4m3", spread=1.0):
    """(Q, S) on the GPU and their values in 64 bits."""
    x = draw(rows, cols, seed, spread=spread).cuda()
    q, s = tl.quantize_fp8(x, dtype=FMT[fmt])
    return q, s, ref.values(host(q), exps(s))


def check_product(c, av, bv, k):
    want, mag = ref.product(av, bv)
    got = host(c)
    err = np.abs(got - want)
    assert (err <= ref.gemm_bound(want, mag, k)).all(), float((err / ref.gemm_bound(want, mag, k)).max())
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 2.0 ** -8 * norm


GEMMS = [(1, 1, 1), (1, 16, 128), (1, 4096, 1024), (2, 17, 100), (5, 333, 1025), (16, 64, 127), (17, 40, 384),
         (32, 100, 129), (33, 65, 511), (64, 512, 2048), (65, 64, 128), (65, 1, 300), (100, 1000, 1000), (128, 128, 256),
         (129, 127, 255), (200, 300, 1), (256, 256, 1024), (257, 259, 900), (500, 64, 3000), (1000, 1100, 640),
         (300, 200, 1111), (70, 90, 2177)]


@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm(M, N, K):
    a, sa, av = operand(M, K, M + K)
    b, sb, bv = operand(N, K, N + 2 * K)
    c = tl.gemm_fp8(a, sa, b, sb)
    check_product(c, av, bv, K)
    # rows back to back, at any byte, where the quantiser padded them
    assert torch.equal(tl.gemm_fp8(a.contiguous(), sa, b.contiguous(), sb), c)


@pytest.mark.parametrize("K", [1, 5, 15, 16, 17, 31, 64, 80, 100, 112, 127, 128, 129, 143, 145, 192, 250, 255, 257, 400])
@pytest.mark.parametrize("M,N", [(70, 90), (300, 1400), (1900, 1990), (3500, 3600)])
def test_gemm_short_rows_and_partial_slices(M, N, K):
    # every element is 1: C is K exactly (rounded), whatever repeats a byte shows;
    # then an infinity or a NaN in one place, which only its row and column see
    one = torch.ones((M, K), device="cuda"), torch.ones((N, K), device="cuda")
    (a, sa), (b, sb) = (tl.quantize_fp8(x, dtype=torch.float8_e5m2) for x in one)
    want = torch.full((M, N), float(K), device="cuda").bfloat16()
    assert torch.equal(tl.gemm_fp8(a, sa, b, sb), want)
    for k in sorted({0, K // 2, max(K - 17, 0), K - 1}):
        bits = a.clone().view(torch.uint8)
        bits[M - 1, k] = 0x7C  # infinity
        c = tl.gemm_fp8(bits.view(a.dtype), sa, b, sb)
        assert bool(torch.isposinf(c[M - 1]).all()) and torch.equal(c[:M - 1], want[:M - 1]), k


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M,N,K", [(3, 200, 700), (30, 48, 300), (60, 64, 1200), (130, 140, 520), (520, 640, 333)])
def test_gemm_formats(M, N, K, fa, fb):
    a, sa, av = operand(M, K, M + K, fa)
    b, sb, bv = operand(N, K, N + 2 * K, fb)
    check_product(tl.gemm_fp8(a, sa, b, sb), av, bv, K)


# sizes that reach each kernel of the choice; the large ones against a product
# in float64 on the GPU
@pytest.mark.parametrize("M,N,K,kernel,last", [
    (7, 520, 1300, "rows16", ""), (20, 5000, 1300, "rows32", ""), (520, 9, 1300, "rows16", ""),
    (5001, 30, 1300, "rows32", ""), (300, 1400, 1300, "t64x64", ""), (1500, 1400, 1000, "t64x64", ""),
    (1900, 1990, 2100, "t128x128x128_w2x4_s4", ""), (2048, 2031, 3001, "t128x128x128_w2x4_s4", ""),
    (2000, 3900, 2500, "t128x128x128_w2x2_s2", ""), (3600, 3500, 300, "t256x256", ""),
    (3585, 3583, 1290, "t256x256", ""), (4096, 4096, 128, "t256x256", ""), (3500, 3600, 100, "t256x256", ""),
    (4095, 4097, 520, "t256x256", "rows16"), (4128, 4090, 300, "t256x256", "rows32"), (4070, 4106, 700, "t256x256", "rows16")])
def test_gemm_every_kernel(M, N, K, kernel, last):
    assert tl.gemm_fp8_kernel(M, N, K).startswith(kernel)
    assert tl.gemm_fp8_kernel(M, N, K, piece=1).startswith(last) and bool(tl.gemm_fp8_kernel(M, N, K, piece=1)) == bool(last)
    fa = "e5m2" if M % 2 else "e4m3"
    a, sa = tl.quantize_fp8(draw(M, K, 1).cuda(), dtype=FMT[fa])
    b, sb = tl.quantize_fp8(draw(N, K, 2).cuda())

    def v(q, s):
        e = (s.contiguous().view(torch.uint8).double() - 127).t().repeat_interleave(128, 1)[:, :K]
        return q.double() * torch.exp2(e)
    av, bv = v(a, sa), v(b, sb)
    want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    c = tl.gemm_fp8(a, sa, b, sb)
    assert torch.equal(tl.gemm_fp8(a.contiguous(), sa, b.contiguous(), sb), c)
    c = c.double()
    off = (2.0 ** -10 + (K / 8 + 16) * 2.0 ** -24) * mag
    assert bool(((c - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all())
    assert float((c - want).norm()) <= 2.0 ** -8 * float(want.norm())


def test_gemm_random_shapes():
    import random
    r = random.Random(7)
    for i in range(60):
        M, N, K = (max(1, int(2 ** r.uniform(0, top))) for top in (11.5, 11.5, 12))
        fa, fb = r.choice(["e4m3", "e5m2"]), r.choice(["e4m3", "e5m2"])
        a, sa = tl.quantize_fp8(draw(M, K, i, spread=0.5).cuda(), dtype=FMT[fa])
        b, sb = tl.quantize_fp8(draw(N, K, i + 100, spread=0.5).cuda(), dtype=FMT[fb])

        def v(q, s):
            e = (s.contiguous().view(torch.uint8).double() - 127).t().repeat_interleave(128, 1)[:, :K]
            return q.double() * torch.exp2(e)
        av, bv = v(a, sa), v(b, sb)
        want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
        off = (2.0 ** -10 + (K / 8 + 16) * 2.0 ** -24) * mag
        c = tl.gemm_fp8(a, sa, b, sb)
        assert torch.equal(tl.gemm_fp8(a.contiguous(), sa, b.contiguous(), sb), c), (M, N, K, fa, fb)
        c = c.double()
        assert bool(((c - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all()), (M, N, K, fa, fb)


def test_gemm_two_at_once():
    # two products on two streams, over and over, each against its own result
    sets = []
    for M, N, K, s in ((300, 900, 700, 1), (4, 3000, 1500, 2)):
        a, sa, _ = operand(M, K, s)
        b, sb, _ = operand(N, K, s + 10)
        sets.append((a, sa, b, sb, tl.gemm_fp8(a, sa, b, sb)))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for st, x in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append((tl.gemm_fp8(*x[:4]), x[4]))
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c, want in got)


def test_matrix_instruction_alignment():
    # what gemm_bound rests on: a product 13 binades below the largest of its
    # group of eight survives, and groups are added to 26 binades; the large
    # product is cancelled exactly by the next block
    for rows in (16, 65, 300):
        for n, j, kept in ((1, 13, 1), (7, 13, 7), (8, 13, 8), (127, 13, 127), (127, 26, 120)):
            a, b = torch.zeros(rows, 256), torch.zeros(16, 256)
            a[:, 0], b[:, 0], a[:, 128], b[:, 128] = 1, 1, -1, 1
            a[:, 1:1 + n], b[:, 1:1 + n] = 2.0 ** -(j // 2), 2.0 ** -(j - j // 2)
            sa = torch.full((2, -(-rows // 16) * 16), 127, dtype=torch.uint8, device="cuda")[:, :rows]
            sb = torch.full((2, 16), 127, dtype=torch.uint8, device="cuda")
            c = tl.gemm_fp8(a.to(FMT["e5m2"]).cuda(), sa, b.to(FMT["e5m2"]).cuda(), sb)
            assert bool((c.float() >= kept * 2.0 ** -j * (1 - 2.0 ** -8)).all()), (rows, n, j)


def test_gemm_exact_small_integers():
    # integers and powers of two: every sum is exact, and so is its bfloat16
    for M, N, K in ((4, 30, 260), (90, 70, 260), (400, 500, 300)):
        g = torch.Generator().manual_seed(M)
        a = torch.randint(-1, 2, (M, K), generator=g).float()
        b = torch.randint(-1, 2, (N, K), generator=g).float()
        nb = -(-K // 128)
        ea, eb = torch.randint(0, 2, (nb, -(-M // 4) * 4), generator=g), torch.randint(0, 2, (nb, -(-N // 4) * 4), generator=g)
        sa, sb = ((127 + e).to(torch.uint8).cuda() for e in (ea, eb))
        c = tl.gemm_fp8(a.to(FMT["e4m3"]).cuda(), sa[:, :M], b.to(FMT["e4m3"]).cuda(), sb[:, :N])
        av = ref.values(a.double().numpy(), ea[:, :M].numpy())
        bv = ref.values(b.double().numpy(), eb[:, :N].numpy())
        want = torch.from_numpy(av @ bv.T).to(torch.bfloat16)
        assert torch.equal(c.cpu(), want)


def test_gemm_strided_unaligned_and_padded():
    # rows at odd bytes with gaps, C inside a larger matrix, NaN in every gap
    for M, N, K in ((5, 70, 300), (90, 110, 385), (515, 640, 250)):
        a, sa, av = operand(M, K, 3)
        b, sb, bv = operand(N, K, 4)

        def inside(q, off, ld):
            buf = torch.full((off + q.shape[0] * ld,), 0x7F, dtype=torch.uint8, device="cuda")
            v = buf[off:].view(q.shape[0], ld)[:, :q.shape[1]]
            v.copy_(q.view(torch.uint8))
            return v.view(q.dtype)
        a2, b2 = inside(a, 3, K + 5), inside(b, 1, K + 14)
        out = torch.full((M + 2, N + 7), -3.0, dtype=torch.bfloat16, device="cuda")
        c = out[1:M + 1, 3:N + 3]
        assert tl.gemm_fp8(a2, sa, b2, sb, out=c) is c
        assert torch.equal(c, tl.gemm_fp8(a, sa, b, sb))
        check_product(c, av, bv, K)
        out[1:M + 1, 3:N + 3] = -3.0
        assert (out == -3.0).all()


def test_gemm_scales_past_the_last_row_do_not_matter():
    for M, N in ((3, 5), (67, 71), (301, 299)):
        a, sa, _ = operand(M, 256, 1)
        b, sb, _ = operand(N, 256, 2)
        want = tl.gemm_fp8(a, sa, b, sb)

        def poisoned(s, rows):
            t = torch.full((s.shape[0], -(-rows // 16) * 16), 255, dtype=torch.uint8, device="cuda")
            t[:, :rows] = s.view(torch.uint8)
            return t[:, :rows]
        assert torch.equal(tl.gemm_fp8(a, poisoned(sa, M), b, poisoned(sb, N)), want)


def test_gemm_nan_reaches_its_row_and_column_only():
    for M, N, K in ((6, 40, 300), (80, 90, 300), (520, 530, 300)):
        a, sa, _ = operand(M, K, 1)
        b, sb, _ = operand(N, K, 2)
        clean = tl.gemm_fp8(a, sa, b, sb)
        a.view(torch.uint8)[M // 2, 290] = 0x7F   # NaN value in the tail of K
        sb = sb.contiguous().view(torch.uint8)
        sb = torch.nn.functional.pad(sb, (0, -N % 4))[:, :N]
        sb[1, N // 3] = 255                       # NaN scale
        c = tl.gemm_fp8(a, sa, b, sb)
        want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        want[M // 2], want[:, N // 3] = True, True
        assert torch.equal(c.isnan(), want)
        assert torch.equal(c[~want], clean[~want])


def test_gemm_extreme_scales():
    # 2^127 2^-127 = 1, products past float's range, and below it
    one = torch.ones(2, 128).to(FMT["e4m3"]).cuda()
    s = lambda v: torch.full((1, 4), v, dtype=torch.uint8, device="cuda")[:, :2]  # noqa: E731
    assert (tl.gemm_fp8(one, s(254), one, s(0)) == 128).all()
    assert (tl.gemm_fp8(one, s(254), one, s(254)) == float("inf")).all()
    assert (tl.gemm_fp8(one, s(0), one, s(0)) == 0).all()


def test_gemm_empty():
    z = lambda r, c: torch.zeros(r, c).to(FMT["e4m3"]).cuda()  # noqa: E731
    s = lambda c, r: torch.zeros(-(-c // 128), -(-max(r, 1) // 16) * 16, dtype=torch.uint8, device="cuda")[:, :r]  # noqa: E731
    for M, N in ((3, 9), (200, 300)):
        out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
        assert (tl.gemm_fp8(z(M, 0), s(0, M), z(N, 0), s(0, N), out=out) == 0).all()
    assert tl.gemm_fp8(z(0, 64), s(64, 0), z(5, 64), s(64, 5)).shape == (0, 5)
    assert tl.gemm_fp8(z(5, 64), s(64, 5), z(0, 64), s(64, 0)).shape == (5, 0)


def test_gemm_refusals():
    a, sa, _ = operand(8, 256, 1)
    b, sb, _ = operand(12, 256, 2)
    bad = [dict(A=a[:, :128]), dict(SA=sa[:1]), dict(SB=sa), dict(A=a.float()), dict(SA=sa.view(torch.uint8).float()),
           dict(B=b.cpu()), dict(SA=sa.cpu()), dict(A=a.t()), dict(A=a[:1].expand(8, 256)),
           dict(out=torch.empty(8, 12, device="cuda")), dict(out=torch.empty(12, 8, dtype=torch.bfloat16, device="cuda")),
           dict(out=torch.empty(12, 8, dtype=torch.bfloat16, device="cuda").t()),
           dict(out=torch.empty(8, 12, dtype=torch.bfloat16))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            tl.gemm_fp8(**{**dict(A=a, SA=sa, B=b, SB=sb), **kw})


def test_rows_longer_than_32_bit_offsets():
    # lda of 2^26: a 64-row tile's offsets pass 2^31 and still fit in 32 bits; of
    # 2^27 they do not, and 64-bit addresses take over
    M, N, K, ld = 70, 4100, 1000, 1 << 26
    a, sa, av = operand(M, K, 1)
    b, sb, bv = operand(N, K, 2)
    buf = torch.empty((M - 1) * ld + K, dtype=torch.uint8, device="cuda")
    for m, step, kernel in ((M, ld, "t64x64"), (M // 2, 2 * ld, "rows")):
        assert tl.gemm_fp8_kernel(m, N, K, lda=step).startswith(kernel)
        big = buf[:(m - 1) * step + K].as_strided((m, K), (step, 1))
        big.copy_(a[:m].view(torch.uint8))
        s = sa.view(torch.uint8)[:, :m]
        check_product(tl.gemm_fp8(big.view(a.dtype), s, b, sb), av[:m], bv, K)


def test_more_than_2_to_the_31_elements():
    M, K = 66000, 33000
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x[:M // 2] = torch.randn((M // 2, K), device="cuda")
    x[M // 2:] = torch.randn((M - M // 2, K), device="cuda")
    q, s, qt, st = tl.quantize_fp8(x, transpose=True)
    r, c = M // 128 * 128 - 256, K // 128 * 128 - 256  # the last blocks of rows, of columns
    for got, want in ((q[r:], 0), (s[:, r:], 1), (qt[:, r:], 2), (st[r // 128:], 3)):
        assert torch.equal(got.contiguous().view(torch.uint8),
                           tl.quantize_fp8(x[r:], transpose=True)[want].contiguous().view(torch.uint8))
    for got, want in ((q[:, c:], 0), (s[c // 128:], 1), (qt[c:], 2), (st[:, c:], 3)):
        assert torch.equal(got.contiguous().view(torch.uint8),
                           tl.quantize_fp8(x[:, c:], transpose=True)[want].contiguous().view(torch.uint8))
    # a product of as many results: its last rows against those of the last rows alone
    w, ws = tl.quantize_fp8(torch.randn((K, 200), device="cuda"))
    a, sa = q[:, :200], s[:2]
    y = tl.gemm_fp8(a, sa, w, ws)
    assert y.shape == (M, K) and y.numel() > 2 ** 31
    for rows in (slice(0, 128), slice(r, M)):
        want = tl.gemm_fp8(a[rows], sa[:, rows], w, ws).double()
        assert float((y[rows].double() - want).norm()) <= 2.0 ** -7 * float(want.norm())  # two roundings


def test_on_another_stream_and_replayed_from_a_graph():
    x = draw(130, 300, 1, torch.bfloat16).cuda()
    w = draw(200, 300, 2, torch.bfloat16).cuda()

    def step():
        xq = tl.quantize_fp8(x, transpose=True)
        wq = tl.quantize_fp8(w, block="square", transpose=True)
        return tl.gemm_fp8(xq[0], xq[1], wq[0], wq[1]), xq[2], wq[3]
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    same = lambda p, q: all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(p, q))  # noqa: E731
    assert same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for r in range(4):
        x.mul_(2.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, step()), r


# ---- linear_fp8 -------------------------------------------------------------------

def linear_reference(x, w, gy, grad_fmt="e4m3"):
    """(y, dx, dw), and their sums of magnitudes, of float64 matrices."""
    xv, wv, gv = ref.values(*ref.quantize(x)), ref.values(*ref.quantize(w, block="square")), ref.values(*ref.quantize(gy, grad_fmt))
    xt, gt = ref.values(*ref.quantize(x.T.copy())), ref.values(*ref.quantize(gy.T.copy(), grad_fmt))
    return ref.product(xv, wv), ref.product(gv, wv.T), ref.product(gt, xt)


@pytest.mark.parametrize("grad_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (3, 130, 257), (65, 64, 128), (150, 200, 300), (260, 520, 390)])
def test_linear_and_gradients(M, N, K, grad_fmt):
    x = draw(M, K, 1, torch.bfloat16, 0.5).cuda().requires_grad_()
    w = draw(N, K, 2, torch.bfloat16, 0.5).cuda().requires_grad_()
    gy = draw(M, N, 3, torch.bfloat16, 0.5).cuda()
    y = tl.linear_fp8(x, w, grad_dtype=FMT[grad_fmt])
    y.backward(gy)
    for got, (want, mag), k in zip((y, x.grad, w.grad), linear_reference(host(x), host(w), host(gy), grad_fmt), (K, N, M)):
        assert got.dtype == torch.bfloat16
        err = np.abs(host(got) - want)
        assert (err <= ref.gemm_bound(want, mag, k)).all()


def test_linear_gradient_is_that_of_the_unrounded_layer():
    # against differences of the unquantised layer: e4m3 rounds a value by at
    # most 2^-4 of itself, so each gradient is within (2 2^-4 + 2^-8) of the
    # sum of magnitudes of its terms, plus the product's own bound
    M, N, K, h = 20, 24, 40, 1e-3
    x, w, c = (draw(r, k, s, spread=0.3).double() for r, k, s in ((M, K, 1), (N, K, 2), (M, N, 3)))
    xg, wg = x.float().cuda().requires_grad_(), w.float().cuda().requires_grad_()
    (tl.linear_fp8(xg, wg) * c.float().cuda()).sum().backward()
    f = lambda a, b: float(((a @ b.t()) * c).sum())  # noqa: E731
    for p, grad, mag, move in ((x, xg.grad, c.abs() @ w.abs(), lambda d: (x + d, w)),
                               (w, wg.grad, c.abs().t() @ x.abs(), lambda d: (x, w + d))):
        assert grad.dtype == torch.float32 and grad.shape == p.shape
        for i, j in ((0, 0), (p.shape[0] - 1, K - 1), (7, 11)):
            d = torch.zeros_like(p)
            d[i, j] = h
            diff = (f(*move(d)) - f(*move(-d))) / (2 * h)
            assert abs(float(grad[i, j]) - diff) <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10) * float(mag[i, j])


def test_linear_shapes_strides_and_partial_gradients():
    w = draw(48, 96, 2, torch.float16, 0.3).cuda()
    x3 = draw(10, 96, 1, torch.float16, 0.3).cuda().view(2, 5, 96)
    y = tl.linear_fp8(x3, w)
    assert y.shape == (2, 5, 48) and y.dtype == torch.float16 and not y.requires_grad
    assert torch.equal(y.reshape(10, 48), tl.linear_fp8(x3.reshape(10, 96), w))
    assert torch.equal(tl.linear_fp8(x3[1, 2], w), y[1, 2])
    # column-major x and w, every other row of x
    xt = x3.reshape(10, 96).t().contiguous().t()
    assert torch.equal(tl.linear_fp8(xt, w.t().contiguous().t()), y.reshape(10, 48))
    assert torch.equal(tl.linear_fp8(x3[:, ::2], w), y[:, ::2])
    # a broadcast gradient, and one input only
    for need_x, need_w in ((True, False), (False, True), (True, True)):
        a, b = x3.clone().requires_grad_(need_x), w.clone().requires_grad_(need_w)
        tl.linear_fp8(a, b).sum().backward()
        assert (a.grad is not None) == need_x and (b.grad is not None) == need_w
        if need_x and need_w:
            both = a.grad, b.grad
    a, b = x3.clone().requires_grad_(), w.clone().requires_grad_()
    tl.linear_fp8(a, b).backward(torch.ones(2, 5, 48, dtype=torch.float16, device="cuda"))
    assert torch.equal(a.grad, both[0]) and torch.equal(b.grad, both[1])
    # a broadcast x: every row the same memory
    assert torch.equal(tl.linear_fp8(x3[0, :1].expand(7, 96), w), y[0, :1].expand(7, 48))
    with pytest.raises(ValueError):
        tl.linear_fp8(x3, w[:, :95])
    with pytest.raises(ValueError):
        tl.linear_fp8(x3, w.cpu())
    # parameters that want gradients, where none are recorded
    a, b = x3.clone().requires_grad_(), w.clone().requires_grad_()
    with torch.no_grad():
        z = tl.linear_fp8(a, b)
    assert torch.equal(z, y) and not z.requires_grad
    # second derivatives are refused, not wrong
    (gx,) = torch.autograd.grad(tl.linear_fp8(a, b).float().square().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_linear_without_rows():
    w = draw(48, 96, 2, torch.bfloat16).cuda().requires_grad_()
    x = torch.zeros(0, 96, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = tl.linear_fp8(x, w)
    assert y.shape == (0, 48)
    y.backward(torch.zeros_like(y))
    assert x.grad.shape == (0, 96) and (w.grad == 0).all() and w.grad.shape == w.shape


def test_linear_step_replayed_from_a_graph():
    M, N, K = 130, 90, 200
    x = draw(M, K, 1, torch.bfloat16, 0.5).cuda().requires_grad_()
    w = draw(N, K, 2, torch.bfloat16, 0.5).cuda().requires_grad_()
    gy = draw(M, N, 3, torch.bfloat16, 0.5).cuda()

    def step():
        y = tl.linear_fp8(x, w)
        return (y.detach(),) + torch.autograd.grad(y, (x, w), gy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for r in range(4):
        with torch.no_grad():
            x.mul_(-1.5)
            gy.add_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(p, q) for p, q in zip(held, want)), r


def test_linear_refuses_forward_mode():
    x, w = draw(20, 40, 1).cuda(), draw(30, 40, 2).cuda()
    want = tl.linear_fp8(x, w)
    ad = torch.autograd.forward_ad
    with ad.dual_level():
        assert torch.equal(tl.linear_fp8(x, w), want)
        for a, b in ((ad.make_dual(x, torch.ones_like(x)), w), (x, ad.make_dual(w, torch.ones_like(w)))):
            with pytest.raises(NotImplementedError):
                tl.linear_fp8(a, b)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                tl.linear_fp8(a, b)
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda t: tl.linear_fp8(t, w), (x,), (x,))


# ---- special values of the 16-bit types, other types of the layer, long rows ----

@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_every_pattern_of_16_bits(dtype, fmt, block):
    # in order (a block's values are alike: borders of scales, subnormals, all of
    # a block NaN or infinite) and mixed
    bits = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16)
    mixed = bits[torch.randperm(2 ** 16, generator=torch.Generator().manual_seed(1))]
    small = mixed[(mixed.int() & 0x7FFF) < 0x0400]  # the smallest: subnormals and zeros among them
    for x in (bits.view(512, 128), mixed.view(512, 128), mixed[:65520].view(252, 260), small[:2040].view(15, 136)):
        x = x.contiguous().view(dtype)
        q, s, qt, st = tl.quantize_fp8(x.cuda(), dtype=FMT[fmt], block=block, transpose=True)
        check_image(host(x), fmt, block, q, s)
        check_image(np.ascontiguousarray(host(x).T), fmt, block, qt, st)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_16_bit_borders(dtype, fmt):
    # a block's largest value on the largest of the format times 2^k, next above
    # and next below, beside values that end halfway between two of the format
    top, t = ref.TABLE[fmt][-1], ref.TABLE[fmt]
    rows = []
    for k in (-100, -40, -16, -8, -3, 0, 5) if dtype == torch.bfloat16 else (-20, -16, -8, -3, 0):
        if top * 2.0 ** k > torch.finfo(dtype).max:
            continue
        big = torch.tensor([top * 2.0 ** k], dtype=dtype).view(torch.int16)
        for step in (-1, 0, 1):
            v = float((big + step).view(dtype))
            mids = np.concatenate([(t[:-1] + t[1:]) / 2, t])[:127] * 2.0 ** k
            rows.append(np.concatenate([[v], np.minimum(mids, abs(v)), np.zeros(127 - len(mids))]))
    x = torch.from_numpy(np.array(rows)).to(dtype)
    q, s, qt, st = tl.quantize_fp8(x.cuda(), dtype=FMT[fmt], transpose=True)
    check_image(host(x), fmt, "row", q, s)
    check_image(np.ascontiguousarray(host(x).T), fmt, "row", qt, st)


@pytest.mark.parametrize("xd,wd", [(torch.float32, torch.float32), (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.bfloat16), (torch.float16, torch.bfloat16)])
@pytest.mark.parametrize("M,N,K", [(5, 130, 257), (300, 520, 390), (900, 700, 1100)])
def test_linear_of_other_types(M, N, K, xd, wd):
    # values that every type holds in full; results are the bfloat16 ones, and over
    # all elements within one rounding of them, which a lost slice would exceed
    x, w, gy = (draw(r, c, s, torch.float32, 0.3).to(xd if s != 2 else wd) for r, c, s in ((M, K, 1), (N, K, 2), (M, N, 3)))
    want = linear_reference(host(x), host(w), host(gy))
    xg, wg = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = tl.linear_fp8(xg, wg)
    dx, dw = torch.autograd.grad(y, (xg, wg), gy.cuda())
    for got, dtype, (ref_, mag), k in zip((y, dx, dw), (xd, xd, wd), want, (K, N, M)):
        assert got.dtype == dtype and torch.equal(got, got.bfloat16().to(dtype))
        err = np.abs(host(got) - ref_)
        assert (err <= ref.gemm_bound(ref_, mag, k)).all()
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(ref_)


def check_on_gpu(c, a, sa, b, sb, K):
    def v(q, s):
        e = (s.contiguous().view(torch.uint8).double() - 127).t().repeat_interleave(128, 1)[:, :K]
        return q.double() * torch.exp2(e)
    av, bv = v(a, sa), v(b, sb)
    want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    off = (2.0 ** -10 + (K / 8 + 16) * 2.0 ** -24) * mag
    c = c.double()
    assert bool(((c - want).abs() <= 2.0 ** -8 * (want.abs() + off) + off).all())
    assert float((c - want).norm()) <= 2.0 ** -8 * float(want.norm())


def test_gemm_random_shapes_over_all_elements():
    # over all elements a rounding is 0.42 2^-8 of the norm; one element lost of a
    # row of 4096 adds 2^-6
    import random
    r = random.Random(11)
    for i in range(40):
        M, N, K = (max(1, int(2 ** r.uniform(0, top))) for top in (11.5, 11.5, 12))
        a, sa = tl.quantize_fp8(draw(max(M, 4), K, i, spread=0.3).cuda()[:M], dtype=FMT[r.choice(["e4m3", "e5m2"])])
        b, sb = tl.quantize_fp8(draw(max(N, 40), K, i + 100, spread=0.3).cuda())
        print(M, max(N, 40), K, flush=True)
        check_on_gpu(tl.gemm_fp8(a, sa, b, sb), a, sa, b, sb, K)


@pytest.mark.parametrize("M,N,K", [(1, 50257, 300), (1, 17000, 4200), (16, 33000, 700), (33, 16400, 1030), (20000, 2, 1300)])
def test_gemm_few_rows_and_many_columns(M, N, K):
    a, sa = tl.quantize_fp8(draw(M, K, 1, spread=0.3).cuda())
    b, sb = tl.quantize_fp8(draw(N, K, 2, spread=0.3).cuda())
    c = tl.gemm_fp8(a, sa, b, sb)
    check_on_gpu(c, a, sa, b, sb, K)
    assert torch.equal(tl.gemm_fp8(a.contiguous(), sa, b.contiguous(), sb), c)


@pytest.mark.parametrize("K", [1000, 1023, 1025, 2049, 4095, 4097, 4100])
@pytest.mark.parametrize("M,N", [(5, 100), (20, 300), (300, 1400), (1900, 1990), (3500, 3600)])
def test_gemm_counts_the_last_elements_once(M, N, K):
    one = torch.ones((N, K), device="cuda").to(FMT["e4m3"])
    sb = torch.full((-(-K // 128), -(-N // 16) * 16), 127, dtype=torch.uint8, device="cuda")[:, :N]
    sa = torch.full((-(-K // 128), -(-M // 16) * 16), 127, dtype=torch.uint8, device="cuda")[:, :M]
    for count in (1, 2, 17, 130):
        a = torch.zeros((M, K), device="cuda")
        a[:, K - count:] = 1
        a[::2, 0] = -1  # and the first
        want = torch.full((M, N), float(count), device="cuda")
        want[::2] -= 1
        a = a.to(FMT["e4m3"])
        assert torch.equal(tl.gemm_fp8(a, sa, one, sb), want.bfloat16()), count
        ld = -(-K // 128) * 128
        ap, bp = (torch.full((r, ld), 0x7F, dtype=torch.uint8, device="cuda") for r in (M, N))  # NaN behind the rows
        ap[:, :K], bp[:, :K] = a.view(torch.uint8), one.view(torch.uint8)
        assert torch.equal(tl.gemm_fp8(ap.view(a.dtype)[:, :K], sa, bp.view(a.dtype)[:, :K], sb), want.bfloat16()), count
