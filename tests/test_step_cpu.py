"""CPU: argument checks of the feed-forward block, the cross entropy and clipping,
their buffers' sizes, and the pins of their plain forms."""
import ctypes

import pytest
import torch

import step_ref as ref

tl = pytest.importorskip("tiled_software_pipelined_amd.lib")
P = ctypes.c_void_p
A = P(256)


def d(v, w):
    return w if v is None else v


def fwd(M=4, K=8, F=16, N=8, dtype=1, act=0, x=A, ldx=None, wg=A, ldg=None, wu=A, ldu=None, wd=A, ldd=None, y=A, ldy=None, keep=15,
        saved=A, scratch=A):
    return tl._lib.tgemm_ffn_forward(M, K, F, N, dtype, act, x, d(ldx, K), wg, d(ldg, K), wu, d(ldu, K), wd, d(ldd, F), y,
                                     d(ldy, N), keep, saved, scratch, None)


def bwd(M=4, K=8, F=16, N=8, dtype=1, act=0, x=A, ldx=None, wg=A, ldg=None, wu=A, ldu=None, wd=A, ldd=None, dy=A, lddy=None, keep=15,
        saved=A, dx=A, lddx=None, dg=A, lddg=None, du=A, lddu=None, dd=A, lddd=None, scratch=A):
    return tl._lib.tgemm_ffn_backward(M, K, F, N, dtype, act, x, d(ldx, K), wg, d(ldg, K), wu, d(ldu, K), wd, d(ldd, F), dy,
                                      d(lddy, N), keep, saved, dx, d(lddx, K), dg, d(lddg, K), du, d(lddu, K), dd, d(lddd, F),
                                      scratch, None)


COMMON = [
    (dict(M=-1), -1), (dict(M=2 ** 30 + 1), -1), (dict(K=2 ** 22 + 1), -1), (dict(F=-3), -1), (dict(N=2 ** 40), -1), (dict(keep=16), -1),
    (dict(keep=-1), -1), (dict(dtype=0), -1), (dict(dtype=2), -1), (dict(act=-1), -1), (dict(act=4), -1), (dict(ldx=7), -1),
    (dict(ldg=7), -1), (dict(ldu=7), -1), (dict(ldd=15), -1), (dict(ldx=2 ** 22 + 1), -1), (dict(ldd=2 ** 62), -1), (dict(x=None), -2),
    (dict(wg=None), -2), (dict(wu=None), -2), (dict(wd=None), -2), (dict(saved=None), -2), (dict(scratch=None, keep=1), -2), (dict(x=P(257)), -3),
    (dict(wd=P(3)), -3), (dict(saved=P(128)), -3), (dict(scratch=P(64)), -3)]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(y=None), -2), (dict(ldy=7), -1), (dict(y=P(1)), -3)])
def test_ffn_forward_refuses(kw, code):
    assert fwd(**kw) == code and tl.last_error()


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), -2), (dict(lddy=7), -1), (dict(dx=None), -2), (dict(dg=None), -2), (dict(du=None), -2), (dict(dd=None), -2),
    (dict(lddx=7), -1), (dict(lddd=15), -1), (dict(du=P(1)), -3)])
def test_ffn_backward_refuses(kw, code):
    assert bwd(**kw) == code and tl.last_error()


def test_ffn_sizes():
    n = (ctypes.c_int64 * 3)()
    assert tl._lib.tgemm_ffn_bytes(4, 8, 16, 8, 15, None) == -2
    assert tl._lib.tgemm_ffn_bytes(4, 8, 2 ** 23, 8, 15, n) == -1
    assert tl._lib.tgemm_ffn_bytes(100, 64, 1000, 64, 0, n) == 0 and n[0] == 0 and n[1] >= 2 * 100 * 1000 and n[2] == 0
    assert tl._lib.tgemm_ffn_bytes(100, 64, 1000, 64, 15, n) == 0 and n[0] == 3 * 2 * 100 * 1024 and n[2] >= 2 * 200000
    assert tl._lib.tgemm_ffn_bytes(100, 64, 1000, 64, tl.FFN_DOWN, n) == 0 and n[0] == 2 * 100 * 1024  # h alone is kept, rows of whole lines
    assert tl._lib.tgemm_ffn_bytes(0, 64, 1000, 64, 15, n) == 0
    assert tl._lib.tgemm_ffn_bytes(2 ** 30, 2 ** 22, 2 ** 22, 2 ** 22, 1, n) == 0 and min(n) > 2 ** 52


def test_bytes_kept_for_the_backward_pass():
    """Six for each token and inner unit where a gradient passes the activation, two for w_down's alone."""
    for keep in range(16):
        assert tl._ffn_bytes(100, 64, 1000, 72, keep)[0] == max(1, (6 if keep & 7 else 2 if keep else 0) * 100 * 1024)


@pytest.mark.parametrize("kw", [dict(M=0, N=0), dict(M=0)])
def test_ffn_of_no_rows_needs_no_device(kw):
    assert fwd(**kw, x=None, y=None, keep=0, saved=None) == 0 and tl.last_error() == ""


def xf(M=4, V=32, K=8, dtype=1, x=A, ldx=None, w=A, ldw=None, target=A, ignore=-100, reduction=2, keep=0, loss=A, saved=A, scratch=A):
    return tl._lib.tgemm_xent_forward(M, V, K, dtype, x, d(ldx, K), w, d(ldw, K), target, ignore, reduction, keep, loss, saved, scratch,
                                      None)


def xb(M=4, V=32, K=8, dtype=1, x=A, ldx=None, w=A, ldw=None, target=A, reduction=2, dloss=A, saved=A, keep=3, dx=A, lddx=None, dw=A,
       lddw=None, scratch=A):
    return tl._lib.tgemm_xent_backward(M, V, K, dtype, x, d(ldx, K), w, d(ldw, K), target, reduction, dloss, saved, keep, dx,
                                       d(lddx, K), dw, d(lddw, K), scratch, None)


XCOMMON = [
    (dict(M=-1), -1), (dict(M=2 ** 30 + 1), -1), (dict(V=2 ** 30 + 1), -1), (dict(V=-1), -1), (dict(K=2 ** 22 + 1), -1), (dict(dtype=0), -1),
    (dict(reduction=3), -1), (dict(reduction=-1), -1), (dict(ldx=7), -1), (dict(ldw=7), -1), (dict(ldw=2 ** 23), -1), (dict(x=None), -2),
    (dict(w=None), -2), (dict(target=None), -2), (dict(target=P(4)), -3), (dict(x=P(1)), -3), (dict(w=P(1)), -3), (dict(saved=None), -2),
    (dict(saved=P(8)), -3), (dict(scratch=None), -2), (dict(scratch=P(8)), -3)]


@pytest.mark.parametrize("kw,code", XCOMMON + [
    (dict(loss=None), -2), (dict(loss=P(2)), -3), (dict(keep=4), -1), (dict(keep=8, V=2 ** 28 + 1), -1)])
def test_xent_forward_refuses(kw, code):
    assert xf(**kw) == code and tl.last_error()


@pytest.mark.parametrize("kw,code", XCOMMON + [
    (dict(keep=4), -1), (dict(dloss=None), -2), (dict(dloss=P(2)), -3), (dict(dx=None), -2), (dict(dw=None), -2), (dict(lddx=7), -1),
    (dict(lddw=7), -1), (dict(dw=P(1)), -3)])
def test_xent_backward_refuses(kw, code):
    assert xb(**kw) == code and tl.last_error()


def test_xent_sizes():
    n = (ctypes.c_int64 * 3)()
    assert tl._lib.tgemm_xent_bytes(4, 8, 16, 3, None) == -2 and tl._lib.tgemm_xent_bytes(4, 8, 16, 4, n) == -1
    for M, V, K in ((8192, 128256, 4096), (1, 2 ** 30, 64), (2 ** 20, 50000, 64), (0, 10, 8), (10, 0, 8), (7, 9, 0)):
        assert tl._lib.tgemm_xent_bytes(M, V, K, 3, n) == 0
        # dz: at most 512 MB or 16 KB a row, never all of a large M V (rows up to a multiple of 64); x gathered; dx's
        # float sums; 64 MB of shared tiles
        rows = M + 63
        assert n[2] <= max(2 ** 29 * rows // max(M, 1), 2 ** 14 * rows) + 512 * rows + 2 * rows * (K + 64) + 4 * M * K + 2 ** 26 + 2 ** 20
    one = n[0], n[1]
    assert tl._lib.tgemm_xent_bytes(7, 9, 0, 0, n) == 0 and (n[0], n[1], n[2]) == (*one, 0)
    # kept powers: rows of whole lines, 16 bits each, and what the loss's rows were joined from
    assert tl._lib.tgemm_xent_bytes(100, 1000, 64, 8 + 3, n) == 0 and 2 * 100 * 1024 < n[0] < 2 * 100 * 1024 + 2 ** 15
    assert tl._lib.tgemm_xent_bytes(4, 2 ** 28 + 1, 16, 8, n) == -1 and tl._lib.tgemm_xent_bytes(0, 9, 8, 11, n) == 0


MOST_ROWS = 2 ** 26 - 128


@pytest.mark.parametrize("call", [
    lambda: fwd(M=2 ** 30, F=2 ** 20), lambda: fwd(M=2 ** 30, F=8, N=2 ** 22, keep=0), lambda: fwd(M=2 ** 20, K=2 ** 22, F=2 ** 22, N=8, keep=2),
    lambda: bwd(M=2 ** 30, F=2 ** 20), lambda: bwd(M=2 ** 20, K=2 ** 22, F=2 ** 22, keep=2), lambda: bwd(M=2 ** 30, K=2 ** 22, keep=1),
    lambda: xf(M=MOST_ROWS, V=2 ** 20), lambda: xf(M=2 ** 20, V=2 ** 30), lambda: xf(M=MOST_ROWS, V=2 ** 28, keep=8), lambda: xf(M=MOST_ROWS + 1),
    lambda: xb(M=MOST_ROWS, V=2 ** 20, keep=11), lambda: xb(M=2 ** 24, V=9000, K=2 ** 22, keep=1), lambda: xb(M=2 ** 26, V=8)])
def test_launches_that_no_grid_holds_are_refused_first(call):
    """Before the device is looked at, and so before anything is queued."""
    assert call() == -1 and ("too many tiles" in tl.last_error() or "out of range" in tl.last_error())


def test_launches_that_a_grid_holds():
    """Without a device the calls end where it is looked for, with their arguments found right."""
    n = (ctypes.c_int64 * 3)()
    assert tl._lib.tgemm_xent_bytes(MOST_ROWS, 64, 8, 3, n) == 0 and tl._lib.tgemm_xent_bytes(MOST_ROWS + 1, 64, 8, 3, n) == -1
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    calls = [lambda: xf(M=MOST_ROWS, V=64), lambda: xb(M=MOST_ROWS, V=64), lambda: xf(M=1, V=2 ** 30, K=7), lambda: xb(M=1, V=2 ** 30, K=7),
             lambda: xf(M=800, V=2 ** 27, K=7), lambda: fwd(M=2 ** 28, K=7, F=8, N=8), lambda: bwd(M=2 ** 28, K=7, F=8, N=8)]
    codes = {c() for c in calls}
    assert len(codes) == 1 and -1 not in codes


def clip(tensors=2, counts=(5, 7), dtypes=(0, 1), ins=(64, 128), outs=(64, 128), max_norm=1.0, eps=1e-6, norm=A, ws=A, size=1 << 20):
    p = lambda v: None if v is None else (P * len(v))(*v)  # noqa: E731
    return tl._lib.tgemm_clip(tensors, p(ins), p(outs), (ctypes.c_int64 * len(counts))(*counts), (ctypes.c_int32 * len(dtypes))(*dtypes),
                              max_norm, eps, norm, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tensors=-1), -1), (dict(counts=(5, -1)), -1), (dict(counts=(2 ** 40, 1)), -1), (dict(max_norm=-1.0), -1),
    (dict(max_norm=float("nan")), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(dtypes=(0, 2)), -1),
    (dict(dtypes=(0, 9)), -1), (dict(size=8), -1), (dict(norm=None), -2), (dict(ws=None), -2), (dict(ins=None), -2), (dict(outs=None), -2),
    (dict(ins=(64, None)), -2), (dict(outs=(None, 128)), -2), (dict(ins=(66, 128)), -3), (dict(outs=(64, 129)), -3), (dict(norm=P(2)), -3),
    (dict(ws=P(8)), -3)])
def test_clip_refuses(kw, code):
    assert clip(**kw) == code and tl.last_error()


@pytest.mark.parametrize("kw", [
    dict(ins=(64, 80), outs=(64, 80)), dict(ins=(80, 64), outs=(80, 64), counts=(7, 9)), dict(ins=(64, 128), outs=(64, 140), counts=(32, 7)),
    dict(ins=(64, 128), outs=(140, 200), counts=(5, 7)), dict(ins=(64, 128), outs=(256, 272)), dict(ins=(64, 128), outs=(60, 128)),
    dict(tensors=3, ins=(64, 1024, 4096), outs=(64, 1024, 4096), counts=(2000, 1, 1), dtypes=(1, 1, 1))])
def test_clip_refuses_tensors_that_share_elements(kw):
    assert clip(**kw) == -1 and "overlap" in tl.last_error()


@pytest.mark.parametrize("kw", [
    dict(ins=(64, 84), outs=(64, 84)), dict(ins=(64, 78), outs=(1024, 2048), dtypes=(1, 1)), dict(ins=(64, 64), outs=(1024, 64), counts=(5, 0)),
    dict(ins=(64, 128), outs=(128 + 16, 64 + 20))])
def test_clip_takes_neighbours_and_inputs_that_share_elements(kw):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert clip(**kw) == clip() != -1 and "overlap" not in tl.last_error()


def test_clip_sizes():
    c = lambda *v: tl._lib.tgemm_clip_workspace_bytes(len(v), (ctypes.c_int64 * len(v))(*v))  # noqa: E731
    assert c() == 256 and c(0) == 256 and c(1) == 264 and c(8192, 0, 8193) == 256 + 8 * 3 and c(-1) == -1 and c(2 ** 41) == -1
    assert c(2 ** 40) <= 256 + 8 * 16385
    assert tl._lib.tgemm_clip_workspace_bytes(1, None) == -1


def test_binding_refuses_before_any_launch():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    x, wg, wd, t = b(4, 8), b(16, 8), b(8, 16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        tl.gated_ffn(x, wg, wg, wd)
    with pytest.raises(TypeError, match="float32"):
        tl.gated_ffn(x.float(), wg, wg, wd)
    with pytest.raises(ValueError, match="activation"):
        tl.gated_ffn(x, wg, wg, wd, activation="tanh")
    with pytest.raises(ValueError, match="GPU"):
        tl.linear_cross_entropy(x, wg, t)
    with pytest.raises(ValueError, match="reduction"):
        tl.linear_cross_entropy(x, wg, t, reduction="batch")
    with pytest.raises(TypeError, match="int64|float32"):
        tl.linear_cross_entropy(x.float(), wg, t)
    for grads, error in (([], ValueError), ([x], ValueError)):
        with pytest.raises(error):
            tl.clip_grad_norm(grads, 1.0)
    for limit in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="max_norm"):
            tl.clip_grad_norm([x], limit)
    with pytest.raises(ValueError, match="out"):
        tl.clip_grad_norm([x], 1.0, out=[])
    meta = torch.empty(4, 8, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="GPU"):
        tl.gated_ffn(meta, wg, wg, wd)


def test_dense():
    t = torch.zeros(2, 3, 4, 5)
    assert tl._dense(t) and tl._dense(t.permute(2, 0, 3, 1)) and tl._dense(t[:0]) and tl._dense(torch.zeros(()))
    assert tl._dense(t.to(memory_format=torch.channels_last)) and tl._dense(t[:1]) and tl._dense(t[1])
    assert not tl._dense(t[:, :, :, :4]) and not tl._dense(t[:, 1:]) and not tl._dense(torch.zeros(1).expand(5))
    assert not tl._dense(t.transpose(0, 1)[1])


def test_package_names():
    import tiled_software_pipelined_amd as pkg
    assert all(getattr(pkg, n) is getattr(tl, n) for n in ("gated_ffn", "linear_cross_entropy", "clip_grad_norm"))


@pytest.mark.parametrize("name", list(tl.ACTIVATIONS))
def test_plain_activations(name):
    """The oracle's activations and slopes against torch's own and against differences."""
    g = torch.linspace(-8, 8, 4001, dtype=torch.float64) + 1e-4
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
    a, slope, second = ref.act(g, name)
    assert torch.allclose(a, f(g), rtol=1e-12, atol=1e-13)
    h = 1e-5
    assert torch.allclose(slope, (f(g + h) - f(g - h)) / (2 * h), atol=1e-8)
    assert ((ref.act(g + h, name)[1] - ref.act(g - h, name)[1]) / (2 * h)).abs().max() <= second + 1e-6


def test_plain_forms_agree_with_autograd():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).half()  # noqa: E731
    leaves, dy = [r(7, 6), r(9, 6), r(9, 6), r(5, 9)], r(7, 5)
    want = ref.ffn(*leaves, "gelu", dy)
    x, wg, wu, wd = wide = [t.double().requires_grad_() for t in leaves]
    y = (torch.nn.functional.gelu(x @ wg.t()) * (x @ wu.t())) @ wd.t()
    grads = torch.autograd.grad(y, wide, dy.double())
    for name, v in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y, *grads)):
        assert torch.allclose(want[name][0], v, rtol=1e-10, atol=1e-10)
    x, w, t = r(8, 6), r(11, 6), torch.tensor([0, 3, -100, 10, 5, 5, -100, 1])
    for how in ("mean", "sum", "none"):
        by = torch.linspace(-1, 2, 8).double() if how == "none" else 0.7
        want = ref.xent(x, w, t, reduction=how, dloss=by)
        wide = [v.double().requires_grad_() for v in (x, w)]
        loss = torch.nn.functional.cross_entropy(wide[0] @ wide[1].t(), t, reduction=how)
        grads = torch.autograd.grad(loss, wide, torch.as_tensor(by, dtype=torch.float64).expand(loss.shape))
        for name, v in zip(("loss", "dx", "dw"), (loss, *grads)):
            assert torch.allclose(want[name][0], v, rtol=1e-10, atol=1e-10)


def test_bounds_reject_a_planted_mistake():
    """The bounds are tight enough to see one wrong term among many (planted here, in the plain form's place)."""
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731
    x, w, t = r(16, 64), (r(200, 64).float() / 8).bfloat16(), torch.randint(0, 200, (16,), generator=g)
    want = ref.xent(x, w, t, dloss=1.0)
    ref.check({k: v for k, (v, _) in want.items()}, want)
    short = ref.xent(x[:, :63], w[:, :63], t, dloss=1.0)
    with pytest.raises(AssertionError):
        ref.check({"loss": short["loss"][0]}, want, ("loss",))
    wrong = ref.xent(x, w, (t + 1) % 200, dloss=1.0)
    for name in ("dx", "dw"):
        with pytest.raises(AssertionError):
            ref.check({name: wrong[name][0]}, want, (name,))
