"""GPU: the cross entropy of a linear layer's logits against a plain form in 64 bits."""
import pytest
import torch

import step_ref as ref

tl = pytest.importorskip("tiled_software_pipelined_amd.lib")
pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]


def make(M, V, K, dtype, seed=0, ignored=0.25, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7919 * M + 31 * K + V)
    x = (torch.randn((M, K), generator=g, device="cuda") * scale).to(dtype)
    w = (torch.randn((V, K), generator=g, device="cuda") / max(K, 1) ** 0.5).to(dtype)
    target = torch.randint(0, max(V, 1), (M,), generator=g, device="cuda")
    gone = torch.rand((M,), generator=g, device="cuda") < ignored
    if M:
        gone[0] = False
    return x, w, torch.where(gone, -100, target)


def run(x, w, target, dloss=1.0, reduction="mean", ignore=-100, **kw):
    x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    loss = tl.linear_cross_entropy(x, w, target, ignore, reduction, **kw)
    g = torch.as_tensor(dloss, dtype=torch.float32, device=x.device).expand(loss.shape)
    dx, dw = torch.autograd.grad(loss, (x, w), g)
    return {"loss": loss.detach(), "dx": dx, "dw": dw}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,V,K", [
    (1, 1, 1), (1, 2, 3), (2, 7, 5), (1, 1000, 64), (5, 129, 16), (64, 128, 64), (65, 127, 66), (33, 1000, 100), (130, 513, 200),
    (200, 3001, 72), (700, 300, 520), (2050, 4100, 40), (3, 50257, 24), (515, 2049, 1000), (4100, 5, 9)])
def test_sizes(M, V, K, dtype):
    x, w, t = make(M, V, K, dtype)
    ref.check(run(x, w, t, 3.0), ref.xent(x, w, t, dloss=3.0))
    with torch.no_grad():
        ref.check({"loss": tl.linear_cross_entropy(x, w, t)}, ref.xent(x, w, t))


@pytest.mark.parametrize("M,V,K,dtype", [
    (1000, 30001, 520, torch.bfloat16), (4100, 9001, 1032, torch.float16), (2050, 33000, 264, torch.bfloat16),
    (9000, 33001, 72, torch.float16), (40000, 9000, 136, torch.bfloat16), (1024, 2048, 1024, torch.float16),
    (1030, 4100, 2056, torch.bfloat16), (800, 1001, 333, torch.float16), (4200, 777, 90, torch.bfloat16)])
def test_large_sizes(M, V, K, dtype):
    """Every tile of every product, one piece of the vocabulary and several, weights copied to lines."""
    x, w, t = make(M, V, K, dtype)
    ref.check(run(x, w, t, 100.0), ref.xent(x, w, t, dloss=100.0))


@pytest.mark.parametrize("M,V", [(1, 4200001), (3, 4194560)])
def test_a_few_rows_and_millions_of_words(M, V):
    """dz in pieces although it is small: its 64 rows are read by 32-bit offsets."""
    x, w, t = make(M, V, 8, torch.bfloat16, ignored=0.0)
    assert tl._xent_bytes(M, V, 8, 3)[2] < 2 ** 30
    ref.check(run(x, w, t), ref.xent(x, w, t, dloss=1.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_reductions(reduction, dtype):
    x, w, t = make(150, 700, 96, dtype, ignored=0.5)
    g = torch.linspace(-2, 3, 150, device="cuda") if reduction == "none" else 0.3
    ref.check(run(x, w, t, g, reduction), ref.xent(x, w, t, reduction=reduction, dloss=g))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2.0 ** -30, 1e-6, 65536.0, 2.0 ** 40])
def test_gradients_of_scaled_losses(size, dtype):
    """The loss's own gradient may be of any size: results keep their digits as far as their type goes."""
    x, w, t = make(70, 300, 64, dtype)
    got, want = run(x, w, t, size), ref.xent(x, w, t, dloss=size)
    for k in ("dx", "dw"):
        top = torch.finfo(dtype).max
        fits = want[k][0].abs() < top / 2
        over = want[k][0].abs() > top * 2
        assert ((got[k].double() - want[k][0]).abs() <= want[k][1])[fits].all() and got[k][over].isinf().all()


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("dloss", [1.9, -1.1, 1000.3])
def test_the_losses_factor_is_not_rounded(dloss, reduction):
    """Of 256 words as likely as each other, p - 1 and p hold in bfloat16: dx is rounded once, not by a factor that
    is common to all rows as well."""
    M, V, K = 60, 256, 40
    x, w, t = make(M, V, K, torch.bfloat16, ignored=0.0)
    got = run(torch.zeros_like(x), w, t, dloss, reduction)["dx"].double()
    c = float(torch.tensor(dloss, dtype=torch.float32)) / (M if reduction == "mean" else 1)
    p = torch.full((M, V), 2.0 ** -8, dtype=torch.float64, device="cuda")
    p[torch.arange(M), t] -= 1
    want, size = c * (p @ w.double()), abs(c) * (p.abs() @ w.double().abs())
    assert ((got - want).abs() <= 2.0 ** -8 * 1.001 * want.abs() + (V + 20) * 2.0 ** -24 * size).all()


def test_small_probabilities_in_float16():
    """dw rows of unlikely words come from probabilities around 2^-23, below float16's normal numbers."""
    K, V, M = 64, 2000, 90
    x, w, t = make(M, V, K, torch.float16, ignored=0.0)
    x[:, 0], w[:, 0] = 4.0, -4.0
    w[0, 0] = 0.0
    t[:] = 0
    want = ref.xent(x, w, t, reduction="sum", dloss=1024.0)
    got = run(x, w, t, 1024.0, "sum")
    ref.check(got, want)
    small = want["dw"][0][1:]
    p = torch.softmax(x.double() @ w.double().t(), 1)[:, 1:]
    assert p.max() < 2.0 ** -14 and p.median() < 2.0 ** -22
    # the roundings of dz and of dw are 2^-11 of each value
    assert (got["dw"].double()[1:] - small).norm() / small.norm() < 2e-3


@pytest.mark.parametrize("scale", [0.0, 1e-3, 30.0, 300.0])
def test_flat_and_peaked_rows(scale):
    x, w, t = make(140, 600, 128, torch.bfloat16, scale=scale)
    ref.check(run(x, w, t), ref.xent(x, w, t, dloss=1.0))


def test_rows_that_do_not_count():
    x, w, t = make(300, 500, 64, torch.bfloat16, ignored=0.6)
    x[t == -100] = float("nan")  # whatever they hold
    t[1] = -100
    x[1] = float("inf")
    got = run(x, w, t)
    keep = t != -100
    want = ref.xent(x[keep], w, t[keep], dloss=1.0)
    ref.check({**got, "dx": got["dx"][keep]}, want)
    assert not got["dx"][~keep].any()
    clean = torch.where(keep[:, None], x, 1.0)
    again = run(clean, w, t)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_no_row_counts():
    x, w, t = make(40, 100, 32, torch.float16)
    t[:] = -100
    got = run(x, w, t)
    assert got["loss"].isnan() and not got["dx"].any() and not got["dw"].any()
    assert run(x, w, t, reduction="sum")["loss"] == 0 and not run(x, w, t, 1.0, "none")["loss"].any()


@pytest.mark.parametrize("ignore", [0, 7, -1, 2 ** 40])
def test_other_ignore_indices(ignore):
    x, w, t = make(60, 90, 40, torch.bfloat16, ignored=0.0)
    t[::3] = ignore
    ref.check(run(x, w, t, ignore=ignore), ref.xent(x, w, t, ignore, dloss=1.0))


@pytest.mark.parametrize("bad", [-1, 500, 2 ** 33, -2 ** 62])
def test_targets_outside_the_vocabulary_make_nan(bad):
    x, w, t = make(100, 500, 64, torch.bfloat16, ignored=0.1)
    t[10] = bad
    each = run(x, w, t, 1.0, "none")
    rest = [i for i in range(100) if i != 10]
    assert each["loss"][10].isnan() and each["loss"][rest].isfinite().all()
    assert each["dx"][10].isnan().all() and each["dx"][rest].isfinite().all() and each["dw"].isnan().all()
    assert run(x, w, t)["loss"].isnan()


def test_logits_that_are_not_finite():
    x, w, t = make(80, 200, 64, torch.bfloat16, ignored=0.0)
    x[3, 0] = float("nan")
    x[4, 0] = float("inf")
    got = run(x, w, t, 1.0, "none")
    rest = [i for i in range(80) if i not in (3, 4)]
    assert got["loss"][3].isnan() and not got["loss"][4].isfinite()
    ref.check({"loss": got["loss"][rest], "dx": got["dx"][rest]}, ref.xent(x[rest], w, t[rest], reduction="none", dloss=1.0), ("loss", "dx"))


@pytest.mark.parametrize("M,V", [(0, 10), (5, 0), (0, 0)])
def test_empty_sizes(M, V):
    x, w, t = make(M, V, 16, torch.bfloat16)
    t[:] = -100
    got = run(x, w, t, reduction="sum")
    assert got["loss"] == 0 and got["dx"].shape == x.shape and got["dw"].shape == w.shape
    assert not got["dx"].any() and not got["dw"].any()
    assert run(x, w, t, reduction="none")["loss"].shape == (M,)
    x0, w0, t0 = make(6, 9, 0, torch.bfloat16)  # no features: every word as likely
    ref.check(run(x0, w0, t0), ref.xent(x0, w0, t0, dloss=1.0))


def test_gradients_against_differences():
    x, w, t = make(7, 11, 6, torch.float16)
    got, bounds = run(x, w, t), ref.xent(x, w, t, dloss=1.0)
    wide = [x.double().cpu(), w.double().cpu()]
    keep = (t != -100).cpu()

    def value():
        z = (wide[0] @ wide[1].t())[keep]
        return float((torch.logsumexp(z, 1) - z.gather(1, t.cpu()[keep][:, None])[:, 0]).mean())

    for name, v in zip(("dx", "dw"), wide):
        flat = v.view(-1)
        for i in range(flat.numel()):
            old = flat[i].item()
            flat[i] = old + 1e-5
            up = value()
            flat[i] = old - 1e-5
            down = value()
            flat[i] = old
            assert abs(got[name].double().cpu().reshape(-1)[i].item() - (up - down) / 2e-5) <= bounds[name][1].cpu().reshape(-1)[i].item() + 1e-8


def test_strides_axes_and_single_gradients():
    x, w, t = make(60, 300, 70, torch.bfloat16)
    wide = torch.full((300, 79), float("nan"), dtype=w.dtype, device="cuda")
    wide[:, 3:73] = w
    apart = torch.full((60, 75), float("nan"), dtype=w.dtype, device="cuda")
    apart[:, 1:71] = x
    want = run(x, w, t)
    got = run(apart[:, 1:71], wide[:, 3:73], t)
    assert all(torch.equal(got[k], want[k]) for k in want)
    got = run(x.view(3, 20, 70), w, t.view(3, 20))
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["dx"].view(60, 70), want["dx"])
    got = run(x, w, torch.stack([t, t], 1)[:, 0])  # a target with a stride
    assert torch.equal(got["dw"], want["dw"])
    one = x.detach().requires_grad_()
    assert torch.equal(torch.autograd.grad(tl.linear_cross_entropy(one, w, t), one)[0], want["dx"])
    one = w.detach().requires_grad_()
    assert torch.equal(torch.autograd.grad(tl.linear_cross_entropy(x, one, t), one)[0], want["dw"])
    single = tl.linear_cross_entropy(x[0], w, t[0])
    assert single.shape == () and torch.equal(single, tl.linear_cross_entropy(x[:1], w, t[:1]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_several_pieces_of_the_vocabulary(dtype):
    """More logits than one piece holds: dx is summed over pieces, the last of them partial."""
    M, V, K = 33000, 20001, 24
    x, w, t = make(M, V, K, dtype)
    n = tl._xent_bytes(M, V, K, 3)[2]
    assert n < 2 * M * V
    got = run(x, w, t)
    some = torch.arange(0, M, 97, device="cuda")
    count = int((t != -100).sum())
    want = ref.xent(x[some], w, t[some], reduction="sum", dloss=1.0 / count)
    ref.check({"dx": got["dx"][some]}, want, ("dx",))
    # dw: added up over blocks of rows
    dw, bound = 0.0, 0.0
    for rows in torch.arange(M, device="cuda").split(4096):
        v, b = ref.xent(x[rows], w, t[rows], reduction="sum", dloss=1.0 / count)["dw"]
        dw, bound = dw + v, bound + b
    assert ((got["dw"].double() - dw).abs() <= bound + ref.U[dtype] * dw.abs()).all()
    assert torch.equal(run(x, w, t)["dx"], got["dx"])


@pytest.fixture
def powers(monkeypatch):
    """The powers are kept whatever K is."""
    monkeypatch.setattr(tl, "POWERS_LEAST", 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,V,K", [
    (1, 1, 1), (1, 2, 3), (2, 7, 5), (1, 1000, 64), (5, 129, 16), (64, 128, 64), (65, 127, 66), (33, 1000, 100), (130, 513, 200),
    (2050, 4100, 40), (3, 50257, 24), (4100, 5, 9), (17, 2049, 8), (1030, 6001, 264)])
def test_kept_powers(M, V, K, dtype, powers):
    x, w, t = make(M, V, K, dtype)
    got = run(x, w, t, 3.0)
    ref.check(got, ref.xent(x, w, t, dloss=3.0, kept=True))
    assert torch.equal(run(x, w, t, 3.0, keep_bytes=0)["loss"], got["loss"])


@pytest.mark.parametrize("scale", [0.0, 1e-3, 30.0, 300.0])
@pytest.mark.parametrize("dtype", DTYPES)
def test_kept_powers_of_flat_and_peaked_rows(scale, dtype, powers):
    x, w, t = make(140, 600, 128, dtype, scale=scale)
    for reduction, dloss in (("mean", 1024.0), ("none", torch.linspace(-1, 2, 140, device="cuda"))):
        ref.check(run(x, w, t, dloss, reduction), ref.xent(x, w, t, reduction=reduction, dloss=dloss, kept=True))


def test_kept_powers_of_likely_targets(powers):
    """p - 1 of a target that is nearly certain is not lost to the powers' rounding."""
    x, w, t = make(100, 300, 64, torch.bfloat16, ignored=0.0)
    w[:, 0], x[:, 0] = -4.0, 2.0
    w[5, 0], t[:] = 4.0, 5  # 16 above the others
    want = ref.xent(x, w, t, reduction="sum", dloss=1.0, kept=True)
    got = run(x, w, t, reduction="sum")
    ref.check(got, want)
    p = torch.softmax(x.double() @ w.double().t(), 1)[:, 5]
    assert p.min() > 0.99 and (1 - p).median() < 2.0 ** -9
    row = got["dw"][5].double()  # the sum of (p - 1) x: dz's and dw's roundings are 2^-8 of each value
    assert (row - want["dw"][0][5]).norm() < 2.0 ** -8 * 2 * ((1 - p)[:, None] * x.double().abs()).sum(0).norm()


def test_kept_powers_in_pieces(powers):
    """More logits than one piece of dz holds; a saved state above 2^31 bytes."""
    M, V, K = 33000, 33001, 24
    x, w, t = make(M, V, K, torch.bfloat16)
    assert tl._xent_bytes(M, V, K, 11)[0] > 2 ** 31 and tl._xent_bytes(M, V, K, 11)[2] < 2 ** 30
    got = run(x, w, t)
    some = torch.arange(0, M, 97, device="cuda")
    by = 1.0 / int((t != -100).sum())
    ref.check({"dx": got["dx"][some]}, ref.xent(x[some], w, t[some], reduction="sum", dloss=by, kept=True), ("dx",))
    dw, bound = 0.0, 0.0  # added up over blocks of rows
    for rows in torch.arange(M, device="cuda").split(4096):
        v, b = ref.xent(x[rows], w, t[rows], reduction="sum", dloss=by, kept=True)["dw"]
        dw, bound = dw + v, bound + b
    assert ((got["dw"].double() - dw).abs() <= bound + ref.U[torch.bfloat16] * dw.abs()).all()


@pytest.mark.parametrize("bad", [-1, 500, 2 ** 33])
def test_kept_powers_of_rows_without_a_number(bad, powers):
    x, w, t = make(100, 500, 64, torch.bfloat16, ignored=0.1)
    t[10:13] = torch.tensor([bad, 3, 4], device="cuda")
    x[11, 0], x[12, 0] = float("nan"), float("inf")
    x[t == -100] = float("nan")
    got, rest = run(x, w, t, 1.0, "none"), [i for i in range(100) if i not in (10, 11, 12)]
    assert got["loss"][10].isnan() and got["dx"][10:13].isnan().all() and got["dw"].isnan().all()
    assert got["loss"][rest].isfinite().all() and not got["dx"][t == -100].any()
    keep = [i for i in rest if int(t[i]) != -100]
    want = ref.xent(x[keep], w, t[keep], reduction="none", dloss=1.0, kept=True)
    ref.check({"dx": got["dx"][keep]}, want, ("dx",))


@pytest.mark.parametrize("M,V", [(0, 10), (5, 0), (0, 0)])
def test_kept_powers_of_empty_sizes(M, V, powers):
    x, w, t = make(M, V, 16, torch.bfloat16)
    t[:] = -100
    got = run(x, w, t, reduction="sum")
    assert got["loss"] == 0 and not got["dx"].any() and not got["dw"].any()


def test_kept_powers_serve_a_graph_twice(powers):
    """The backward pass only reads them; single gradients are the same bits."""
    x, w, t = make(120, 700, 96, torch.bfloat16)
    want = run(x, w, t)
    x, w = x.requires_grad_(), w.requires_grad_()
    loss = tl.linear_cross_entropy(x, w, t)
    for inputs, names in (((x, w), ("dx", "dw")), ((x,), ("dx",)), ((w,), ("dw",)), ((x, w), ("dx", "dw"))):
        for g, name in zip(torch.autograd.grad(loss, inputs, retain_graph=True), names):
            assert torch.equal(g, want[name])


def test_kept_powers_captured_and_replayed(powers):
    test_captured_and_replayed()


def test_bytes_that_may_be_kept():
    x, w, t = make(64, 1000, 512, torch.bfloat16)
    bits = {}
    for keep in (0, 2 * 64 * 1024 - 1, 2 * 64 * 1024, float("inf")):
        x.requires_grad_()
        loss = tl.linear_cross_entropy(x, w, t, keep_bytes=keep)
        bits[keep] = loss.grad_fn.saved_tensors[3].numel()
    a, b, c, d = bits.values()
    assert a == b and c == d and c >= a + 2 * 64 * 1024
    with torch.no_grad():
        assert torch.equal(tl.linear_cross_entropy(x, w, t), loss)


def test_captured_and_replayed():
    x, w, t = make(100, 1000, 64, torch.bfloat16)
    x, w = x.requires_grad_(), w.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(tl.linear_cross_entropy(x, w, t), (x, w))
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = tl.linear_cross_entropy(x, w, t)
        out = (loss, *torch.autograd.grad(loss, (x, w)))
    for seed in range(3):
        nx, nw, nt = make(100, 1000, 64, torch.bfloat16, seed=50 + seed)
        with torch.no_grad():
            x.copy_(nx), w.copy_(nw), t.copy_(nt)
        want = run(nx, nw, nt)
        g.replay()
        torch.cuda.synchronize()
        for name, o in zip(("loss", "dx", "dw"), out):
            assert torch.equal(o, want[name]), (seed, name)


def test_streams_side_by_side():
    cases = [make(M, 900, 128, torch.bfloat16, seed=M) for M in (1, 60, 400)]
    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    got = []
    for c in cases:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(run(*c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[k], g[k]) for k in w)


def test_same_bits_every_time():
    x, w, t = make(600, 9000, 256, torch.bfloat16)
    first = run(x, w, t)
    for _ in range(3):
        again = run(x, w, t)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_no_write_outside_the_outputs():
    M, V, K = 37, 75, 33
    x, w, t = make(M, V, K, torch.bfloat16)
    held = {k: torch.full((r + 2, K + 5), 7.0, dtype=torch.bfloat16, device="cuda") for k, r in {"dx": M, "dw": V}.items()}
    loss, dloss = torch.full((M + 2,), 7.0, device="cuda"), torch.ones(M, device="cuda")
    saved, s1, s2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in tl._xent_bytes(M, V, K, 3))
    at = lambda k: (held[k][1:].data_ptr(), K + 5)  # noqa: E731
    tl._call(x.device, tl._lib.tgemm_xent_forward, M, V, K, tl.BF16, x.data_ptr(), K, w.data_ptr(), K, t.data_ptr(), -100, 0, 0,
             loss[1:].data_ptr(), saved.data_ptr(), s1.data_ptr())
    tl._call(x.device, tl._lib.tgemm_xent_backward, M, V, K, tl.BF16, x.data_ptr(), K, w.data_ptr(), K, t.data_ptr(), 0,
             dloss.data_ptr(), saved.data_ptr(), 3, *at("dx"), *at("dw"), s2.data_ptr())
    got = run(x, w, t, 1.0, "none")
    assert torch.equal(loss[1:-1], got["loss"]) and loss[0] == 7 and loss[-1] == 7
    for k, v in held.items():
        assert torch.equal(v[1:-1, :-5], got[k]) and (v[0] == 7).all() and (v[-1] == 7).all() and (v[:, -5:] == 7).all(), k


def test_derivatives_that_are_refused():
    x, w, t = make(5, 16, 8, torch.bfloat16)
    x.requires_grad_()
    one = torch.ones((), device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad(tl.linear_cross_entropy(x, w, t), x, one, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    with torch.autograd.forward_ad.dual_level(), pytest.raises(RuntimeError):
        tl.linear_cross_entropy(torch.autograd.forward_ad.make_dual(x.detach(), torch.ones_like(x)), w, t)


def test_refusals_on_the_gpu():
    x, w, t = make(5, 16, 8, torch.bfloat16)
    with pytest.raises(TypeError, match="int64"):
        tl.linear_cross_entropy(x, w, t.int())
    with pytest.raises(TypeError, match="w must have"):
        tl.linear_cross_entropy(x, w.half(), t)
    for bad in ((x, w[:, :7], t), (x, w[0], t), (x, w, t[:4]), (x, w, t.cpu()), (x, w, t[:, None])):
        with pytest.raises(ValueError):
            tl.linear_cross_entropy(*bad)
    for keep in (-1, float("nan")):
        with pytest.raises(ValueError, match="keep_bytes"):
            tl.linear_cross_entropy(x, w, t, keep_bytes=keep)
    for ignore in (2 ** 63, 0.5):
        with pytest.raises(ValueError, match="ignore_index"):
            tl.linear_cross_entropy(x, w, t, ignore_index=ignore)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("base", [1, 16, 128, 256])
def test_nearly_certain_targets_of_large_logits(base, dtype, kept, monkeypatch):
    """Logits base^2 (+ 12 for the target), all of them whole numbers that float holds: neither the loss nor p - 1 loses
    digits to their size."""
    monkeypatch.setattr(tl, "POWERS_LEAST", 0)
    M, V = 64, 256
    x = torch.tensor([[float(base), 1.0]], device="cuda").to(dtype).expand(M, 2).contiguous()
    w = torch.tensor([[float(base), 0.0]], device="cuda").to(dtype).repeat(V, 1)
    w[5, 1] = 12.0
    t = torch.full((M,), 5, device="cuda")
    got = run(x, w, t, 1024.0, "sum", keep_bytes=2 ** 34 * kept)
    others = (V - 1) * torch.exp(torch.tensor(-12.0, dtype=torch.float64))
    loss = torch.log1p(others)
    # the sum of powers is near one, and each addition to it is off by up to 2^-24: 64 of them in a lane, 64 for the pieces
    far = 130 * 2.0 ** -24
    assert abs(float(got["loss"]) / M - float(loss)) <= far + 2.0 ** -22 * float(loss)
    left = others / (1 + others)  # 1 - p
    want = -1024 * left * 12  # the one column in which the words differ: dx = sum of dz w
    u = ref.U[dtype]
    assert ((got["dx"][:, 1].double() - want).abs() <= (2 * u * left + far + 2.0 ** -20) * 1024 * 12 + 2.0 ** -25).all()
    dw = got["dw"][5, 1].double()
    assert abs(dw + M * 1024 * left) <= (2 * u * left + far + 2.0 ** -20) * 1024 * M


@pytest.mark.parametrize("dtype", DTYPES)
def test_kept_powers_do_not_add_a_rounding(dtype):
    """With the unit matrix for w, dx is dz: each element is off by dz's rounding and a small part of one."""
    M, K = 256, 512
    g = torch.Generator(device="cuda").manual_seed(9)
    x = (torch.randn((M, K), generator=g, device="cuda") * 0.7).to(dtype)
    w = torch.eye(K, dtype=dtype, device="cuda")
    t = torch.randint(0, K, (M,), generator=g, device="cuda")
    scale = 2.0 ** 10
    z = x.double()
    want = scale * (torch.softmax(z, 1) - torch.nn.functional.one_hot(t, K))
    dx = {}
    for keep in (0, 2 ** 30):
        dx[keep] = run(x, w, t, scale, "sum", keep_bytes=keep)["dx"].double()
        off = (dx[keep] - want).abs() / want.abs()
        # dz is rounded; the logits are exact, p is good to 2^-19, and a kept power to half a step of 10 or 12 bits
        power = {torch.bfloat16: 2.0 ** -10, torch.float16: 2.0 ** -12}[dtype]
        assert off.max() <= ref.U[dtype] + 2.0 ** -18 + (power * 1.01 if keep else 0), (keep, float(off.max() / ref.U[dtype]))
    assert abs(float(((dx[2 ** 30] - want) / want).mean())) < 2.0 ** -15


@pytest.mark.parametrize("M,V,K", [(90, 700, 64), (200, 3001, 520), (33000, 20001, 24)])
def test_a_rows_gradient_does_not_depend_on_other_rows_factors(M, V, K):
    """Float16 and a loss for each row: a row's dx keeps its digits whatever the largest factor of the batch is."""
    x, w, t = make(M, V, K, torch.float16, ignored=0.1)
    by = torch.exp2(torch.linspace(-3, 3, M, device="cuda"))
    by[1::7] *= -1
    by[5], t[5] = 2.0 ** 60, 1  # its own dx is past the type
    by[6] = 0.0
    by[7], t[7] = float("nan"), 2
    some = torch.arange(0, M, max(1, M // 500), device="cuda")
    some = some[(some != 5) & (some != 7)]
    for keep in (0, 2 ** 34):
        dx = run(x, w, t, by, "none", keep_bytes=keep)["dx"]
        want = ref.xent(x[some], w, t[some], reduction="none", dloss=by[some])
        ref.check({"dx": dx[some]}, want, ("dx",))
        # each row against the largest of its own
        for rows, values in zip(some.split(64), want["dx"][0].split(64)):
            off = (dx[rows].double() - values).norm(dim=1)
            assert (off <= 2e-3 * values.norm(dim=1)).all()
        assert dx[7].isnan().all() and not dx[t == -100].any()


def test_rows_factors_of_all_sizes_serve_dw():
    x, w, t = make(130, 500, 72, torch.float16, ignored=0.1)
    by = torch.exp2(torch.linspace(-28, 6, 130, device="cuda"))
    for keep in (0, 2 ** 34):
        ref.check(run(x, w, t, by, "none", keep_bytes=keep), ref.xent(x, w, t, reduction="none", dloss=by))
        one = w.detach().requires_grad_()
        (alone,) = torch.autograd.grad(tl.linear_cross_entropy(x, one, t, reduction="none", keep_bytes=keep), one, by)
        ref.check({"dw": alone}, ref.xent(x, w, t, reduction="none", dloss=by), ("dw",))


def test_as_many_rows_as_a_grid_holds():
    """A wave for each row: 2^26 - 128 of them."""
    M, V, K = 2 ** 26 - 128, 40, 8
    x, w, t = make(M, V, K, torch.bfloat16)
    some = torch.cat([torch.arange(0, M, 200003, device="cuda"), torch.arange(M - 300, M, device="cuda")])
    one = x.requires_grad_()
    loss = tl.linear_cross_entropy(one, w, t, reduction="none")
    (dx,) = torch.autograd.grad(loss, one, torch.ones((), device="cuda").expand(M))
    want = ref.xent(x.detach()[some], w, t[some], reduction="none", dloss=1.0)
    ref.check({"loss": loss.detach()[some], "dx": dx[some]}, want, ("loss", "dx"))
    with pytest.raises(tl.TgemmError, match="out of range"):
        tl.linear_cross_entropy(x.detach()[:1].expand(M + 1, K), w, t[:1].expand(M + 1))


@pytest.mark.parametrize("M,V,K,dtype", [
    (1, 3001, 512, torch.bfloat16), (130, 1000, 520, torch.float16), (700, 2049, 1000, torch.bfloat16), (1030, 4100, 2056, torch.bfloat16),
    (1030, 4100, 2056, torch.float16), (2050, 9001, 777, torch.float16), (4100, 12000, 513, torch.bfloat16), (70000, 9000, 512, torch.bfloat16)])
def test_logits_made_again_for_long_rows(M, V, K, dtype):
    """The backward pass of batches whose powers do not fit: no power is kept though K is at least 512."""
    x, w, t = make(M, V, K, dtype)
    some = torch.arange(0, M, max(1, M // 2000), device="cuda")
    got = run(x, w, t, 100.0, keep_bytes=0)
    by = 100.0 / int((t != -100).sum())
    want = ref.xent(x[some], w, t[some], reduction="sum", dloss=by, kept=False)
    ref.check({"dx": got["dx"][some]}, want, ("dx",))
    if len(some) == M:
        ref.check({"dw": got["dw"]}, want, ("dw",))
    else:  # added up over blocks of rows
        dw, bound = 0.0, 0.0
        for rows in torch.arange(M, device="cuda").split(4096):
            v, b = ref.xent(x[rows], w, t[rows], reduction="sum", dloss=by, kept=False)["dw"]
            dw, bound = dw + v, bound + b
        assert ((got["dw"].double() - dw).abs() <= bound + ref.U[dtype] * dw.abs()).all()


@pytest.mark.parametrize("M,V,K,dtype", [
    (3000, 2001, 513, torch.bfloat16), (3001, 3001, 1025, torch.float16), (2999, 1500, 777, torch.float16), (4000, 70000, 521, torch.bfloat16)])
def test_rows_at_odd_elements(M, V, K, dtype):
    """w copied to lines for the backward pass, from 3000 tokens on, in one piece and in several, or read where it is."""
    x, w, t = make(M, V, K, dtype)
    wide = torch.nn.functional.pad(w, (1, 7), value=float("nan"))[:, 1:-7]
    for keep in (0, 2 ** 34):
        want = ref.xent(x, w, t, dloss=100.0, kept=keep > 0)
        ref.check(run(x, w, t, 100.0, keep_bytes=keep), want)
        ref.check(run(x, wide, t, 100.0, keep_bytes=keep), want)


@pytest.mark.parametrize("K", [64, 520])
def test_rows_scales_captured_and_replayed(K):
    """Float16 and a loss for each row: as many launches whatever the rows' factors are."""
    x, w, t = make(100, 1000, K, torch.float16)
    x, w, by = x.requires_grad_(), w.requires_grad_(), torch.ones(100, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(tl.linear_cross_entropy(x, w, t, reduction="none"), (x, w), by)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = tl.linear_cross_entropy(x, w, t, reduction="none")
        out = (loss, *torch.autograd.grad(loss, (x, w), by))
    for seed in range(3):
        nx, nw, nt = make(100, 1000, K, torch.float16, seed=50 + seed)
        nby = torch.exp2(torch.linspace(-20.0 * seed, 4.0, 100, device="cuda"))
        with torch.no_grad():
            x.copy_(nx), w.copy_(nw), t.copy_(nt), by.copy_(nby)
        want = run(nx, nw, nt, nby, "none")
        g.replay()
        torch.cuda.synchronize()
        for name, o in zip(("loss", "dx", "dw"), out):
            assert torch.equal(o, want[name]), (seed, name)


def test_factors_that_are_not_finite_stay_in_their_rows():
    for dtype in DTYPES:
        x, w, t = make(90, 400, 64, dtype, ignored=0.0)
        by = torch.linspace(0.5, 2, 90, device="cuda")
        clean = run(x, w, t, by, "none")
        by[4], by[40] = float("inf"), float("nan")
        got = run(x, w, t, by, "none")
        rows = [i for i in range(90) if i not in (4, 40)]
        assert torch.equal(got["dx"][rows], clean["dx"][rows]) and torch.equal(got["loss"], clean["loss"])
        assert not got["dx"][[4, 40]].isfinite().any() and not got["dw"].isfinite().any()
