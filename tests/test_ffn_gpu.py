"""GPU: the gated feed-forward block and its gradients against a plain form in 64 bits."""
import itertools

import pytest
import torch

import step_ref as ref

tl = pytest.importorskip("tiled_software_pipelined_amd.lib")
pytestmark = pytest.mark.gpu
NAMES = ("dx", "dw_gate", "dw_up", "dw_down")


def make(M, K, F, N, dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7919 * M + 31 * K + F + N)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return [t.to(dtype) for t in (r(M, K) * scale, r(F, K) / max(K, 1) ** 0.5, r(F, K) / max(K, 1) ** 0.5, r(N, F) / max(F, 1) ** 0.5, r(M, N))]


def run(leaves, dy, act, needs=(True,) * 4):
    leaves = [t.detach().requires_grad_(n) for t, n in zip(leaves, needs)]
    y = tl.gated_ffn(*leaves, activation=act)
    wanted = [t for t, n in zip(leaves, needs) if n]
    grads = iter(torch.autograd.grad(y, wanted, dy))
    return {"y": y.detach(), **{name: next(grads) for name, n in zip(NAMES, needs) if n}}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,F,N", [
    (1, 1, 1, 1), (3, 5, 2, 9), (1, 64, 128, 64), (7, 8, 16, 24), (16, 100, 33, 70), (17, 65, 66, 67), (32, 512, 1024, 256),
    (33, 64, 64, 64), (65, 127, 129, 63), (130, 200, 513, 77), (63, 2050, 70, 2050), (300, 264, 520, 264),
    (2050, 72, 4100, 136), (1030, 1000, 2100, 515), (5, 4096, 3, 2), (2, 3, 4096, 5), (4099, 8, 9, 10)])
def test_sizes(M, K, F, N, dtype):
    *leaves, dy = make(M, K, F, N, dtype)
    ref.check(run(leaves, dy, "silu"), ref.ffn(*leaves, "silu", dy))
    with torch.no_grad():
        ref.check({"y": tl.gated_ffn(*leaves)}, ref.ffn(*leaves, "silu"))


@pytest.mark.parametrize("M,K,F,N,dtype", [
    (4100, 520, 5128, 4104, torch.bfloat16), (2050, 2056, 5000, 2056, torch.float16), (1500, 1032, 8200, 4100, torch.bfloat16),
    (520, 2056, 2056, 2056, torch.float16), (3000, 640, 9001, 650, torch.float16), (600, 3000, 6001, 3001, torch.bfloat16),
    (4100, 4104, 520, 72, torch.float16), (800, 333, 517, 129, torch.bfloat16), (4100, 90, 130, 70, torch.bfloat16)])
def test_large_sizes(M, K, F, N, dtype):
    """Every tile of every product, whole rounds of them and rests that are shared out along k; rows copied to lines."""
    *leaves, dy = make(M, K, F, N, dtype)
    ref.check(run(leaves, dy, "silu"), ref.ffn(*leaves, "silu", dy))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", list(tl.ACTIVATIONS))
@pytest.mark.parametrize("M", [9, 150])
def test_activations(act, M, dtype):
    *leaves, dy = make(M, 96, 200, 80, dtype, scale=3.0)
    ref.check(run(leaves, dy, act), ref.ffn(*leaves, act, dy))


@pytest.mark.parametrize("act", list(tl.ACTIVATIONS))
def test_activations_over_their_range(act):
    """Gate values from far below to far above, each alone in its product: h itself."""
    g = torch.cat([torch.linspace(-30, 30, 1201), torch.tensor([-200.0, -88.5, 88.5, 200.0, 0.0, -0.0, 1e-6, -1e-6])]).to(torch.float16)
    F = g.numel()
    x, one = torch.ones(40, 1, dtype=torch.float16, device="cuda"), torch.ones(F, 1, dtype=torch.float16, device="cuda")
    eye = torch.eye(F, dtype=torch.float16, device="cuda")
    gd = g.double()
    want = ref.act(gd, act)[0]
    for rows in (1, 40):  # the kernel for few rows, the tiles
        y = tl.gated_ffn(x[:rows], g[:, None].cuda(), one, eye, activation=act).double().cpu()
        # two roundings to float16; the activation is good to 2^-20 of its value and 2^-23 of its argument
        bound = 2 * 2.0 ** -11 * want.abs() + 2.0 ** -24 + 2.0 ** -20 * want.abs() + 2.0 ** -23 * gd.abs() * (gd > -20)
        assert ((y - want).abs() <= bound).all(), float(((y - want).abs() - bound).max())


@pytest.mark.parametrize("act", list(tl.ACTIVATIONS))
def test_activations_at_the_ends_of_bfloat16(act):
    """Where act is 0 or its argument, so are the gradients 0 or those of a product, up to 1e30."""
    big = torch.tensor([1e4, -1e4, 1e20, -1e20, 1e30, -1e30], dtype=torch.bfloat16, device="cuda")
    F = big.numel()
    one = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    eye = torch.eye(F, dtype=torch.bfloat16, device="cuda")
    for rows in (1, 40):
        got = run([one(rows, 1), big[:, None], one(F, 1), eye], one(rows, F), act)
        up = big > 0
        assert torch.equal(got["y"], torch.where(up, big, 0).expand(rows, F))
        # dg = act'(g) = 1 or 0, du = act(g)
        assert torch.equal(got["dw_gate"][:, 0], torch.where(up, float(rows), 0.0).bfloat16())
        assert ((got["dw_up"][:, 0].double() - rows * torch.where(up, big, 0).double()).abs() <= 2.0 ** -8 * rows * big.abs().double()).all()


@pytest.mark.parametrize("needs", [n for n in itertools.product((False, True), repeat=4) if any(n)])
def test_only_the_gradients_that_are_asked_for(needs):
    *leaves, dy = make(70, 96, 130, 64, torch.bfloat16)
    got = run(leaves, dy, "gelu", needs)
    assert set(got) == {"y"} | {n for n, k in zip(NAMES, needs) if k}
    ref.check(got, ref.ffn(*leaves, "gelu", dy), got)


def test_gradients_against_differences():
    """Float16 inputs, and differences of the form in 64 bits: no formula of the derivative in between."""
    *leaves, dy = make(6, 12, 10, 8, torch.float16)
    got = run(leaves, dy, "gelu_tanh")
    wide = [t.double().cpu() for t in leaves]

    def value():
        g, u = wide[0] @ wide[1].t(), wide[0] @ wide[2].t()
        return float(((ref.act(g, "gelu_tanh")[0] * u) @ wide[3].t() * dy.double().cpu()).sum())

    for name, t in zip(NAMES, wide):
        bound = ref.ffn(*leaves, "gelu_tanh", dy)[name][1].cpu()
        flat = t.view(-1)
        for i in range(0, flat.numel(), 7):
            old = flat[i].item()
            flat[i] = old + 1e-5
            up = value()
            flat[i] = old - 1e-5
            down = value()
            flat[i] = old
            assert abs(got[name].double().cpu().reshape(-1)[i].item() - (up - down) / 2e-5) <= bound.reshape(-1)[i].item() + 1e-7


@pytest.mark.parametrize("M", [4, 100])
def test_strides_and_views(M):
    K, F, N, t = 70, 90, 50, torch.bfloat16
    x, wg, wu, wd, dy = make(M, K, F, N, t)
    both = torch.cat([wg, wu])  # one tensor of both projections
    wide = torch.full((N, F + 13), float("nan"), dtype=t, device="cuda")
    wide[:, 5:5 + F] = wd
    apart = torch.full((M, K + 3), float("nan"), dtype=t, device="cuda")
    apart[:, 1:1 + K] = x
    views = [apart[:, 1:1 + K], both[:F], both[F:], wide[:, 5:5 + F]]
    want = ref.ffn(x, wg, wu, wd, "silu", dy)
    ref.check(run(views, dy, "silu"), want)
    ref.check(run([x.t().contiguous().t(), wg.t().contiguous().t(), wu, wd], dy, "silu"), want)  # columns apart: copies
    ref.check({"y": tl.gated_ffn(*views)}, want, ("y",))
    # a broadcast gradient, and more axes
    ones = torch.ones((), dtype=t, device="cuda").expand(M, N)
    ref.check(run([x, wg, wu, wd], ones, "silu"), ref.ffn(x, wg, wu, wd, "silu", ones))
    y = tl.gated_ffn(x.view(2, M // 2, K), wg, wu, wd)
    assert y.shape == (2, M // 2, N) and torch.equal(y.view(M, N), tl.gated_ffn(x, wg, wu, wd))
    assert torch.equal(tl.gated_ffn(x[0], wg, wu, wd), tl.gated_ffn(x[:1], wg, wu, wd)[0])


@pytest.mark.parametrize("M,K,F,N", [(0, 8, 8, 8), (4, 0, 8, 8), (4, 8, 0, 8), (4, 8, 8, 0), (40, 0, 8, 8), (40, 8, 0, 8)])
def test_empty_sizes(M, K, F, N):
    *leaves, dy = make(M, K, F, N, torch.bfloat16)
    got = run(leaves, dy, "silu")
    assert got["y"].shape == (M, N) and not got["y"].any() or K and F
    for name, t in zip(NAMES, leaves):
        assert got[name].shape == t.shape and not got[name].any()


def test_values_that_are_not_finite_stay_in_their_rows():
    *leaves, dy = make(200, 80, 96, 64, torch.bfloat16)
    clean = tl.gated_ffn(*leaves)
    leaves[0][3, 5], leaves[0][150, 0] = float("nan"), float("inf")
    y = tl.gated_ffn(*leaves)
    rows = [i for i in range(200) if i not in (3, 150)]
    assert torch.equal(y[rows], clean[rows]) and y[3].isnan().all() and not y[150].isfinite().any()
    few = tl.gated_ffn(leaves[0][:8], *leaves[1:])
    assert few[3].isnan().all() and few[[0, 1, 2, 4, 5, 6, 7]].isfinite().all()


def test_same_bits_every_time():
    *leaves, dy = make(500, 512, 1376, 512, torch.bfloat16)
    first = run(leaves, dy, "silu")
    for _ in range(3):
        again = run(leaves, dy, "silu")
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_captured_and_replayed():
    *leaves, dy = make(100, 128, 344, 128, torch.bfloat16)
    leaves = [t.requires_grad_() for t in leaves]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(tl.gated_ffn(*leaves), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):  # two graphs with workspaces of one pool
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            y = tl.gated_ffn(*leaves)
            outs.append((y, *torch.autograd.grad(y, leaves, dy)))
        graphs.append(g)
    for seed in range(3):
        *new, ndy = make(100, 128, 344, 128, torch.bfloat16, seed=100 + seed)
        with torch.no_grad():
            for t, n in zip((*leaves, dy), (*new, ndy)):
                t.copy_(n)
        want = run(new, ndy, "silu")
        for g, out in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            for name, o in zip(("y",) + NAMES, out):
                assert torch.equal(o, want[name]), (seed, name)


def test_streams_side_by_side():
    cases = [make(M, 256, 700, 256, torch.bfloat16, seed=M) for M in (1, 40, 300)]
    want = [run(c[:4], c[4], "silu") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append(run(c[:4], c[4], "silu"))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[k], g[k]) for k in w)


def test_no_write_outside_the_outputs():
    """Rows of y and of the gradients end at odd places: what stands behind them stays."""
    M, K, F, N = 37, 33, 35, 39
    *leaves, dy = make(M, K, F, N, torch.bfloat16)
    x, wg, wu, wd = leaves
    held = {k: torch.full((r + 2, c + 5), 7.0, dtype=torch.bfloat16, device="cuda") for k, (r, c) in
            {"y": (M, N), "dx": (M, K), "dw_gate": (F, K), "dw_up": (F, K), "dw_down": (N, F)}.items()}
    sizes = tl._ffn_bytes(M, K, F, N, 15)
    saved, s1, s2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)
    at = lambda k: (held[k][1:].data_ptr(), held[k].shape[1])  # noqa: E731
    p = lambda t: (t.data_ptr(), t.shape[1])  # noqa: E731
    tl._call(x.device, tl._lib.tgemm_ffn_forward, M, K, F, N, tl.BF16, 0, *p(x), *p(wg), *p(wu), *p(wd), *at("y"), 15,
             saved.data_ptr(), s1.data_ptr())
    tl._call(x.device, tl._lib.tgemm_ffn_backward, M, K, F, N, tl.BF16, 0, *p(x), *p(wg), *p(wu), *p(wd), *p(dy), 15,
             saved.data_ptr(), *at("dx"), *at("dw_gate"), *at("dw_up"), *at("dw_down"), s2.data_ptr())
    got = run(leaves, dy, "silu")
    for k, t in held.items():
        assert torch.equal(t[1:-1, :-5], got[k]) and (t[0] == 7).all() and (t[-1] == 7).all() and (t[:, -5:] == 7).all(), k


def test_derivatives_that_are_refused():
    *leaves, dy = make(5, 8, 16, 8, torch.bfloat16)
    x = leaves[0].requires_grad_()
    (g,) = torch.autograd.grad(tl.gated_ffn(*leaves), x, dy.requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    with torch.autograd.forward_ad.dual_level(), pytest.raises(RuntimeError):
        dual = torch.autograd.forward_ad.make_dual(leaves[0].detach(), torch.ones_like(leaves[0]))
        tl.gated_ffn(dual, *leaves[1:])


def test_refusals_on_the_gpu():
    x, wg, wu, wd, _ = make(4, 8, 16, 8, torch.bfloat16)
    with pytest.raises(TypeError, match="w_up"):
        tl.gated_ffn(x, wg, wu.half(), wd)
    for bad in ([x, wg[:, :7], wu, wd], [x, wg, wu[:15], wd], [x, wg, wu, wd[:, :15]], [x, wg[0], wu[0], wd], [x[0, 0], wg, wu, wd]):
        with pytest.raises(ValueError, match="feed-forward"):
            tl.gated_ffn(*bad)
    with pytest.raises(ValueError, match="one GPU"):
        tl.gated_ffn(x, wg, wu.cpu(), wd)


CLOSED = {"silu": (10.0, 20.0), "gelu": (3.0, 5.4), "gelu_tanh": (3.0, 4.6)}


@pytest.mark.parametrize("needs", [(True,) * 4, (True, False, False, False), (False, True, False, False), (False, False, True, False),
                                   (False, True, True, True), (False, True, False, True), (False, False, True, True)])
@pytest.mark.parametrize("act", list(CLOSED))
def test_gradients_of_closed_gates_in_float16(act, needs):
    """act(g) and act'(g) u of closed gates are below float16's normal numbers (silu(-20) -4e-8); a scaled loss makes their
    products with dh numbers that the type holds, to its precision."""
    M, F, t = 40, 200, torch.float16
    lo, hi = CLOSED[act]
    gate = -torch.linspace(lo, hi, F, device="cuda").to(t)
    dy = (torch.rand(M, F, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 4000 + 4000).to(t)
    one = lambda *s: torch.ones(*s, dtype=t, device="cuda")  # noqa: E731
    got = run([one(M, 1), gate[:, None], one(F, 1), torch.eye(F, dtype=t, device="cuda")], dy, act, needs)
    g = gate.double()
    a, d, _ = ref.act(g, act)
    da, dd = dy.double() * a, dy.double() * d
    assert da.abs().min() > 2.0 ** -14 and dd.abs().min() > 2.0 ** -14 and a.abs().min() < 2.0 ** -14
    # dg and du are rounded once, then the results; sums of 40 and the activation: 2^-15
    near = 2.0 ** -11 * 2 + 2.0 ** -15
    if needs[2]:
        want = da.sum(0)
        assert ((got["dw_up"][:, 0].double() - want).abs() <= near * want.abs()).all()
    if needs[1]:
        want = dd.sum(0)
        assert ((got["dw_gate"][:, 0].double() - want).abs() <= near * want.abs()).all()
    if needs[3]:  # h itself is an operand in float16
        want, size = (dy.double().t() @ a.expand(M, F).contiguous()), dy.double().sum(0)[:, None]
        assert ((got["dw_down"].double() - want).abs() <= near * want.abs() + 2.0 ** -25 * size).all()
    if needs[0]:
        want = dd @ g[:, None] + da.sum(1, keepdim=True)
        size = dd.abs() @ g.abs()[:, None] + da.abs().sum(1, keepdim=True)
        assert ((got["dx"].double() - want).abs() <= (2.0 ** -11 + 2.0 ** -14) * size + 2.0 ** -11 * want.abs()).all()


def test_projections_beyond_float16():
    """u = 2.4e5: act'(g) u has no place in the type, its product with a small dy has."""
    t = torch.float16
    gate = torch.tensor([-6e4, -30.0, -17.0, 17.0, 30.0, 200.0], dtype=t, device="cuda")
    F = gate.numel()
    up = torch.full((F, 1), 6e4, dtype=t, device="cuda")
    x, eye, dy = torch.full((40, 1), 4.0, dtype=t, device="cuda"), torch.eye(F, dtype=t, device="cuda"), torch.full((40, F), 2.0 ** -12, dtype=t, device="cuda")
    u = 4 * float(up[0, 0])
    for act in tl.ACTIVATIONS:
        got = run([x, gate[:, None], up, eye], dy, act, (False, True, True, False))
        a, d, _ = ref.act(4 * gate.double(), act)
        for name, want in {"dw_gate": 160 * 2.0 ** -12 * d * u, "dw_up": 160 * 2.0 ** -12 * a}.items():
            # two roundings; g and u in 24 bits, the activation and 40 additions: 2^-14
            assert ((got[name][:, 0].double() - want).abs() <= (2 * 2.0 ** -11 + 2.0 ** -14) * want.abs() + 160 * 2.0 ** -25).all(), (act, name)


@pytest.mark.parametrize("M,K,F,N", [(0, 8, 8, 8), (4, 0, 8, 8), (4, 8, 0, 8), (4, 8, 8, 0), (40, 0, 8, 8), (40, 8, 0, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_empty_sizes_one_by_one(M, K, F, N, dtype):
    *leaves, dy = make(M, K, F, N, dtype)
    got = run(leaves, dy, "silu")
    assert got["y"].shape == (M, N)
    assert not got["y"].any()
    for name, t in zip(NAMES, leaves):
        assert got[name].shape == t.shape and not got[name].any()


@pytest.mark.parametrize("M,K,F,N,dtype", [
    (3000, 513, 640, 72, torch.bfloat16), (3001, 1025, 1003, 130, torch.float16), (3100, 640, 777, 521, torch.float16), (2999, 1025, 515, 70, torch.bfloat16)])
def test_rows_at_odd_elements(M, K, F, N, dtype):
    """Weights and x copied to lines, from 3000 tokens on, or read where they are; views of wider rows as well."""
    *leaves, dy = make(M, K, F, N, dtype)
    want = ref.ffn(*leaves, "silu", dy)
    got = run(leaves, dy, "silu")
    ref.check(got, want)
    wide = [torch.nn.functional.pad(t, (1, 7), value=float("nan"))[:, 1:-7] for t in leaves]
    ref.check(run(wide, dy, "silu"), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", list(tl.ACTIVATIONS))
def test_gradients_of_values_that_are_not_finite_stay_in_their_rows(act, dtype):
    *leaves, dy = make(200, 80, 96, 64, dtype)
    clean = run(leaves, dy, act)
    rows = [i for i in range(200) if i not in (3, 150, 170)]
    leaves[0][3, 5], leaves[0][150, 0], dy[170, 1] = float("nan"), float("inf"), float("nan")
    got = run(leaves, dy, act)
    assert torch.equal(got["dx"][rows], clean["dx"][rows]) and torch.equal(got["y"][rows], clean["y"][rows])
    assert got["y"][3].isnan().all() and not got["y"][150].isfinite().any() and torch.equal(got["y"][170], clean["y"][170])
    if act == "relu":  # a comparison has no value for a gate without one: its slope is 0
        assert got["dx"][170].isnan().all() and not got["dw_down"].isfinite().all()
    else:
        assert got["dx"][[3, 170]].isnan().all() and got["dw_up"].isnan().all() and got["dw_gate"].isnan().all()


def test_float16_captured_and_replayed():
    *leaves, dy = make(100, 128, 344, 128, torch.float16)
    leaves = [t.requires_grad_() for t in leaves]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(tl.gated_ffn(*leaves, activation="gelu"), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = tl.gated_ffn(*leaves, activation="gelu")
        out = (y, *torch.autograd.grad(y, leaves, dy))
    for seed in range(3):
        *new, ndy = make(100, 128, 344, 128, torch.float16, seed=100 + seed)
        with torch.no_grad():
            for t, n in zip((*leaves, dy), (*new, ndy)):
                t.copy_(n)
        want = run(new, ndy, "gelu")
        g.replay()
        torch.cuda.synchronize()
        for name, o in zip(("y",) + NAMES, out):
            assert torch.equal(o, want[name]), (seed, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", list(tl.ACTIVATIONS))
def test_gradients_of_a_token_have_one_rounding(act, dtype):
    """One token, x = 1 and units of their own: the results are dg and du, rounded once; act(g) and act'(g) u are not."""
    F = 4096
    g = torch.Generator(device="cuda").manual_seed(11)
    gate, up, dy = [(torch.randn(F, generator=g, device="cuda") * s).to(dtype) for s in (2.0, 1.0, 1.0)]
    one = torch.ones(1, 1, dtype=dtype, device="cuda")
    got = run([one, gate[:, None], up[:, None], torch.eye(F, dtype=dtype, device="cuda")], dy[None], act)
    a, d, _ = ref.act(gate.double(), act)
    u, v, w = ref.U[dtype], up.double(), dy.double()
    for name, want, size in (("dw_gate", w * d * v, w * v), ("dw_up", w * a, w)):
        # g and u in 24 bits are exact here; the activation: 2^-18 of its terms
        off = (got[name][:, 0].double() - want).abs()
        assert (off <= u * want.abs() + 2.0 ** -18 * size.abs() * (1 + gate.double().abs()) + ref.TINY[dtype]).all(), name
