"""GPU: gradient clipping against 64 bits, and a training step of the operators together."""
import math

import pytest
import torch

import step_ref as ref

tl = pytest.importorskip("tiled_software_pipelined_amd.lib")
pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def make(shapes, dtypes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale).to(dtypes[i % len(dtypes)]) for i, s in enumerate(shapes)]


def want(grads, max_norm, eps=1e-6):
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    return norm, min(1.0, max_norm / (norm + eps))


def check(got, norm, before, wanted):
    n, f = wanted
    assert abs(float(norm) - n) <= 2 * 2.0 ** -24 * n
    for a, b in zip(got, before):
        v = b.double() * f  # the factor and the product in float are rounded, then the product to the type
        assert ((a.double() - v).abs() <= (3 * 2.0 ** -24 + HALF[b.dtype] * (b.dtype != torch.float32)) * v.abs() + LEAST[b.dtype]).all()


@pytest.mark.parametrize("shapes", [[(1,)], [()], [(3, 5), (7,)], [(4096,), (8191,), (8193,)], [(1000, 333)] * 5, [(0,), (5,), (0, 7)],
                                    [(17,)] * 300, [(1 << 24,), (3,)], [(20000019,)]])
@pytest.mark.parametrize("dtypes", [(torch.float32,), (torch.bfloat16,), (torch.float16,), (torch.bfloat16, torch.float32, torch.float16)])
def test_sizes_and_types(shapes, dtypes):
    for limit in (0.5, 1e9):
        grads = make(shapes, dtypes)
        before = [t.clone() for t in grads]
        limit = min(limit * want(before, 0)[0], limit) if limit < 1 else limit
        norm = tl.clip_grad_norm(grads, limit)
        assert norm.shape == () and norm.dtype == torch.float32
        check(grads, norm, before, want(before, limit))
        if limit == 1e9:
            assert all(torch.equal(a, b) for a, b in zip(grads, before))
        out = [torch.full_like(t, 9) for t in before]
        again = tl.clip_grad_norm(before, limit, out=out)
        assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(out, grads))


def test_many_small_elements_and_large_ones():
    grads = [torch.full((50_000_000,), 1e-3, device="cuda"), torch.full((10,), 1e19, device="cuda")]
    assert abs(float(tl.clip_grad_norm(grads[:1], 1e9)) / (1e-3 * math.sqrt(5e7)) - 1) < 1e-6
    n, f = want(grads, 1.0)  # squares beyond float
    norm = tl.clip_grad_norm(grads, 1.0)
    assert abs(float(norm) / n - 1) < 1e-6 and abs(float(grads[1][0]) / (1e19 * f) - 1) < 1e-6
    tiny = [torch.full((1000,), 1e-30, device="cuda")]
    assert abs(float(tl.clip_grad_norm(tiny, 1.0)) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6


def test_not_finite():
    a, b = torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16)
    b[3] = float("inf")
    norm = tl.clip_grad_norm([a, b], 1.0)
    assert norm.isinf() and not a.any() and b[3].isnan() and not b[[0, 1, 49]].any()
    a, b = torch.ones(100, device="cuda"), torch.ones(50, device="cuda")
    a[7] = float("nan")
    assert tl.clip_grad_norm([a, b], 1.0).isnan() and a.isnan().all() and b.isnan().all()
    z = [torch.zeros(5, device="cuda")]
    assert tl.clip_grad_norm(z, 0.0) == 0 and not z[0].any()
    z = [torch.ones(5, device="cuda")]
    assert tl.clip_grad_norm(z, float("inf")) > 0 and (z[0] == 1).all()


def test_layouts_neighbours_and_versions():
    held = torch.full((1003,), 5.0, dtype=torch.bfloat16, device="cuda")
    part = held[1:1002]  # starts and ends off every boundary
    turned = torch.randn(40, 30, device="cuda").t()
    last = torch.randn(2, 8, 4, 4, device="cuda").to(memory_format=torch.channels_last)
    before = [t.clone() for t in (part, turned, last)]
    v = part._version
    norm = tl.clip_grad_norm([part, turned, last], 1.0)
    check([part, turned, last], norm, before, want(before, 1.0))
    assert held[0] == 5 and (held[1002:] == 5).all() and part._version > v
    with torch.inference_mode():
        t = torch.ones(4, device="cuda")
        tl.clip_grad_norm([t], 1.0)
    assert abs(float(t.norm()) - 1) < 1e-5


def test_refusals_on_the_gpu():
    a, b = torch.ones(6, device="cuda"), torch.ones(6, device="cuda")
    with pytest.raises(ValueError, match="twice"):
        tl.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(ValueError, match="twice"):
        tl.clip_grad_norm([a, b], 1.0, out=[a, a])
    with pytest.raises(ValueError, match="another"):
        tl.clip_grad_norm([a, b], 1.0, out=[b, torch.ones(6, device="cuda")])
    for bad in ([a.cpu(), b], [a, b.cpu()], [a, torch.ones(6, 2, device="cuda")[:, 0]]):
        with pytest.raises(ValueError):
            tl.clip_grad_norm(bad, 1.0)
    with pytest.raises(TypeError):
        tl.clip_grad_norm([a.double()], 1.0)
    for o in (b.half(), b[:5], b.view(2, 3), b.cpu()):
        with pytest.raises(ValueError, match="out must"):
            tl.clip_grad_norm([a], 1.0, out=[o])
    assert (a == 1).all() and (b == 1).all()
    norm = tl.clip_grad_norm([a[:0], b, a[:0]], 1.0)  # empty tensors may come twice
    assert abs(float(norm) - 6 ** 0.5) < 1e-6


def test_captured_and_replayed_and_streams():
    shapes = [(300, 70), (70,), (1000,)] * 50  # more tensors than a launch takes
    grads = make(shapes, (torch.bfloat16, torch.float32))
    out = [torch.empty_like(t) for t in grads]
    tl.clip_grad_norm(grads, 1.0, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = tl.clip_grad_norm(grads, 1.0, out=out)
    for seed in range(3):
        new = make(shapes, (torch.bfloat16, torch.float32), seed=seed + 1, scale=0.01 if seed == 1 else 1.0)
        for t, n in zip(grads, new):
            t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        side = [torch.empty_like(t) for t in new]
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            other = tl.clip_grad_norm(new, 1.0, out=side)
        torch.cuda.synchronize()
        assert torch.equal(norm, other) and all(torch.equal(a, b) for a, b in zip(out, side))


def test_a_training_step_of_a_block_and_its_head():
    """Block, loss, gradients, clipping and the orthogonalised update, as a program runs
    them together; each link against 64 bits on the values that reached it."""
    M, K, F, V, t = 150, 128, 344, 1000, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = r(M, K).to(t)
    weights = [(r(F, K) / K ** 0.5).to(t), (r(F, K) / K ** 0.5).to(t), (r(K, F) / F ** 0.5).to(t), (r(V, K) / K ** 0.5).to(t)]
    weights = [w.requires_grad_() for w in weights]
    target = torch.randint(0, V, (M,), generator=g, device="cuda")
    target[::5] = -100
    wg, wu, wd, head = weights
    y = tl.gated_ffn(x, wg, wu, wd)
    y.retain_grad()
    loss = tl.linear_cross_entropy(y, head, target)
    loss.backward()
    plain = [w.detach() for w in weights]
    want_loss = ref.xent(y.detach(), plain[3], target, dloss=1.0)
    ref.check({"loss": loss, "dx": y.grad, "dw": head.grad}, want_loss)
    block = ref.ffn(x, *plain[:3], "silu", y.grad)
    ref.check({"y": y, "dw_gate": wg.grad, "dw_up": wu.grad, "dw_down": wd.grad}, block, ("y", "dw_gate", "dw_up", "dw_down"))
    grads = [w.grad for w in weights]
    before = [v.clone() for v in grads]
    limit = 0.5 * want(before, 0)[0]
    norm = tl.clip_grad_norm(grads, limit)
    check(grads, norm, before, want(before, limit))
    with torch.no_grad():
        for w, v in zip(weights, grads):
            update = tl.orthogonalize(v)
            # five steps bring singular values near one
            s = torch.linalg.svdvals(update.float())
            assert update.shape == w.shape and 0.3 < float(s.median()) < 1.3
            w -= 0.02 * update
    after = tl.linear_cross_entropy(tl.gated_ffn(x, *weights[:3]), head, target)
    assert after.isfinite()


def test_tensors_that_share_elements_are_refused():
    """Those would be scaled twice; tensors that are only read may share some."""
    t, far = torch.ones(1000, device="cuda"), torch.ones(1000, device="cuda")
    for grads, out in (([t[:600], t[500:]], None), ([t, far, t[10:20]], None), ([t.view(torch.bfloat16)[:7], t[3:5]], None),
                       ([t[:500], far[:500]], [t[100:600], torch.empty(500, device="cuda")]),
                       ([t[:500], far[:500]], [torch.empty(500, device="cuda"), t[100:600]]),
                       ([far[:500], far[500:]], [t[:500], t[499:999]])):
        with pytest.raises(tl.TgemmError, match="overlap"):
            tl.clip_grad_norm(grads, 1.0, out=out)
    assert (t == 1).all() and (far == 1).all()
    parts = [t[:500], t[500:]]
    assert abs(float(tl.clip_grad_norm(parts, 1.0)) - 1000 ** 0.5) < 1e-4 and abs(float(t.norm()) - 1) < 1e-5
    t.fill_(1)
    out = [far[:600], torch.empty(500, device="cuda")]
    tl.clip_grad_norm([t[:600], t[500:]], 1100 ** 0.5 / 2, out=out)
    assert (t == 1).all() and all(((o - 0.5).abs() < 1e-6).all() for o in out) and (far[600:] == 1).all()


def test_quotients_without_a_value():
    for value, limit, eps in ((float("inf"), float("inf"), 1e-6), (0.0, 0.0, 0.0)):
        t = torch.full((7,), value, device="cuda")
        tl.clip_grad_norm([t], limit, eps)
        assert t.isnan().all()
