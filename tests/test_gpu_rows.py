"""permute_rows / unpermute_rows and their gradients against plain loops in
64 bits on the CPU, on the plans of dispatch and dispatch_slots.

Tolerances, from the arithmetic alone: a copied row is exact. A sum of n fp32
products differs from the exact one by at most n * 2^-23 of the sum of the
terms' magnitudes (each product and each addition is off by at most 2^-24 of
what it yields, and n <= 2^20 here), and the rounding to bf16 adds at most 2^-8
of the value (fp32: 2^-24)."""

import pytest
import torch

import sparse_top_mixture_b200 as stm

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}

# (T, H, E, k): one token, one column vector, k past eight slots, odd batches,
# widths off every power of two, more blocks than are resident at once
SHAPES = [(1, 8, 1, 1), (1, 7168, 256, 8), (3, 40, 5, 5), (257, 256, 8, 2), (65, 264, 16, 9), (33, 72, 256, 17),
          (500, 2048, 64, 6), (20000, 16, 4, 1), (2, 8200, 250, 250)]
TYPES = [("bf16", torch.bfloat16), ("bf16", torch.float32), ("f32", torch.float32)]


def _problem(shape, dtype="bf16"):
    T, H, E, k = shape
    return stm.Problem(T=T, H=H, E=E, k=k, I=8, dtype=dtype)


def _plan(p, empty, seed=0):
    g = torch.Generator().manual_seed(seed)
    sel = torch.rand(p.T, p.E, generator=g).topk(p.k, 1).indices
    if empty:
        sel[torch.rand(p.T, p.k, generator=g) < empty] = -1
        sel[0] = -1  # a token without any row
    plan = stm.dispatch_slots(p, sel.cuda())
    return sel, plan


def _positions(p, sel):
    """pos [T, k] (-1 for none) and the rows in use, by a stable sort."""
    ids = sel.reshape(-1)
    order = [q for e in range(p.E) for q in (ids == e).nonzero().reshape(-1).tolist()]
    pos = torch.full((p.T * p.k,), -1, dtype=torch.long)
    pos[torch.tensor(order, dtype=torch.long)] = torch.arange(len(order))
    return pos.reshape(p.T, p.k), len(order)


def _rand(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _within(got, ref, terms, n):
    got = got.cpu()
    bound = HALF_STEP[got.dtype] * ref.abs() + n * 2.0 ** -23 * terms + 2.0 ** -133
    assert bool(((got.double() - ref).abs() <= bound).all()), float(((got.double() - ref).abs() - bound).max())


def _gather(y, pos):
    """[T, k, H] in 64 bits, zeros where a slot has no row."""
    return torch.where((pos >= 0)[:, :, None], y.double()[pos.clamp(min=0)], 0.0)


@pytest.mark.parametrize("empty", [0.0, 0.4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_permute_and_its_gradient(shape, dtype, empty):
    p = _problem(shape, dtype)
    sel, plan = _plan(p, empty)
    pos, used = _positions(p, sel)
    x = _rand((p.T, p.H), p.torch_dtype, 1)
    got = stm.permute_rows(p, x.cuda(), plan).cpu()
    ref = torch.zeros(p.T * p.k, p.H, dtype=p.torch_dtype)
    t, j = (pos >= 0).nonzero(as_tuple=True)
    ref[pos[t, j]] = x[t]
    assert torch.equal(got, ref)

    dxp = _rand((p.T * p.k, p.H), p.torch_dtype, 2)
    rows = _gather(dxp, pos)
    dxp[used:] = float("nan")  # rows without a pair are not read
    dx = stm.permute_rows_backward(p, dxp.cuda(), plan)
    _within(dx, rows.sum(1), rows.abs().sum(1), p.k)


@pytest.mark.parametrize("empty", [0.0, 0.4])
@pytest.mark.parametrize("dtype,y_dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_unpermute_and_its_gradient(shape, dtype, y_dtype, empty):
    p = _problem(shape, dtype)
    sel, plan = _plan(p, empty)
    pos, used = _positions(p, sel)
    y = _rand((p.T * p.k, p.H), y_dtype, 3)
    w = _rand((p.T, p.k), torch.float32, 4)
    shared = _rand((p.T, p.H), torch.float32, 5)
    dout = _rand((p.T, p.H), p.torch_dtype, 6)
    rows, wd = _gather(y, pos), w.double()[:, :, None]
    y[used:] = float("nan")
    w[pos < 0] = float("inf")  # the weight of a slot without a row is not used
    wd = torch.where((pos >= 0)[:, :, None], wd, 0.0)
    yc, wc = y.cuda(), w.cuda()

    terms = (wd * rows)
    _within(stm.unpermute_rows(p, yc, plan, wc), terms.sum(1), terms.abs().sum(1), p.k + 1)
    _within(stm.unpermute_rows(p, yc, plan), rows.sum(1), rows.abs().sum(1), p.k)
    s = shared.double()
    _within(stm.unpermute_rows(p, yc, plan, wc, shared.cuda()), terms.sum(1) + s, terms.abs().sum(1) + s.abs(), p.k + 2)

    dy, dw = stm.unpermute_rows_backward(p, dout.cuda(), yc, plan, wc)
    ref = torch.zeros(p.T * p.k, p.H, dtype=torch.float64)
    t, j = (pos >= 0).nonzero(as_tuple=True)
    ref[pos[t, j]] = wd[t, j] * dout.double()[t]
    assert dy.dtype == y_dtype
    _within(dy, ref, ref.abs(), 1)
    prod = rows * dout.double()[:, None]
    _within(dw, prod.sum(2), prod.abs().sum(2), p.H)
    assert bool((dw.cpu()[pos < 0] == 0).all())
    dy1, dw1 = stm.unpermute_rows_backward(p, dout.cuda(), yc, plan)  # weights of 1: rows are copies
    ref1 = torch.zeros(p.T * p.k, p.H, dtype=y_dtype)
    ref1[pos[t, j]] = dout[t].to(y_dtype)
    assert torch.equal(dy1.cpu(), ref1) and torch.equal(dw1, dw)


# each number of slots, with enough tokens for several vectors a thread, widths that leave some of them without one,
# and a width below them
@pytest.mark.parametrize("dtype,y_dtype", TYPES)
@pytest.mark.parametrize("shape", [(2400, 2056, 8, 1), (1200, 2056, 8, 2), (1200, 2056, 8, 3), (600, 2056, 8, 4),
                                   (600, 2056, 8, 5), (600, 2056, 8, 6), (600, 2056, 8, 7), (600, 2056, 8, 8),
                                   (600, 2056, 16, 9), (130000, 40, 4, 1)])
def test_every_number_of_slots(shape, dtype, y_dtype):
    test_unpermute_and_its_gradient(shape, dtype, y_dtype, 0.3)
    test_permute_and_its_gradient(shape, dtype, 0.3)


def test_rows_beyond_32_bits():
    """More than 2^31 sorted elements: row movement there and back, checked whole."""
    p = _problem((40000, 7168, 16, 8))
    _, plan = _plan(p, 0.0)
    x = torch.randn(p.T, p.H, device="cuda").bfloat16()
    rows = stm.permute_rows(p, x, plan)
    w = torch.full((p.T, p.k), 0.125, device="cuda")
    assert torch.equal(stm.unpermute_rows(p, rows, plan, w), x)  # eight equal rows times 1/8: exact
    at = plan["pair_pos"].long()
    assert torch.equal(rows[at[-8:]], x[-1:].expand(8, -1))
    dy, dw = stm.unpermute_rows_backward(p, x, rows, plan, w)
    assert torch.equal(dy[at[-8:]], (x[-1:] * 0.125).expand(8, -1))
    norm = (x.double() ** 2).sum(1)
    assert bool(((dw.double() - norm[:, None]).abs() <= p.H * 2.0 ** -23 * norm[:, None]).all())


def test_infinite_and_nan_rows_stay_in_their_token():
    p = _problem((40, 64, 8, 2))
    sel, plan = _plan(p, 0.0)
    pos, _ = _positions(p, sel)
    y = _rand((p.T * p.k, p.H), torch.bfloat16, 3)
    y[pos[7, 1], 5] = float("nan")
    y[pos[9, 0], 6] = float("inf")
    out = stm.unpermute_rows(p, y.cuda(), plan, torch.ones(p.T, p.k, device="cuda")).cpu()
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[7, 5], [9, 6]] and torch.isnan(out[7, 5]) and out[9, 6] == float("inf")


def test_results_are_the_same_every_time():
    p = _problem((700, 1160, 16, 4))
    _, plan = _plan(p, 0.2)
    y, dout = _rand((p.T * p.k, p.H), torch.bfloat16, 1).cuda(), _rand((p.T, p.H), torch.bfloat16, 2).cuda()
    w = torch.rand(p.T, p.k, device="cuda")
    first = (stm.unpermute_rows(p, y, plan, w), *stm.unpermute_rows_backward(p, dout, y, plan, w))
    for _ in range(5):
        again = (stm.unpermute_rows(p, y, plan, w), *stm.unpermute_rows_backward(p, dout, y, plan, w))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_plan_out_of_range_touches_nothing_else():
    """Positions outside [0, T*k) are slots without a row."""
    p = _problem((10, 64, 4, 2))
    _, plan = _plan(p, 0.0)
    plan["pair_pos"][3] = 1 << 30
    plan["pair_pos"][5] = -7
    y = _rand((p.T * p.k, p.H), torch.bfloat16, 1).cuda()
    pos = plan["pair_pos"].cpu().long().reshape(p.T, p.k)
    pos[(pos < 0) | (pos >= p.T * p.k)] = -1
    rows = _gather(y.cpu(), pos)
    _within(stm.unpermute_rows(p, y, plan), rows.sum(1), rows.abs().sum(1), p.k)
    dy, dw = stm.unpermute_rows_backward(p, y[: p.T].contiguous(), y, plan)
    assert dw.reshape(-1)[3] == 0 and dw.reshape(-1)[5] == 0
    stm.permute_rows(p, y[: p.T].contiguous(), plan)
    torch.cuda.synchronize()


def test_empty_batch():
    p = _problem((0, 64, 4, 2))
    plan = {"pair_pos": torch.empty(0, dtype=torch.int32, device="cuda"),
            "offsets": torch.zeros(5, dtype=torch.int32, device="cuda")}
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    rows = stm.permute_rows(p, x, plan)
    w = torch.empty(0, 2, device="cuda", requires_grad=True)
    out = stm.unpermute_rows(p, rows, plan, w)
    out.sum().backward()
    assert rows.shape == (0, 64) and out.shape == (0, 64) and x.grad.shape == (0, 64) and w.grad.shape == (0, 2)


@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_autograd_matches_the_formula_and_differences(y_dtype):
    """Gradients through both operators around one weight per expert, in the
    way experts of a caller's own are trained."""
    dtype = "f32" if y_dtype == torch.float32 else "bf16"
    p = _problem((50, 48, 6, 3), dtype)
    sel, plan = _plan(p, 0.2)
    pos, _ = _positions(p, sel)
    x = _rand((p.T, p.H), p.torch_dtype, 1).cuda().requires_grad_(True)
    w = torch.rand(p.T, p.k).cuda().requires_grad_(True)
    shared = _rand((p.T, p.H), torch.float32, 2).cuda().requires_grad_(True)
    scale = _rand((p.E,), torch.float32, 3).cuda().requires_grad_(True)
    dout = _rand((p.T, p.H), p.torch_dtype, 4).cuda()
    row_e = torch.searchsorted(plan["offsets"][1:].long(), torch.arange(p.T * p.k, device="cuda"), right=True)
    row_e = row_e.clamp(max=p.E - 1)

    def layer(x, w, shared, scale):
        rows = stm.permute_rows(p, x, plan)
        y = (rows.float() * scale[row_e][:, None]).to(y_dtype)
        return stm.unpermute_rows(p, y, plan, w, shared)

    layer(x, w, shared, scale).backward(dout)
    # the formula, in 64 bits
    xd, wd, sd = x.detach().cpu().double(), w.detach().cpu().double(), scale.detach().cpu().double()
    gd, has = dout.cpu().double(), (pos >= 0).double()
    se = sd[sel.clamp(min=0)] * has
    ref_x = ((wd * se).sum(1)[:, None] * gd)
    ref_w = se * (xd * gd).sum(1)[:, None]
    ref_s = torch.zeros(p.E, dtype=torch.float64)
    ref_s.index_add_(0, sel.clamp(min=0).reshape(-1), (has * wd * (xd * gd).sum(1)[:, None]).reshape(-1))
    # every gradient passes at most three roundings to y_dtype / the problem's dtype on its way
    tol = 4 * HALF_STEP[y_dtype] + 100 * 2.0 ** -23
    mag = (xd.abs() * gd.abs()).sum(1)[:, None]
    assert float((x.grad.cpu().double() - ref_x).abs().max()) <= tol * float(((wd * se).abs().sum(1)[:, None] * gd.abs()).max())
    assert float((w.grad.cpu().double() - ref_w).abs().max()) <= tol * float((se.abs() * mag).max())
    assert float((scale.grad.cpu().double() - ref_s).abs().max()) <= tol * float((has * wd * mag).sum())
    assert torch.equal(shared.grad, dout.float())
    if y_dtype == torch.float32:  # bilinear: a central difference is the derivative, up to rounding
        d = torch.randn(p.T, p.k, generator=torch.Generator().manual_seed(8)).cuda()
        f = lambda a: float((layer(x, a, shared, scale).double() * dout.double()).sum())  # noqa: E731
        with torch.no_grad():
            diff = (f(w + d) - f(w - d)) / 2
        exact = float((w.grad.double() * d.double()).sum())
        size = float((se.abs() * mag * (wd + d.cpu().double().abs())).sum() + (shared.detach().abs() * dout.abs()).sum())
        assert abs(diff - exact) <= 2.0 ** -20 * size


def test_only_asked_gradients_are_computed():
    p = _problem((9, 32, 4, 2))
    _, plan = _plan(p, 0.0)
    y = _rand((p.T * p.k, p.H), torch.bfloat16, 1).cuda()
    w = torch.rand(p.T, p.k, device="cuda")
    wl = w.clone().requires_grad_(True)
    stm.unpermute_rows(p, y, plan, wl).float().sum().backward()
    yl = y.clone().requires_grad_(True)
    stm.unpermute_rows(p, yl, plan, w).float().sum().backward()
    both_y, both_w = stm.unpermute_rows_backward(p, torch.ones(p.T, p.H, device="cuda").bfloat16(), y, plan, w)
    assert torch.equal(wl.grad, both_w) and torch.equal(yl.grad, both_y)
    assert not stm.unpermute_rows(p, y, plan, w).requires_grad
    with torch.no_grad():
        assert not stm.unpermute_rows(p, yl, plan, wl).requires_grad


def test_captured_and_on_a_stream_of_its_own():
    p = _problem((300, 512, 16, 4))
    sel, plan = _plan(p, 0.1)
    x = _rand((p.T, p.H), torch.bfloat16, 1).cuda()
    w = torch.rand(p.T, p.k, device="cuda")
    dout = _rand((p.T, p.H), torch.bfloat16, 2).cuda()

    def step():
        rows = stm.permute_rows(p, x, plan)
        out = stm.unpermute_rows(p, rows, plan, w)
        dy, dw = stm.unpermute_rows_backward(p, dout, rows, plan, w)
        return out, stm.permute_rows_backward(p, dy, plan), dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for seed in (3, 4):
        x.copy_(_rand((p.T, p.H), torch.bfloat16, seed))
        w.copy_(torch.rand(p.T, p.k, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_a_training_step_captured_with_its_backward():
    p = _problem((300, 512, 16, 4))
    _, plan = _plan(p, 0.1)
    x = _rand((p.T, p.H), torch.bfloat16, 1).cuda().requires_grad_(True)
    w = torch.rand(p.T, p.k, device="cuda", requires_grad=True)
    dout = _rand((p.T, p.H), torch.bfloat16, 2).cuda()

    def step():
        out = stm.unpermute_rows(p, stm.permute_rows(p, x, plan) * 2, plan, w)
        return (out.detach(), *torch.autograd.grad(out, (x, w), dout))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for seed in (3, 4):
        with torch.no_grad():
            x.copy_(_rand((p.T, p.H), torch.bfloat16, seed))
            dout.copy_(_rand((p.T, p.H), torch.bfloat16, seed + 9))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_gradients_of_outputs_that_are_views():
    """An expanded or transposed gradient of the output reaches the kernels whole."""
    p = _problem((16, 16, 4, 2))
    _, plan = _plan(p, 0.0)
    w = torch.rand(p.T, p.k, device="cuda")
    for pick in (lambda o: o.sum(), lambda o: (o.t() * torch.arange(256, device="cuda").view(16, 16).bfloat16()).sum()):
        x = _rand((p.T, p.H), torch.bfloat16, 1).cuda().requires_grad_(True)
        out = stm.unpermute_rows(p, stm.permute_rows(p, x, plan), plan, w)
        out.retain_grad()
        pick(out).backward()
        dy, _ = stm.unpermute_rows_backward(p, out.grad.contiguous(), torch.zeros_like(stm.permute_rows(p, x.detach(), plan)),
                                            plan, w)
        assert torch.equal(x.grad, stm.permute_rows_backward(p, dy, plan))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("front", [1, 3, 8])
def test_gradients_at_any_offset(front, dtype):
    """A gradient that autograd cuts out of a longer one: contiguous, at an offset of `front` elements."""
    p = _problem((16, 40, 4, 2), dtype)
    _, plan = _plan(p, 0.2)
    w = torch.rand(p.T, p.k, device="cuda", requires_grad=True)
    x = _rand((p.T, p.H), p.torch_dtype, 1).cuda().requires_grad_(True)
    a = torch.zeros(front, dtype=p.torch_dtype, device="cuda", requires_grad=True)

    def cut(t, seed):
        g = _rand((front + t.numel(),), p.torch_dtype, seed).cuda()
        torch.cat([a, t.reshape(-1)]).backward(g)
        return g[front:].view(t.shape).clone()

    rows = stm.permute_rows(p, x, plan)
    dxp = cut(rows, 2)
    assert torch.equal(x.grad, stm.permute_rows_backward(p, dxp, plan))
    y = rows.detach().requires_grad_(True)
    dout = cut(stm.unpermute_rows(p, y, plan, w), 3)
    dy, dw = stm.unpermute_rows_backward(p, dout, y.detach(), plan, w.detach())
    assert torch.equal(y.grad, dy) and torch.equal(w.grad, dw)


def test_forward_mode_is_refused():
    """A tensor with a tangent need not require a gradient; its tangent must not be lost in silence."""
    from torch.autograd import forward_ad

    p = _problem((6, 32, 4, 2))
    _, plan = _plan(p, 0.0)
    x = _rand((p.T, p.H), torch.bfloat16, 1).cuda()
    y = _rand((p.T * p.k, p.H), torch.bfloat16, 2).cuda()
    w, shared = torch.rand(p.T, p.k, device="cuda"), torch.rand(p.T, p.H, device="cuda")
    calls = [(lambda t: stm.permute_rows(p, t, plan), x), (lambda t: stm.unpermute_rows(p, t, plan, w), y),
             (lambda t: stm.unpermute_rows(p, y, plan, t), w), (lambda t: stm.unpermute_rows(p, y, plan, w, t), shared)]
    for call, t in calls:
        with forward_ad.dual_level():
            call(t)  # no tangent: nothing to refuse
            for leaf in (t, t.clone().requires_grad_(True)):
                dual = forward_ad.make_dual(leaf, torch.ones_like(t))
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    call(dual)
                with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                    call(dual)
        with pytest.raises((NotImplementedError, RuntimeError)):
            torch.func.jvp(call, (t,), (torch.ones_like(t),))


def _loss(p, plan, w, y_dtype=torch.bfloat16):
    y = _rand((p.T * p.k, p.H), y_dtype, 1).cuda().requires_grad_(True)
    return stm.unpermute_rows(p, y, plan, w).float().sum()


def test_a_plan_that_is_overwritten_before_the_backward_pass():
    """The library writes given buffers through their addresses; autograd has to know."""
    p = _problem((12, 32, 4, 2))
    sel = torch.rand(p.T, p.E, device="cuda").topk(p.k, 1).indices
    plan = stm.dispatch_noalloc(p, sel)
    w = torch.rand(p.T, p.k, device="cuda", requires_grad=True)
    x = _rand((p.T, p.H), torch.bfloat16, 1).cuda().requires_grad_(True)
    for loss in (lambda: _loss(p, plan, w), lambda: stm.permute_rows(p, x, plan).float().sum()):
        loss().backward()  # a plan that stays: nothing to refuse
        late = loss()
        again = stm.dispatch_noalloc(p, sel.flip(0).contiguous(), out=plan)
        assert again["pair_pos"] is plan["pair_pos"]
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            late.backward()


@pytest.mark.parametrize("kind", ["SparseMoE", "Mx4SparseMoE", "graph"])
def test_routing_weights_that_are_overwritten_before_the_backward_pass(kind):
    p = stm.Problem(T=12, H=64, E=4, k=2, I=32)
    g = torch.Generator().manual_seed(0)
    dev = {name: torch.randn(*s, generator=g).bfloat16().cuda()
           for name, s in (("gate_w", (4, 64)), ("gate_up", (4, 64, 64)), ("down", (4, 64, 32)))}
    moe = (stm.Mx4SparseMoE if kind == "Mx4SparseMoE" else stm.SparseMoE)(p, dev)
    x = _rand((p.T, p.H), torch.bfloat16, 1).cuda()
    rw, sel = torch.empty(p.T, p.k, device="cuda"), torch.empty(p.T, p.k, dtype=torch.int64, device="cuda")
    run = stm.GraphedForward(moe, x, None, rw, sel) if kind == "graph" else lambda: moe(x, None, rw, sel)
    run()
    plan = stm.dispatch(p, sel)
    _loss(p, plan, rw).backward()
    late = _loss(p, plan, rw)
    run()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        late.backward()


def test_refusals():
    p = _problem((4, 32, 4, 2))
    _, plan = _plan(p, 0.0)
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    bad = [lambda: stm.permute_rows(p, x.float(), plan), lambda: stm.permute_rows(p, x[:3], plan),
           lambda: stm.permute_rows(p, x.t().contiguous().t(), plan), lambda: stm.permute_rows(p, x.cpu(), plan),
           lambda: stm.permute_rows(p, x, {**plan, "pair_pos": plan["pair_pos"].long()}),
           lambda: stm.permute_rows(p, x, {**plan, "offsets": plan["offsets"][:-1]}),
           lambda: stm.unpermute_rows(p, y.half(), plan, w), lambda: stm.unpermute_rows(p, y, plan, w.double()),
           lambda: stm.unpermute_rows(p, y, plan, w, x), lambda: stm.unpermute_rows_backward(p, x[:2], y, plan, w),
           lambda: stm.unpermute_rows_backward(p, x, y[:4], plan, w)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    flat = torch.zeros(4 * 2 + 1, device="cuda")
    with pytest.raises(stm.MoeError) as e:  # not 16-byte aligned
        stm.unpermute_rows(p, y, plan, flat[1:].view(4, 2))
    assert e.value.status == 1
