"""GPU tests of the norms with gate and residual (infini_attn_norm,
infini_attn_residual_norm) and their gradients against float64, within bounds derived from
the roundings (block_ref.py)."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
# one element, fewer than a vector, each number of threads per row, odd widths, the largest
DIMS = [1, 2, 7, 8, 77, 78, 128, 256, 264, 777, 1000, 1024, 1032, 1030, 2048, 2056, 4094, 4095, 4096, 5000, 8192]


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressive_memory_transformer_b200 as m
    assert m.device_status() == 0
    return m


def normal(shape, seed, scale=1.0, shift=0.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).cuda()


def case(rows, dim, dtype, kind, groups, post, seed=0):
    a = dict(x=normal((rows, dim), seed, 2.0, 0.25, dtype),
             b=normal((rows, dim), seed + 1, 0.7, -0.1, dtype), gate=None, pw=None, pb=None,
             w=normal((dim,), seed + 2, 0.1, 1.0), c=None)
    if groups:
        a["gate"] = normal((groups, dim), seed + 3, 0.3, 0.5)
    if post:
        a["pw"] = normal((dim,), seed + 4, 0.1, 0.8)
    if kind:
        a["c"] = normal((dim,), seed + 5, 0.1)
        if post:
            a["pb"] = normal((dim,), seed + 6, 0.1)
    return a


def kwargs(a, kind, alpha):
    return dict(gate=a["gate"], alpha=alpha, post_weight=a["pw"], post_bias=a["pb"],
                pre_weight=a["w"], pre_bias=a["c"], kind=kind, eps=EPS)


def wide(a, alpha, kind):
    d = {n: None if t is None else t.double() for n, t in a.items()}
    return (d["x"], d["b"], d["gate"], alpha, d["pw"], d["pb"], d["w"], d["c"], kind, EPS)


def check(ia, rows, dim, dtype, kind, groups, post, alpha=0.75, seed=0):
    a = case(rows, dim, dtype, kind, groups, post, seed)
    r, h = ia.infini_attn_residual_norm(a["x"], a["b"], **kwargs(a, kind, alpha))
    torch.cuda.synchronize()
    rr, er, rh, eh = ref.residual_norm(*wide(a, alpha, kind))
    ref.within(r, rr, er, ref.half_step(dtype), "r")
    ref.within(h, rh, eh, ref.half_step(dtype), "h")


def check_grads(ia, rows, dim, dtype, kind, groups, post, alpha=0.75, seed=0, dr=True, dh=True):
    a = case(rows, dim, dtype, kind, groups, post, seed)
    g_r = normal((rows, dim), seed + 7, 0.5, 0.0, dtype) if dr else None
    g_h = normal((rows, dim), seed + 8, 1.0, 0.0, dtype) if dh else None
    got = ia.infini_attn_residual_norm_backward(a["x"], a["b"], g_r, g_h,
                                                **kwargs(a, kind, alpha))
    torch.cuda.synchronize()
    args = (*wide(a, alpha, kind), None if g_r is None else g_r.double(),
            None if g_h is None else g_h.double())
    want, sizes = ref.residual_norm_grads(*args), ref.residual_norm_grad_sizes(*args)
    for name, g, w, m in zip(got._fields, got, want, sizes):
        if g is None:
            continue
        step = ref.half_step(g.dtype)
        # sums over the rows: as many roundings as additions in the worst case
        err = ref.UNITS * m + (rows * ref.F32 * m if g.dim() != 2 or name == "dgate" else 0)
        ref.within(g, torch.zeros_like(g).double() if w is None else w, err, step, name)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_widths(ia, dim, kind, dtype):
    check(ia, 37, dim, dtype, kind, 1, True)


@pytest.mark.parametrize("rows,groups", [(0, 0), (1, 0), (2, 2), (3, 3), (9, 1), (6000, 4),
                                         (2500, 2500), (1200, 300)])
@pytest.mark.parametrize("dim", [136, 1024])
@pytest.mark.parametrize("post", [True, False])
def test_forward_rows_and_gates(ia, rows, groups, dim, post):
    check(ia, rows, dim, BF, 0, groups, post)
    check(ia, rows, dim, F32, 1, groups, post, alpha=1.0)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_widths(ia, dim, kind, dtype):
    check_grads(ia, 37, dim, dtype, kind, 1, True)


@pytest.mark.parametrize("rows,groups", [(0, 2), (1, 0), (2, 2), (9, 1), (6000, 4), (2500, 2500),
                                         (1200, 300), (40000, 1)])
@pytest.mark.parametrize("dim", [136, 1024])
@pytest.mark.parametrize("post", [True, False])
def test_backward_rows_and_gates(ia, rows, groups, dim, post):
    check_grads(ia, rows, dim, BF, 0, groups, post)
    check_grads(ia, rows, dim, F32, 1, groups, post, alpha=1.0)


@pytest.mark.parametrize("dr,dh", [(True, False), (False, True)])
def test_backward_of_one_output(ia, dr, dh):
    check_grads(ia, 50, 264, F32, 1, 5, True, dr=dr, dh=dh)


def test_more_groups_than_a_grid_axis(ia):
    """One gate row per token, for more tokens than one axis of a grid holds."""
    rows, dim = 70001, 8
    a = case(rows, dim, F32, 0, rows, False)
    dr = normal((rows, dim), 9)
    got = ia.infini_attn_residual_norm_backward(a["x"], a["b"], dr, None, gate=a["gate"],
                                                pre_weight=a["w"])
    assert torch.allclose(got.dgate, dr * a["b"], rtol=2.0 ** -22, atol=0)
    two = case(140002, dim, F32, 0, 70001, False, seed=3)
    d2 = normal((140002, dim), 10)
    got = ia.infini_attn_residual_norm_backward(two["x"], two["b"], d2, None, gate=two["gate"])
    want = (d2.double() * two["b"].double()).view(70001, 2, dim)
    assert bool(((got.dgate.double() - want.sum(1)).abs()
                 <= 4 * ref.F32 * want.abs().sum(1)).all())


@pytest.mark.parametrize("dim", [77, 264, 2048])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_plain_norm_is_the_fused_one_without_a_block(ia, dim, kind, dtype):
    x, dh = normal((19, dim), 1, 2.0, 0.5, dtype), normal((19, dim), 2, 1.0, 0.0, dtype)
    w, c = normal((dim,), 3, 0.1, 1.0), normal((dim,), 4, 0.1) if kind else None
    h = ia.infini_attn_norm(x, w, c, kind=kind, eps=EPS)
    r2, h2 = ia.infini_attn_residual_norm(x, pre_weight=w, pre_bias=c, kind=kind, eps=EPS)
    assert torch.equal(h, h2) and torch.equal(r2, x)
    _, _, rh, eh = ref.residual_norm(x.double(), None, None, 1.0, None, None, w.double(),
                                     None if c is None else c.double(), kind, EPS)
    ref.within(h, rh, eh, ref.half_step(dtype))
    dx, dw, dc = ia.infini_attn_norm_backward(x, w, dh, c, kind=kind, eps=EPS)
    got = ia.infini_attn_residual_norm_backward(x, None, None, dh, pre_weight=w, pre_bias=c,
                                                kind=kind, eps=EPS)
    assert torch.equal(dx, got.dx) and torch.equal(dw, got.dpre_weight)
    assert dc is None if c is None else torch.equal(dc, got.dpre_bias)
    assert got.db is None and got.dgate is None and got.dpost_weight is None


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_and_rows_behind(ia, kind, dtype):
    """r over x and h over b; the rows behind the last one stay as they were."""
    rows, dim = 45, 520
    a = case(rows + 4, dim, dtype, kind, 0, True)
    x, b = a["x"][:rows], a["b"][:rows]
    tail = a["x"][rows:].clone(), a["b"][rows:].clone()
    kw = kwargs(a, kind, 0.5)
    r, h = ia.infini_attn_residual_norm(x, b, **kw)
    dr, dh = normal((rows, dim), 8, dtype=dtype), normal((rows, dim), 9, dtype=dtype)
    want = ia.infini_attn_residual_norm_backward(x, b, dr, dh, **kw)
    ia.infini_attn_residual_norm(x, b, r_out=x, h_out=b, **kw)
    assert torch.equal(x, r) and torch.equal(b, h)
    assert torch.equal(a["x"][rows:], tail[0]) and torch.equal(a["b"][rows:], tail[1])
    assert all(t is None or bool(torch.isfinite(t.float()).all()) for t in want)


@pytest.mark.parametrize("dim", [136, 1024, 4096])
def test_rows_off_16_bytes_give_the_same(ia, dim):
    """Storage that starts off a 16-byte boundary takes the scalar loads: same results but
    for the order of a row's sums."""
    for dtype in (BF, F32):
        a = case(21, dim, dtype, 1, 3, True)
        off = {}
        for n, t in a.items():
            base = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            off[n] = base[1:].view(t.shape).copy_(t)
        got = ia.infini_attn_residual_norm(off["x"], off["b"], **kwargs(off, 1, 0.75))
        rr, er, rh, eh = ref.residual_norm(*wide(a, 0.75, 1))
        ref.within(got[0], rr, er, ref.half_step(dtype))
        ref.within(got[1], rh, eh, ref.half_step(dtype))


@pytest.mark.parametrize("dim", [264, 1024, 4096])
@pytest.mark.parametrize("kind", [0, 1])
def test_zero_constant_and_broken_rows(ia, dim, kind):
    """A row of zeros, a constant row, and rows with a NaN or an infinity: each is on its
    own, and the finite ones give what the formula gives."""
    x = normal((6, dim), 1)
    x[0], x[1] = 0.0, 3.0
    x[2, 5], x[3, 0] = float("nan"), float("inf")
    w = normal((dim,), 2, 0.1, 1.0)
    h = ia.infini_attn_norm(x, w, kind=kind, eps=EPS)
    assert not bool(h[0].any())
    if kind:
        # 3 - mean is 0 up to the mean's rounding, scaled by at most 1 / sqrt(eps)
        assert float(h[1].abs().max()) <= 3 * 2 * 64 * ref.F32 * EPS ** -0.5
    assert bool(h[2].isnan().all()) and bool(h[3].isnan().any())
    keep = [4, 5]
    _, _, rh, eh = ref.residual_norm(x[keep].double(), None, None, 1.0, None, None, w.double(),
                                     None, kind, EPS)
    ref.within(h[keep], rh, eh, ref.F32)


def test_large_mean(ia):
    """A layer norm of rows whose mean is a thousand times their spread: the variance comes
    from the distances to the mean."""
    x = normal((8, 1024), 1, 1.0, 1000.0)
    w = torch.ones(1024, device="cuda")
    h = ia.infini_attn_norm(x, w, kind=1, eps=EPS)
    _, _, rh, eh = ref.residual_norm(x.double(), None, None, 1.0, None, None, w.double(), None, 1,
                                     EPS)
    ref.within(h, rh, eh, ref.F32)


def test_gradient_against_differences(ia):
    rows, dim, kind, alpha = 12, 72, 1, 0.75
    a = case(rows, dim, F32, kind, 3, True)
    dr, dh = normal((rows, dim), 7), normal((rows, dim), 8)
    got = ia.infini_attn_residual_norm_backward(a["x"], a["b"], dr, dh, **kwargs(a, kind, alpha))
    base = {n: t.double() for n, t in a.items()}

    def f(d):
        r, _, h, _ = ref.residual_norm(d["x"], d["b"], d["gate"], alpha, d["pw"], d["pb"], d["w"],
                                       d["c"], kind, EPS)
        return float((r * dr.double()).sum() + (h * dh.double()).sum())

    names = dict(x="dx", b="db", gate="dgate", pw="dpost_weight", pb="dpost_bias",
                 w="dpre_weight", c="dpre_bias")
    for i, (n, field) in enumerate(names.items()):
        d = normal(base[n].shape, 20 + i).double()
        step = 1e-5
        slope = (f({**base, n: base[n] + step * d}) - f({**base, n: base[n] - step * d})) / (2 * step)
        g = getattr(got, field).double()
        size = float((g.abs() * d.abs()).sum())
        assert abs(slope - float((g * d).sum())) <= 1e-5 * size + 1e-8 * rows * dim, n


@pytest.mark.parametrize("dim", [200, 1024, 4096, 8192])
def test_same_bits_every_time_on_two_streams_and_in_a_graph(ia, dim):
    a = case(700, dim, BF, 1, 2, True)
    dr, dh = normal((700, dim), 8, dtype=BF), normal((700, dim), 9, dtype=BF)
    kw = kwargs(a, 1, 0.75)
    fwd = lambda **s: ia.infini_attn_residual_norm(a["x"], a["b"], **kw, **s)
    bwd = lambda **s: ia.infini_attn_residual_norm_backward(a["x"], a["b"], dr, dh, **kw, **s)
    want = [*fwd(), *bwd()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [t for _ in range(3) for s in ({}, {"stream": side}) for t in (*fwd(**s), *bwd(**s))]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(t, want[i % len(want)]) for i, t in enumerate(got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = [*fwd(), *bwd()]
    for _ in range(2):
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(again, want))
    a["x"].copy_(normal(a["x"].shape, 50, dtype=BF))
    g.replay()
    assert all(torch.equal(p, q) for p, q in zip(again, [*fwd(), *bwd()]))


def test_binding_refuses(ia):
    x, w = normal((8, 64), 1), normal((64,), 2)
    rn = ia.infini_attn_residual_norm
    for bad in (lambda: rn(x.half(), pre_weight=w), lambda: rn(x, x.bfloat16(), pre_weight=w),
                lambda: rn(x.t(), pre_weight=w), lambda: rn(x, x, gate=normal((3, 64), 3)),
                lambda: rn(x, x, gate=normal((63,), 3)), lambda: rn(x, gate=w),
                lambda: rn(x, post_weight=w), lambda: rn(x, pre_bias=w),
                lambda: rn(x, pre_weight=w.cpu()), lambda: rn(x, pre_weight=w.double()),
                lambda: rn(x, x, r_out=x[:4]), lambda: ia.infini_attn_norm(x, None),
                lambda: ia.infini_attn_residual_norm_backward(x, x, None, None, pre_weight=w),
                lambda: ia.infini_attn_residual_norm_backward(x, x, None, x)):
        with pytest.raises(ValueError):
            bad()
    big = torch.zeros((2, 8200), device="cuda")
    for bad in (lambda: ia.infini_attn_norm(big, torch.ones(8200, device="cuda")),
                lambda: ia.infini_attn_norm(x, w, bias=w, kind=0),
                lambda: ia.infini_attn_norm(x, w, eps=-1.0),
                lambda: ia.infini_attn_norm(x, w, kind=5)):
        with pytest.raises(ia.InfiniError):
            bad()
