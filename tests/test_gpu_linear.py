"""GPU tests of the linear layer (infini_attn_linear) and its gradient against float64,
element by element within bounds derived from the roundings (block_ref.py)."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressive_memory_transformer_b200 as m
    assert m.device_status() == 0
    return m


def normal(shape, seed, scale=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def ok(ia):
    torch.cuda.synchronize()
    assert ia.device_status() == 0, "a bounded device wait ran out"


def inputs(M, K, N, seed, bias=True, res=False):
    return (normal((M, K), seed), normal((K, N), seed + 1, K ** -0.5),
            normal((N,), seed + 2, 0.5, torch.float32) if bias else None,
            normal((M, N), seed + 3) if res else None)


def check_forward(ia, M, K, N, act, bias, res, seed=0):
    x, W, b, r = inputs(M, K, N, seed, bias, res)
    y, pre = ia.infini_attn_linear(x, W, bias=b, act=act, residual=r, save_preact=True)
    ok(ia)
    ry, ey, rp, ep = ref.linear(x, W, b, act, r)
    ref.within(y, ry, ey, ref.BF16, "y")
    ref.within(pre, rp, ep, ref.BF16, "preact")
    assert torch.equal(y, ia.infini_attn_linear(x, W, bias=b, act=act, residual=r))


# few rows (every width of the narrow side), one wave of tiles, ragged tiles in every
# direction, reductions shorter than one step and longer than a ring
@pytest.mark.parametrize("M,K,N", [
    (1, 8, 8), (1, 1024, 4096), (3, 72, 136), (16, 4096, 1024), (17, 512, 640), (33, 4096, 264),
    (64, 64, 8), (65, 64, 8), (100, 200, 72), (127, 1000, 392), (128, 128, 128), (129, 136, 256),
    (255, 2048, 520), (256, 256, 256), (513, 64, 1024), (640, 1160, 2056), (2048, 1024, 1024),
    (5003, 520, 1032), (4097, 2048, 4096)])
def test_forward_sizes(ia, M, K, N):
    check_forward(ia, M, K, N, 4, True, True)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("M", [5, 300, 3000])
@pytest.mark.parametrize("bias,res", [(True, False), (False, True)])
def test_forward_epilogues(ia, act, M, bias, res):
    check_forward(ia, M, 264, 1288, act, bias, res, seed=40)


@pytest.mark.parametrize("M", [0, 1, 40, 700, 2600])
def test_slices_and_rows_left_alone(ia, M):
    """x, W, the residual and the output as slices of wider arrays: the columns beside the
    output and the rows behind it stay as they were."""
    K, N = 200, 1096
    xs, Ws = normal((M + 3, K + 24), 1), normal((K, N + 64), 2, K ** -0.5)
    rs = normal((M + 2, N + 8), 3)
    out = torch.full((M + 5, N + 40), 7.0, dtype=BF, device="cuda")
    x, W, r, y = xs[:M, 8:8 + K], Ws[:, 32:32 + N], rs[:M, :N], out[:M, 16:16 + N]
    got = ia.infini_attn_linear(x, W, act=2, residual=r, out=y)
    ok(ia)
    assert got.data_ptr() == y.data_ptr()
    ry, ey, _, _ = ref.linear(x, W, None, 2, r)
    ref.within(y, ry, ey, ref.BF16)
    out[:M, 16:16 + N] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("M", [1, 200, 3000])
def test_residual_in_place(ia, M):
    x, W, b, r = inputs(M, 512, 1024, 9, True, True)
    want = ia.infini_attn_linear(x, W, bias=b, act=3, residual=r)
    got = ia.infini_attn_linear(x, W, bias=b, act=3, residual=r, out=r)
    ok(ia)
    assert got is r and torch.equal(want, r)


def test_leading_dimensions(ia):
    x, W = normal((2, 5, 64), 1), normal((64, 40), 2, 0.125)
    y = ia.infini_attn_linear(x, W)
    assert y.shape == (2, 5, 40)
    assert torch.equal(y.view(10, 40), ia.infini_attn_linear(x.view(10, 64), W))
    assert torch.equal(y[0, 0], ia.infini_attn_linear(x[0, 0].contiguous(), W)[:40])
    empty = ia.infini_attn_linear(x[:0], W)
    assert empty.shape == (0, 5, 40)


@pytest.mark.parametrize("M", [4, 300, 2600])
def test_not_a_number_stays_in_its_row(ia, M):
    """A NaN or an infinity in one row of x (or of the residual) leaves the others alone."""
    x, W, b, r = inputs(M, 136, 520, 5, True, True)
    clean = ia.infini_attn_linear(x, W, bias=b, act=1, residual=r)
    x[1, 3], r[2, 7] = float("nan"), float("inf")
    y = ia.infini_attn_linear(x, W, bias=b, act=1, residual=r)
    ok(ia)
    assert bool(y[1].isnan().all()) and y[2, 7] == float("inf")
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1], keep[2, 7] = False, False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M,K,N", [
    (1, 64, 64), (7, 8, 8), (64, 136, 72), (65, 1024, 256), (641, 512, 1408), (1000, 72, 2056),
    (4100, 1024, 1024), (20000, 128, 256), (3001, 2048, 4096)])
@pytest.mark.parametrize("act", [0, 4])
def test_backward_sizes(ia, M, K, N, act):
    check_backward(ia, M, K, N, act)


@pytest.mark.parametrize("act", range(5))
def test_backward_activations(ia, act):
    check_backward(ia, 333, 264, 520, act)


def check_backward(ia, M, K, N, act, seed=20):
    x, W, _, _ = inputs(M, K, N, seed)
    dy, pre = normal((M, N), seed + 5, 1.0 / M), normal((M, N), seed + 6, 2.0)
    if act == 1:
        pre[0, 0] = 0.0  # relu'(0) = 0
    dx, dW, db = ia.infini_attn_linear_backward(x, W, dy, act=act, preact=pre if act else None)
    ok(ia)
    for name, got, (r, e), step in zip(("dx", "dW", "dbias"), (dx, dW, db),
                                       ref.linear_backward(x, W, pre, dy, act),
                                       (ref.BF16, ref.BF16, ref.F32)):
        ref.within(got, r, e, step, name)


def test_backward_parts_and_strides(ia):
    """Each gradient alone equals the joint call's; strided operands; a caller workspace."""
    M, K, N = 700, 256, 520
    x, W = normal((M, K + 8), 1)[:, :K], normal((K, N + 8), 2, K ** -0.5)[:, 8:]
    dy, pre = normal((M, 2 * N), 3)[:, N:], normal((M, N + 16), 4)[:, :N]
    ws = torch.empty(ia.linear_backward_workspace_size(M, K, N, 2), dtype=torch.uint8,
                     device="cuda")
    all3 = ia.infini_attn_linear_backward(x, W, dy, act=2, preact=pre, workspace=ws)
    for i, kw in enumerate(({"x_grad": True}, {"W_grad": True}, {"bias_grad": True})):
        off = dict(x_grad=False, W_grad=False, bias_grad=False)
        off.update(kw)
        one = ia.infini_attn_linear_backward(x, W, dy, act=2, preact=pre, **off)
        assert [t is not None for t in one] == [j == i for j in range(3)]
        assert torch.equal(one[i], all3[i])
    ok(ia)
    for got, (r, e), step in zip(all3, ref.linear_backward(x, W, pre, dy, 2),
                                 (ref.BF16, ref.BF16, ref.F32)):
        ref.within(got, r, e, step)
    with pytest.raises(ia.InfiniError):
        ia.infini_attn_linear_backward(x, W, dy, act=2, preact=pre, workspace=ws[:256])


def test_backward_of_no_rows(ia):
    x, W = normal((0, 64), 1), normal((64, 32), 2)
    dx, dW, db = ia.infini_attn_linear_backward(x, W, normal((0, 32), 3))
    ok(ia)
    assert dx.shape == (0, 64) and not bool(dW.any()) and not bool(db.any())


def test_gradient_against_differences(ia):
    """The derivative of sum(dy * y) along random directions of x, W and the bias, from
    float64 differences of the reference forward, against the returned gradients."""
    M, K, N, act = 96, 136, 264, 4
    x, W, b, _ = inputs(M, K, N, 30)
    dy = normal((M, N), 35, 1.0 / M)
    _, pre = ia.infini_attn_linear(x, W, bias=b, act=act, save_preact=True)
    grads = ia.infini_attn_linear_backward(x, W, dy, act=act, preact=pre)
    ok(ia)
    f = lambda x, W, b: float((ref.act(x @ W + b, act) * dy.double()).sum())
    base = [t.double() for t in (x, W, b)]
    for i, g in enumerate(grads):
        d = normal(base[i].shape, 50 + i, dtype=torch.float64)
        h, up, down = 1e-5, list(base), list(base)
        up[i], down[i] = base[i] + h * d, base[i] - h * d
        slope = (f(*up) - f(*down)) / (2 * h)
        # gradients carry a relative bf16 rounding each of themselves, d and preact
        size = float((g.double().abs() * d.abs()).sum())
        assert abs(slope - float((g.double() * d).sum())) <= 4 * ref.BF16 * size


@pytest.mark.parametrize("M", [1, 48, 640, 3000])
def test_same_bits_every_time_on_two_streams_and_in_a_graph(ia, M):
    x, W, b, r = inputs(M, 1024, 1288, 60, True, True)
    want = ia.infini_attn_linear(x, W, bias=b, act=4, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):  # two streams at once
        outs.append(ia.infini_attn_linear(x, W, bias=b, act=4, residual=r))
        outs.append(ia.infini_attn_linear(x, W, bias=b, act=4, residual=r, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, want) for o in outs)
    dy = normal((M, 1288), 61, 0.1)
    grads = ia.infini_attn_linear_backward(x, W, dy)
    y = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ia.infini_attn_linear(x, W, bias=b, act=4, residual=r, out=y)
        again = ia.infini_attn_linear_backward(x, W, dy)
    for _ in range(3):
        y.zero_()
        g.replay()
        assert torch.equal(y, want)
        assert all(torch.equal(p, q) for p, q in zip(again, grads))
    x.copy_(normal(x.shape, 62))  # a replay reads what is in the buffers then
    g.replay()
    assert torch.equal(y, ia.infini_attn_linear(x, W, bias=b, act=4, residual=r))
    ok(ia)


def test_binding_refuses(ia):
    x, W = normal((8, 64), 1), normal((64, 32), 2)
    lin = ia.infini_attn_linear
    for bad in (lambda: lin(x.float(), W), lambda: lin(x, W.cpu()), lambda: lin(x, W.t()),
                lambda: lin(x, W[:32]), lambda: lin(x, W, bias=torch.zeros(32, dtype=BF).cuda()),
                lambda: lin(x, W, residual=x), lambda: lin(x, W, out=x),
                lambda: lin(x[:1].expand(8, 64), W),
                lambda: lin(x.view(2, 4, 64).transpose(0, 1), W),
                lambda: ia.infini_attn_linear_backward(x, W, normal((8, 32), 3), act=2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lin(x[:, :60].contiguous(), W[:60]), lambda: lin(x, W, act=17),
                lambda: lin(x[:, 4:60], W[:56]),
                lambda: lin(x, W, out=x[:, :32])):
        with pytest.raises(ia.InfiniError):
            bad()
