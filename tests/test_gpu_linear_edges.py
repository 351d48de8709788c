"""GPU tests of the linear layer where its first tests do not reach: activations far out on
their negative side and at huge values, slices of one wide array, an empty batch's events,
and products whose reduction is split over pairs of SMs."""
import math

import pytest
import torch

import block_ref as ref
from test_gpu_linear import BF, ia, inputs, normal, ok  # noqa: F401

pytestmark = pytest.mark.gpu


def far_values(lo, hi):
    """Every bf16 value from -hi to -lo."""
    bits = torch.arange(0x10000, dtype=torch.int32).to(torch.int16).view(BF)
    v = bits[torch.isfinite(bits) & (bits <= -lo) & (bits >= -hi)]
    return v.sort().values


def tail_error(v):
    """Relative error that a normal tail Phi(-|v|) = exp(-v^2 / 2) q(|v|) may have in fp32:
    2^-18 for q (a fit within 2^-20, its roundings and a reciprocal), and v^2 2^-22 for the
    exponential, whose argument v^2 log2(e) / 2 has up to three roundings of 2^-24 relative,
    times ln 2."""
    return 2.0 ** -18 + v * v * 2.0 ** -22


@pytest.mark.parametrize("rows,cols", [(40, 8), (400, 72), (4096, 1024)])
def test_gelu_of_negative_values(ia, rows, cols):
    """gelu(v) = -|v| Phi(-|v|) for v < 0: nothing larger stands beside the tail, so it has to
    be right relative to itself. pre is one product with 1, exact."""
    v = far_values(2.0, 13.0)
    # all of them over and over, or as many as there are rows
    pick = torch.arange(rows) % len(v) if rows >= len(v) else \
        torch.linspace(0, len(v) - 1, rows).long()
    v = v[pick].cuda()
    x = torch.zeros(rows, 8, dtype=BF, device="cuda")
    x[:, 0] = v
    W = torch.zeros(8, cols, dtype=BF, device="cuda")
    W[0] = 1.0
    y, pre = ia.infini_attn_linear(x, W, act=ia.ACT_GELU, save_preact=True)
    ok(ia)
    assert torch.equal(pre, v[:, None].expand(rows, cols))
    d = v.double()
    want = -d.abs() * torch.erfc(d.abs() / math.sqrt(2)) / 2
    bound = want.abs() * (ref.BF16 + tail_error(d)) + 2.0 ** -120
    off = (y.double() - want[:, None]).abs() / bound[:, None]
    assert float(off.max()) <= 1.0


def test_gelu_derivative_of_negative_values(ia):
    """gelu'(v) = Phi(v) + v phi(v), in fp32: with one row and dy = 1, dbias is act'(pre)."""
    v = far_values(0.25, 12.0)
    v = v[: len(v) // 8 * 8].cuda()
    n = len(v)
    one = torch.ones(1, n, dtype=BF, device="cuda")
    _, _, got = ia.infini_attn_linear_backward(
        torch.zeros(1, 8, dtype=BF, device="cuda"), torch.zeros(8, n, dtype=BF, device="cuda"),
        one, act=ia.ACT_GELU, preact=v[None])
    ok(ia)
    d = v.double()
    tail = torch.erfc(d.abs() / math.sqrt(2)) / 2
    slope = d * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    bound = (tail + slope.abs()) * tail_error(d) + 2.0 ** -120
    assert float(((got.double() - (tail + slope)).abs() / bound).max()) <= 1.0


@pytest.mark.parametrize("act", [1, 2, 3, 4])
def test_huge_values(ia, act):
    """Values whose squares overflow fp32: every activation here is v or 0 there, its
    derivative 1 or 0."""
    big = torch.tensor([100.0, 1e10, 1.8e19, 2e19, 1e20, 1e30, 3e38, 3.3e38])
    v = torch.cat([big, -big]).to(BF).cuda()
    x = torch.zeros(16, 8, dtype=BF, device="cuda")
    x[:, 0] = v
    W = torch.zeros(8, 8, dtype=BF, device="cuda")
    W[0] = 1.0
    y = ia.infini_attn_linear(x, W, act=act)
    want = torch.where(v > 0, v, torch.zeros_like(v))[:, None].expand(16, 8)
    assert bool((y == want).all())
    for rows in (1, 2000):  # few rows and many take different kernels
        dy = torch.ones(rows, 16, dtype=BF, device="cuda")
        pre = v[None].expand(rows, 16).contiguous()
        _, _, got = ia.infini_attn_linear_backward(
            torch.zeros(rows, 8, dtype=BF, device="cuda"),
            torch.zeros(8, 16, dtype=BF, device="cuda"), dy, act=act, preact=pre)
        # sums of `rows` ones (or zeros) are exact in fp32
        assert torch.equal(got, rows * (v > 0).float())
    ok(ia)


@pytest.mark.parametrize("M", [1, 40, 700, 2600])
def test_slices_of_one_array(ia, M):
    """x, the residual and the output as columns of one array: results as from arrays of
    their own, and the other columns stay as they were."""
    K, N = 200, 1096
    wide = normal((M, 8 + K + N + N + 16), 1)
    x, r, y = wide[:, 8:8 + K], wide[:, 8 + K:8 + K + N], wide[:, 16 + K + N:16 + K + 2 * N]
    W, b = normal((K, N), 2, K ** -0.5), normal((N,), 3, 0.5, torch.float32)
    kw = dict(bias=b, act=ia.ACT_SILU)
    want = ia.infini_attn_linear(x.contiguous(), W, residual=r.contiguous(), **kw)
    before = wide.clone()
    ia.infini_attn_linear(x, W, residual=r, out=y, **kw)
    ok(ia)
    assert torch.equal(y, want)
    y.copy_(before[:, 16 + K + N:16 + K + 2 * N])
    assert torch.equal(wide, before)
    ia.infini_attn_linear(x, W, residual=r, out=r, **kw)
    ok(ia)
    assert torch.equal(r, want)
    r.copy_(before[:, 8 + K:8 + K + N])
    assert torch.equal(wide, before)
    with pytest.raises(ia.InfiniError):  # eight columns of the residual
        ia.infini_attn_linear(x, W, residual=r, out=wide[:, K + N:K + 2 * N], **kw)


def test_events_of_an_empty_batch(ia):
    """The stage events are recorded for no rows too."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in ev:
        e.record()
    busy = normal((4096, 4096), 1, dtype=torch.float32)
    for _ in range(4):
        busy = busy * 0.5
    mark = torch.cuda.Event(enable_timing=True)
    mark.record()
    x, W, dy = normal((0, 64), 1), normal((64, 32), 2), normal((0, 32), 3)
    ia.infini_attn_linear_backward(x, W, dy, stage_events=ev)
    torch.cuda.synchronize()
    times = [mark.elapsed_time(e) for e in ev]
    assert 0 <= times[0] <= times[1] <= times[2]


# parts of the reduction per pair of SMs in dW or dx, by the scratch that they need: the
# partial tiles are fp32. Ragged in all three sizes; 6 parts of 98 k-steps are uneven.
@pytest.mark.parametrize("M,K,N,of", [(8192, 1024, 1024, "dW"), (6838, 616, 1120, "dW"),
                                      (6266, 2808, 216, "dW"), (40000, 512, 512, "dW"),
                                      (1513, 928, 3200, "dx")])
@pytest.mark.parametrize("act", [0, 2])
def test_reduction_split_over_pairs(ia, M, K, N, of, act):
    size = ia.linear_backward_workspace_size(M, K, N, act)
    outputs = K * N if of == "dW" else M * K
    d_bytes = 2 * M * N + 256 if act else 0
    bias_parts = 4 * 450 * N if M > 1024 else 0  # a row of dbias per chunk at most
    assert size > d_bytes + bias_parts + 2 * 4 * outputs * 0.99, "the case is not split any more"
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    x, W, _, _ = inputs(M, K, N, 80)
    dy, pre = normal((M, N), 85, 1.0 / M), normal((M, N), 86, 2.0)
    run = lambda ws: ia.infini_attn_linear_backward(x, W, dy, act=act, preact=pre if act else None,
                                                    workspace=ws)
    got = run(room[:size])
    ok(ia)
    assert bool((room[size:] == 0xA5).all())
    for name, g, (r, e), step in zip(("dx", "dW", "dbias"), got,
                                     ref.linear_backward(x, W, pre, dy, act),
                                     (ref.BF16, ref.BF16, ref.F32)):
        ref.within(g, r, e, step, name)
    assert all(torch.equal(p, q) for p, q in zip(got, run(None)))
