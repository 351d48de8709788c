"""GPU tests of the norms over many rows of every layout: the second and later rows of a
worker against float64, and sums over rows that count each row exactly once."""
import ctypes

import pytest
import torch

import block_ref as ref
from test_gpu_norm import BF, EPS, F32, case, ia, kwargs, normal, wide  # noqa: F401

pytestmark = pytest.mark.gpu

# every number of threads per row and piece size; enough rows for three or more per worker
# (a block works on 8, 4, 2 or 1 rows at a time, up to 296 blocks)
MANY = [(136, 9000), (257, 9000), (778, 5000), (777, 5000), (1024, 5000), (2056, 2500),
        (2047, 2500), (4094, 1500), (4095, 1500), (4096, 1500), (8184, 1100), (8191, 1100),
        (8192, 1100)]


def signs(rows, dim, seed, dtype):
    """Rows of +1 and -1 with a 0 in between for odd widths: their mean is 0, their mean
    square (dim or dim - 1) / dim, so that n(row) is the row times one factor."""
    g = torch.Generator().manual_seed(seed)
    half = dim // 2
    base = torch.cat([torch.ones(half), -torch.ones(half), torch.zeros(dim % 2)])
    order = torch.rand((rows, dim), generator=g).argsort(1)
    return base[order].to(dtype).cuda()


def whole(shape, seed, dtype=F32, most=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype).cuda()


def counted(got, want, factor, terms, name):
    """got is factor times a sum of whole numbers, of at most `terms` terms of magnitude
    up to 2: a row left out, or taken twice, would move some sum by 1 or more. An fp32 sum of
    the kernel's depth (rows of a worker, workers, blocks / 8, 8: below 128 additions here)
    is off by at most 128 2^-24 times the sum of the magnitudes, each term and the factor by a
    few roundings."""
    bound = 140 * ref.F32 * 2 * terms * factor + 2.0 ** -19 * want.abs() * factor
    assert float(bound.max()) < 0.4, "the case cannot tell one row"
    off = (got.double() - factor * want).abs()
    assert bool((off <= bound).all()), f"{name}: off by {float(off.max())}"


@pytest.mark.parametrize("dim,rows", MANY)
@pytest.mark.parametrize("groups", [1, 5])
@pytest.mark.parametrize("kind,dtype", [(0, BF), (1, BF), (0, F32), (1, F32)])
def test_every_row_is_counted_once(ia, dim, rows, groups, kind, dtype):
    """Sums over rows of whole numbers. From dr alone: d = dr, dgate = sum d u, dpost_weight =
    gate sum d n(b), dpost_bias = gate sum d. From dh alone, without b: dpre_weight =
    sum dh n(x), dpre_bias = sum dh."""
    x, b = signs(rows, dim, 1, dtype), signs(rows, dim, 2, dtype)
    dr, dh = whole((rows, dim), 3, dtype), whole((rows, dim), 4, dtype)
    gate = whole((groups, dim), 5) + 2.0 * (whole((groups, dim), 6) >= 0)  # -1 .. 3
    gate = gate.clamp(-2, 2)
    one, zero = torch.ones(dim, device="cuda"), torch.zeros(dim, device="cuda")
    bias = zero if kind else None
    d64, b64 = dr.double(), b.double()
    per_group = lambda t: t.view(groups, rows // groups, dim).sum(1)
    factor = (dim / (dim - dim % 2)) ** 0.5
    # without a post norm: u = b, exact
    got = ia.infini_attn_residual_norm_backward(x, b, dr, None, gate=gate, kind=kind, eps=0.0)
    assert torch.equal(got.dgate.double(), per_group(d64 * b64))
    got = ia.infini_attn_residual_norm_backward(x, b, dr, None, gate=gate, post_weight=one,
                                                post_bias=bias, kind=kind, eps=0.0)
    counted(got.dgate, per_group(d64 * b64), factor, rows // groups, "dgate")
    counted(got.dpost_weight, (gate.double() * per_group(d64 * b64)).sum(0), factor, rows,
            "dpost_weight")
    if kind:
        assert torch.equal(got.dpost_bias.double(), (gate.double() * per_group(d64)).sum(0))
    got = ia.infini_attn_residual_norm_backward(x, None, None, dh, pre_weight=one, pre_bias=bias,
                                                kind=kind, eps=0.0)
    counted(got.dpre_weight, (dh.double() * x.double()).sum(0), factor, rows, "dpre_weight")
    if kind:
        assert torch.equal(got.dpre_bias.double(), dh.double().sum(0))


@pytest.mark.parametrize("dim,rows", MANY)
@pytest.mark.parametrize("kind,dtype", [(0, BF), (1, BF), (0, F32), (1, F32)])
def test_later_rows_of_a_worker(ia, dim, rows, kind, dtype):
    """r, h, dx and db of every row, element by element."""
    a = case(rows, dim, dtype, kind, 5, True, seed=11)
    kw = kwargs(a, kind, 0.75)
    r, h = ia.infini_attn_residual_norm(a["x"], a["b"], **kw)
    rr, er, rh, eh = ref.residual_norm(*wide(a, 0.75, kind))
    ref.within(r, rr, er, ref.half_step(dtype), "r")
    ref.within(h, rh, eh, ref.half_step(dtype), "h")
    del rr, er, rh, eh
    dr, dh = normal((rows, dim), 18, 0.5, 0.0, dtype), normal((rows, dim), 19, 1.0, 0.0, dtype)
    got = ia.infini_attn_residual_norm_backward(a["x"], a["b"], dr, dh, **kw)
    args = (*wide(a, 0.75, kind), dr.double(), dh.double())
    want, sizes = ref.residual_norm_grads(*args), ref.residual_norm_grad_sizes(*args)
    for i, name in ((0, "dx"), (1, "db")):
        ref.within(got[i], want[i], ref.UNITS * sizes[i], ref.half_step(dtype), name)


@pytest.mark.parametrize("dim,rows", [(136, 9000), (1024, 5000), (4096, 1500), (777, 5000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_off_16_bytes_in_the_gradient(ia, dim, rows, dtype):
    """Storage that starts off a 16-byte boundary: other loads, the same gradients."""
    a = case(rows, dim, dtype, 1, 5, True, seed=21)
    dr, dh = normal((rows, dim), 28, 0.5, 0.0, dtype), normal((rows, dim), 29, 1.0, 0.0, dtype)

    def off(t):
        base = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        return base[1:].view(t.shape).copy_(t)

    o = {n: off(t) for n, t in a.items()}
    got = ia.infini_attn_residual_norm_backward(o["x"], o["b"], off(dr), off(dh),
                                                **kwargs(o, 1, 0.75))
    args = (*wide(a, 0.75, 1), dr.double(), dh.double())
    want, sizes = ref.residual_norm_grads(*args), ref.residual_norm_grad_sizes(*args)
    for i, name in ((0, "dx"), (1, "db")):
        ref.within(got[i], want[i], ref.UNITS * sizes[i], ref.half_step(dtype), name)


@pytest.mark.parametrize("dim,rows", [(77, 3000), (520, 5000), (1024, 3000), (4096, 1000),
                                      (8191, 500)])
@pytest.mark.parametrize("kind,dtype", [(0, BF), (1, BF), (0, F32), (1, F32)])
@pytest.mark.parametrize("dx,db", [("x", "b"), ("b", "x"), ("dr", "dh"), ("dh", "dr"),
                                   ("x", "dh"), ("dr", "b")])
def test_gradients_in_place(ia, dim, rows, kind, dtype, dx, db):
    """dx and db may each be x, b, dr or dh itself: bit for bit what other arrays get."""
    from compressive_memory_transformer_b200.block import ResidualNormArgs, ResidualNormGradArgs
    a = case(rows, dim, dtype, kind, 5, True, seed=31)
    t = dict(x=a["x"], b=a["b"], dr=normal((rows, dim), 38, 0.5, 0.0, dtype),
             dh=normal((rows, dim), 39, 1.0, 0.0, dtype))
    want = ia.infini_attn_residual_norm_backward(t["x"], t["b"], t["dr"], t["dh"],
                                                 **kwargs(a, kind, 0.75))
    t = {n: v.clone() for n, v in t.items()}
    p = lambda v: None if v is None else v.data_ptr()
    args = ResidualNormArgs(x=p(t["x"]), b=p(t["b"]), gate=p(a["gate"]), post_weight=p(a["pw"]),
                            post_bias=p(a["pb"]), pre_weight=p(a["w"]), pre_bias=p(a["c"]),
                            rows=rows, gate_groups=5, dim=dim, kind=kind,
                            dtype=ia.DTYPE_BF16 if dtype is BF else ia.DTYPE_F32, alpha=0.75,
                            eps=EPS)
    sums = [None if v is None else torch.empty_like(v) for v in want[2:]]
    grads = ResidualNormGradArgs(p(t["dr"]), p(t["dh"]), p(t[dx]), p(t[db]), *map(p, sums))
    st = ia.raw_call("infini_attn_residual_norm_backward", ctypes.byref(args), ctypes.byref(grads),
                     None, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    got = [t[dx], t[db], *sums]
    assert all(w is None or torch.equal(g, w) for g, w in zip(got, want))
    for n in set(t) - {dx, db}:  # what is not an output stays as it was
        fresh = case(rows, dim, dtype, kind, 5, True, seed=31)
        src = fresh[n] if n in fresh else normal((rows, dim), 38 if n == "dr" else 39,
                                                 0.5 if n == "dr" else 1.0, 0.0, dtype)
        assert torch.equal(t[n], src)


def test_a_gate_row_per_token_of_no_tokens(ia):
    """gate [rows, dim] of an empty batch: empty results, zero sums."""
    x, b, gate = normal((0, 64), 1), normal((0, 64), 2), normal((0, 64), 3)
    w = normal((64,), 4)
    r, h = ia.infini_attn_residual_norm(x, b, gate=gate, pre_weight=w)
    assert r.shape == h.shape == (0, 64)
    got = ia.infini_attn_residual_norm_backward(x, b, x, x, gate=gate, pre_weight=w)
    torch.cuda.synchronize()
    assert got.dx.shape == got.db.shape == got.dgate.shape == (0, 64)
    assert not bool(got.dpre_weight.any())
    with pytest.raises(ValueError):
        ia.infini_attn_residual_norm(w[None], w[None], gate=gate)


def test_block_refuses_a_gate_without_rows(ia):
    """A gate of no groups for a block with tokens is refused, not left out."""
    from test_gpu_block import block_case
    p = block_case(1, 128, 128, 264, 1, 1, 0, 0, False)
    none = torch.empty((0, 128), device="cuda")
    for gates in (dict(attn_gate=none), dict(mlp_gate=none),
                  dict(attn_gate=none, mlp_gate=torch.ones((1, 128), device="cuda"))):
        with pytest.raises(ValueError):
            ia.infini_attn_block_forward(**p, **gates)
