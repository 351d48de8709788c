"""Host checks of the operators around the attention layer that need no GPU: every bad
argument is refused before any CUDA call, by the C ABI with its status and by the binding
with a ValueError; the scratch sizes need no device."""
import ctypes

import pytest
import torch

NULL, SHAPE, UNSUPPORTED, ALIGN, NOMEM, ALIAS = -1, -2, -3, -4, -6, -8
FAKE = 1 << 20  # aligned addresses that are never read
MB = 1 << 24


@pytest.fixture(scope="module")
def ia():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import compressive_memory_transformer_b200 as m
    return m


def linear(ia, **kw):
    from compressive_memory_transformer_b200.block import LinearArgs
    a = dict(x=FAKE, W=FAKE + MB, bias=None, residual=None, y=FAKE + 2 * MB, preact=None, M=128,
             K=64, N=128, act=0)
    a.update(kw)
    return ia.raw_call("infini_attn_linear", ctypes.byref(LinearArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(y=None), NULL),
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(K=60), UNSUPPORTED), (dict(N=124), UNSUPPORTED), (dict(act=5), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED),
    (dict(ldx=56), SHAPE), (dict(ldx=68), SHAPE), (dict(ldw=120), SHAPE), (dict(ldy=-8), SHAPE),
    (dict(ldr=8), SHAPE), (dict(ldp=100), SHAPE), (dict(ldx=1 << 40), SHAPE),
    (dict(x=FAKE + 8), ALIGN), (dict(W=FAKE + MB + 2), ALIGN), (dict(bias=FAKE + 4), ALIGN),
    (dict(residual=FAKE + 8), ALIGN), (dict(y=FAKE + 2 * MB + 8), ALIGN),
    (dict(preact=FAKE + 2), ALIGN),
    (dict(y=FAKE), ALIAS), (dict(y=FAKE + MB), ALIAS), (dict(preact=FAKE), ALIAS),
    (dict(preact=FAKE + 2 * MB), ALIAS), (dict(bias=FAKE + 2 * MB), ALIAS),
    (dict(residual=FAKE + 2 * MB + 16), ALIAS),
    (dict(residual=FAKE + 2 * MB, ldr=256), ALIAS),         # y's place with other rows
    (dict(residual=FAKE + 3 * MB, preact=FAKE + 3 * MB), ALIAS),
])
def test_linear_refuses(ia, kw, code):
    assert linear(ia, **kw) == code


def test_linear_with_no_rows_is_nothing_to_do(ia):
    assert linear(ia, M=0, x=None, y=None) == 0
    assert ia.raw_call("infini_attn_linear", None, None) == NULL


def linear_grad(ia, opts=None, **kw):
    from compressive_memory_transformer_b200.block import LinearGradArgs
    a = dict(x=FAKE, W=FAKE + MB, preact=FAKE + 2 * MB, dy=FAKE + 3 * MB, dx=FAKE + 4 * MB,
             dW=FAKE + 5 * MB, dbias=FAKE + 6 * MB, M=128, K=64, N=128, act=2)
    a.update(kw)
    return ia.raw_call("infini_attn_linear_backward", ctypes.byref(LinearGradArgs(**a)), opts,
                       None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(dy=None), NULL), (dict(preact=None), NULL),
    (dict(dx=None, dW=None, dbias=None), NULL),
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=8, K=4), UNSUPPORTED),
    (dict(act=9), UNSUPPORTED), (dict(lddx=8), SHAPE), (dict(lddw=4), SHAPE),
    (dict(lddy=12), SHAPE),
    (dict(dx=FAKE + 4 * MB + 8), ALIGN), (dict(dbias=FAKE + 4), ALIGN), (dict(dy=FAKE + 2), ALIGN),
    (dict(dx=FAKE), ALIAS), (dict(dx=FAKE + 3 * MB), ALIAS), (dict(dW=FAKE + MB), ALIAS),
    (dict(dW=FAKE + 4 * MB), ALIAS), (dict(dbias=FAKE + 5 * MB), ALIAS),
    (dict(dbias=FAKE + 2 * MB), ALIAS),
])
def test_linear_backward_refuses(ia, kw, code):
    assert linear_grad(ia, **kw) == code


def norm(ia, grad=None, **kw):
    from compressive_memory_transformer_b200.block import ResidualNormArgs, ResidualNormGradArgs
    a = dict(x=FAKE, b=FAKE + MB, gate=FAKE + 2 * MB, post_weight=FAKE + 3 * MB, post_bias=None,
             pre_weight=FAKE + 4 * MB, pre_bias=None, r=FAKE + 5 * MB, h=FAKE + 6 * MB, rows=64,
             gate_groups=1, dim=128, kind=0, dtype=0, alpha=1.0, eps=1e-5)
    a.update(kw)
    p = ctypes.byref(ResidualNormArgs(**a))
    if grad is None:
        return ia.raw_call("infini_attn_residual_norm", p, None)
    g = dict(dr=FAKE + 7 * MB, dh=FAKE + 8 * MB, dx=FAKE + 9 * MB, db=FAKE + 10 * MB,
             dgate=FAKE + 11 * MB, dpost_weight=FAKE + 12 * MB, dpre_weight=FAKE + 13 * MB)
    g.update(grad)
    return ia.raw_call("infini_attn_residual_norm_backward", p,
                       ctypes.byref(ResidualNormGradArgs(**g)), None, None)


COMMON = [
    (dict(x=None), NULL), (dict(b=None), NULL), (dict(b=None, gate=None), NULL),
    (dict(pre_bias=FAKE, pre_weight=None, h=None, kind=1), NULL),
    (dict(post_bias=FAKE, post_weight=None, kind=1), NULL),
    (dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(gate_groups=0), SHAPE),
    (dict(gate_groups=7), SHAPE), (dict(gate_groups=128), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE),
    (dict(dim=8193), UNSUPPORTED), (dict(kind=2), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(pre_bias=FAKE), UNSUPPORTED), (dict(post_bias=FAKE), UNSUPPORTED),
    (dict(x=FAKE + 1), ALIGN), (dict(gate=FAKE + 2), ALIGN), (dict(dtype=1, b=FAKE + 2), ALIGN),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(r=None, h=None), NULL), (dict(pre_weight=None), NULL),
    (dict(h=FAKE + 1), ALIGN),
    (dict(r=FAKE + 16), ALIAS), (dict(h=FAKE + MB - 256), ALIAS), (dict(h=FAKE + 5 * MB), ALIAS),
    (dict(r=FAKE, h=FAKE), ALIAS), (dict(r=FAKE + 2 * MB), ALIAS), (dict(h=FAKE + 4 * MB), ALIAS),
])
def test_residual_norm_refuses(ia, kw, code):
    assert norm(ia, **kw) == code


@pytest.mark.parametrize("kw,grad,code", [(kw, {}, code) for kw, code in COMMON] + [
    ({}, dict(dr=None, dh=None), NULL), (dict(pre_weight=None), dict(dpre_weight=None), NULL),
    (dict(pre_weight=None), dict(dh=None), NULL),
    (dict(b=None, gate=None, post_weight=None), dict(dgate=None, dpost_weight=None), NULL),
    (dict(gate=None), {}, NULL), (dict(post_weight=None), {}, NULL),
    ({}, dict(dpre_bias=FAKE + 14 * MB), NULL), ({}, dict(dpost_bias=FAKE + 14 * MB), NULL),
    ({}, dict(dx=FAKE + 1), ALIGN), ({}, dict(dgate=FAKE + 11 * MB + 1), ALIGN),
    ({}, dict(dx=FAKE + 16), ALIAS), ({}, dict(db=FAKE + 9 * MB), ALIAS),
    ({}, dict(dgate=FAKE + 2 * MB), ALIAS), ({}, dict(dpre_weight=FAKE), ALIAS),
    ({}, dict(dpost_weight=FAKE + 13 * MB), ALIAS),
])
def test_residual_norm_backward_refuses(ia, kw, grad, code):
    assert norm(ia, grad, **kw) == code


def test_empty_norms_and_plain_norm(ia):
    assert norm(ia, rows=0) == 0
    call = lambda *a: ia.raw_call("infini_attn_norm", *a)
    assert call(FAKE, None, None, FAKE + MB, 4, 128, 0, 0, 1e-5, None) == NULL
    assert call(FAKE, FAKE + 2 * MB, None, None, 4, 128, 0, 0, 1e-5, None) == NULL
    assert call(FAKE, FAKE + 2 * MB, FAKE + 3 * MB, FAKE + MB, 4, 128, 0, 0, 1e-5,
                None) == UNSUPPORTED
    back = lambda *a: ia.raw_call("infini_attn_norm_backward", *a)
    assert back(FAKE, None, FAKE, FAKE, None, None, 4, 128, 0, 0, 1e-5, None, None) == NULL
    assert back(FAKE, FAKE + MB, None, FAKE, None, None, 4, 128, 0, 0, 1e-5, None, None) == NULL
    assert back(FAKE, FAKE + MB, FAKE, FAKE, None, FAKE + 2 * MB, 4, 128, 0, 0, 1e-5, None,
                None) == UNSUPPORTED  # a bias with the rms kind


def block(ia, **kw):
    from compressive_memory_transformer_b200.block import BlockArgs
    ptrs = ["x", "Wq", "Wk", "Wv", "Wo", "beta", "attn_norm", "mlp_norm", "W_up", "W_down", "y"]
    a = {n: FAKE + i * MB for i, n in enumerate(ptrs)}
    a.update(B=1, L=128, D_model=256, D_ff=512, H=2, H_kv=1, N=128, d=128, mode=0, act=4, kind=0,
             alpha=1.0, eps=1e-5)
    a.update(kw)
    return ia.raw_call("infini_attn_block_forward", ctypes.byref(BlockArgs(**a)), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(Wo=None), NULL), (dict(beta=None), NULL), (dict(W_up=None), NULL),
    (dict(attn_norm=None), NULL), (dict(mlp_norm=None), NULL), (dict(y=None), NULL),
    (dict(M_in=FAKE), NULL), (dict(z_out=FAKE), NULL), (dict(attn_post_norm_bias=FAKE), NULL),
    (dict(B=0), SHAPE), (dict(L=0), SHAPE), (dict(H=3, H_kv=2), SHAPE), (dict(N=0), SHAPE),
    (dict(L=1 << 31), SHAPE), (dict(attn_gate=FAKE + 20 * MB), SHAPE),
    (dict(mlp_gate=FAKE + 20 * MB, gate_groups=3), SHAPE),
    (dict(L=100), UNSUPPORTED), (dict(D_model=192), UNSUPPORTED), (dict(D_ff=12), UNSUPPORTED),
    (dict(d=64), UNSUPPORTED), (dict(mode=3), UNSUPPORTED), (dict(act=7), UNSUPPORTED),
    (dict(kind=4), UNSUPPORTED), (dict(D_model=8320), UNSUPPORTED),
    (dict(attn_norm_bias=FAKE + 20 * MB), UNSUPPORTED),
    (dict(x=FAKE + 8), ALIGN), (dict(W_down=FAKE + 8), ALIGN), (dict(mlp_norm=FAKE + 2), ALIGN),
    (dict(b_up=FAKE + 20 * MB + 4), ALIGN),
    (dict(y=FAKE), ALIAS), (dict(y=FAKE + 8 * MB), ALIAS), (dict(y=FAKE + 6 * MB), ALIAS),
    (dict(M_out=FAKE + 64, z_out=FAKE + 20 * MB), ALIAS),
])
def test_block_refuses(ia, kw, code):
    assert block(ia, **kw) == code


def test_scratch_sizes(ia):
    assert ia.linear_backward_workspace_size(0, 64, 64, 1) == 0
    assert ia.linear_backward_workspace_size(64, 60, 64, 1) == 0
    assert ia.linear_backward_workspace_size(1024, 64, 128, ia.ACT_SILU) >= 1024 * 128 * 2
    assert ia.residual_norm_backward_workspace_size(0, 64) == 0
    assert ia.residual_norm_backward_workspace_size(10, 64, 3) == 0
    assert ia.residual_norm_backward_workspace_size(64, 64, 2, ia.NORM_LAYER) >= 4 * 64 * 4
    assert ia.block_workspace_size(1, 100, 256, 512, 2, 2, 128) == 0
    assert ia.block_workspace_size(1, 128, 256, 512, 2, 2, 128) >= 128 * (3 * 256 + 512) * 2


def test_binding_refuses_tensors(ia):
    """What the binding itself refuses, on tensors that are not on a GPU (which is one of
    the refusals) or that no matrix in memory can be."""
    x, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ia.infini_attn_linear(x, W)
    with pytest.raises(ValueError):
        ia.infini_attn_linear_backward(x, W, torch.zeros(4, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ia.infini_attn_residual_norm(x, x, pre_weight=torch.ones(64))
    with pytest.raises(ValueError):
        ia.infini_attn_residual_norm_backward(x, x, x, None)
    with pytest.raises(ValueError):
        ia.infini_attn_norm(x, torch.ones(64))
