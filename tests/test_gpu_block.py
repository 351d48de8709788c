"""GPU tests of the operators around the attention layer as they are used together: the
whole block (infini_attn_block_forward) against its fp64 oracle and against its own steps,
and a training step of an MLP half against float64 differentiation.

Tolerances. The layer's own is 1e-2 (rel-F, tests/test_gpu_layer.py). Around it every step
rounds its result to bf16 once, at most 2^-8 relative per element, and the chain from x to
y has four such roundings (h, r, h, m) before y's own: rel-F <= 1e-2 + 5 * 2^-8 = 3e-2 in the
worst case. A training step's gradients pass h, the pre-activation, m, dm, d and the result's
own rounding: six of at most 2^-8, rel-F <= 2.4e-2."""
import numpy as np
import pytest
import torch

import block_ref as ref
import oracle.block as ob
from parity import f64, relf

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


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


def block_case(B, L, D, F, H, Hkv, mode, kind, full, groups=0, state=False, seed=0):
    w = lambda i, r, c: normal((r, c), seed + i, r ** -0.5, dtype=BF)
    v = lambda i, n, s=0.1, m=1.0: normal((n,), seed + i, s, m)
    p = dict(x=normal((B, L, D), seed, dtype=BF), Wq=w(1, D, H * 128), Wk=w(2, D, Hkv * 128),
             Wv=w(3, D, Hkv * 128), Wo=w(4, H * 128, D), beta=v(5, H, 1.0, 0.0), N=128, mode=mode,
             H=H, H_kv=Hkv, W_up=w(6, D, F), W_down=w(7, F, D), attn_norm=v(8, D),
             mlp_norm=v(9, D), act=4)
    if full:
        p.update(b_up=v(10, F, 0.1, 0.0), b_down=v(11, D, 0.1, 0.0), alpha=0.75,
                 attn_post_norm=v(12, D), mlp_post_norm=v(13, D))
    if kind:
        p.update(attn_norm_bias=v(14, D, 0.1, 0.0), mlp_norm_bias=v(15, D, 0.1, 0.0))
        if full:
            p.update(attn_post_norm_bias=v(16, D, 0.1, 0.0), mlp_post_norm_bias=v(17, D, 0.1, 0.0))
    if groups:
        p.update(attn_gate=normal((groups, D), seed + 18, 0.2, 0.5),
                 mlp_gate=normal((groups, D), seed + 19, 0.2, 0.5))
    if state:
        p.update(M_in=normal((B, Hkv, 128, 128), seed + 20, 3.0),
                 z_in=(1 + normal((B, Hkv, 128), seed + 21).abs()) * 50)
    return p


@pytest.mark.parametrize("B,L,D,F,H,Hkv,mode,kind,full,groups,state", [
    (1, 256, 256, 512, 2, 2, 0, 0, False, 0, False),
    (2, 320, 256, 680, 4, 2, 1, 0, True, 2, True),
    (1, 384, 384, 1024, 2, 1, 1, 1, True, 1, False),
    (2, 128, 128, 264, 1, 1, 0, 1, False, 0, True)])
def test_block_matches_the_oracle(ia, B, L, D, F, H, Hkv, mode, kind, full, groups, state):
    p = block_case(B, L, D, F, H, Hkv, mode, kind, full, groups, state)
    y, M, z = ia.infini_attn_block_forward(**p, kind=kind)
    torch.cuda.synchronize()
    assert ia.device_status() == 0
    q = {n: f64(t) if isinstance(t, torch.Tensor) else t for n, t in p.items()}
    ry, rM, rz = ob.block_forward(**q, d=128, layer_norm=bool(kind))
    assert relf(f64(y), ry) <= 3e-2
    assert relf(f64(M), rM) <= 1e-2 and relf(f64(z), rz) <= 1e-2


def test_block_is_its_steps(ia):
    """Bitwise: the block equals its public steps one after another; the caller's workspace,
    stage events, another stream and a captured graph change nothing."""
    p = block_case(2, 256, 256, 512, 2, 1, 1, 0, True, 2)
    want, M, z = ia.infini_attn_block_forward(**p)
    h = ia.infini_attn_norm(p["x"], p["attn_norm"])
    a, M2, z2 = ia.infini_attn_layer_forward(h, p["Wq"], p["Wk"], p["Wv"], p["Wo"], p["beta"], 128,
                                             1, 2, 1)
    r, h = ia.infini_attn_residual_norm(p["x"], a, gate=p["attn_gate"], alpha=0.75,
                                        post_weight=p["attn_post_norm"], pre_weight=p["mlp_norm"])
    m = ia.infini_attn_linear(h, p["W_up"], bias=p["b_up"], act=ia.ACT_GELU_TANH)
    f = ia.infini_attn_linear(m, p["W_down"], bias=p["b_down"])
    y, none = ia.infini_attn_residual_norm(r, f, gate=p["mlp_gate"], alpha=0.75,
                                           post_weight=p["mlp_post_norm"])
    assert none is None and torch.equal(y, want) and torch.equal(M, M2) and torch.equal(z, z2)
    ws = torch.empty(ia.block_workspace_size(2, 256, 256, 512, 2, 1, 128), dtype=torch.uint8,
                     device="cuda")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in ev:
        e.record()
    got = ia.infini_attn_block_forward(**p, workspace=ws, stage_events=ev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ia.infini_attn_block_forward(**p, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(other[0], want)
    assert ev[0].elapsed_time(ev[1]) >= 0 and ev[1].elapsed_time(ev[2]) >= 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = ia.infini_attn_block_forward(**p)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[0], want)
    assert ia.device_status() == 0


def test_block_with_the_plain_residual_in_the_epilogue(ia):
    """alpha = 1 without a post norm or a gate: the residual is added in the down
    projection's epilogue, with one rounding less."""
    p = block_case(1, 256, 256, 512, 2, 2, 0, 0, False)
    y, _, _ = ia.infini_attn_block_forward(**p)
    h = ia.infini_attn_norm(p["x"], p["attn_norm"])
    a, _, _ = ia.infini_attn_layer_forward(h, p["Wq"], p["Wk"], p["Wv"], p["Wo"], p["beta"], 128, 0,
                                           2)
    r, h = ia.infini_attn_residual_norm(p["x"], a, pre_weight=p["mlp_norm"])
    m = ia.infini_attn_linear(h, p["W_up"], act=ia.ACT_GELU_TANH)
    assert torch.equal(y, ia.infini_attn_linear(m, p["W_down"], residual=r))


@pytest.mark.parametrize("tokens", [1, 77, 1500])
@pytest.mark.parametrize("kind", [0, 1])
def test_training_step_of_an_mlp(ia, tokens, kind):
    """norm after the attention with gate and residual, up projection, down projection onto
    the residual stream, and back: every gradient against float64 differentiation."""
    D, F, act = 264, 1096, 3
    x, a = normal((tokens, D), 1, dtype=BF), normal((tokens, D), 2, dtype=BF)
    v = dict(gate=normal((D,), 3, 0.2, 0.5), pw=normal((D,), 4, 0.1, 1.0),
             w=normal((D,), 5, 0.1, 1.0), b1=normal((F,), 6, 0.1), b2=normal((D,), 7, 0.1))
    W1, W2 = normal((D, F), 8, D ** -0.5, dtype=BF), normal((F, D), 9, F ** -0.5, dtype=BF)
    dy = normal((tokens, D), 10, 1.0 / tokens, dtype=BF)
    kw = dict(gate=v["gate"], alpha=0.75, post_weight=v["pw"], pre_weight=v["w"], kind=kind)
    r, h = ia.infini_attn_residual_norm(x, a, **kw)
    m, pre = ia.infini_attn_linear(h, W1, bias=v["b1"], act=act, save_preact=True)
    y = ia.infini_attn_linear(m, W2, bias=v["b2"], residual=r)
    dm, dW2, db2 = ia.infini_attn_linear_backward(m, W2, dy)
    dh, dW1, db1 = ia.infini_attn_linear_backward(h, W1, dm, act=act, preact=pre)
    g = ia.infini_attn_residual_norm_backward(x, a, dy, dh, **kw)
    torch.cuda.synchronize()
    assert ia.device_status() == 0
    t = {n: q.double().requires_grad_() for n, q in
         dict(x=x, a=a, W1=W1, W2=W2, **v).items()}
    rr, _, hh, _ = ref.residual_norm(t["x"], t["a"], t["gate"], 0.75, t["pw"], None, t["w"], None,
                                     kind, 1e-5)
    yy = ref.act(hh @ t["W1"] + t["b1"], act) @ t["W2"] + t["b2"] + rr
    assert relf(f64(y), yy.detach().cpu().numpy()) <= 2.4e-2
    want = torch.autograd.grad((yy * dy.double()).sum(), list(t.values()))
    got = dict(x=g.dx, a=g.db, W1=dW1, W2=dW2, gate=g.dgate, pw=g.dpost_weight, w=g.dpre_weight,
               b1=db1, b2=db2)
    for n, w in zip(t, want):
        assert relf(f64(got[n]), w.cpu().numpy()) <= 2.4e-2, n
    assert np.isfinite(f64(y)).all()
