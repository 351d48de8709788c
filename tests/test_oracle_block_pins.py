"""Pins for the fp64 block oracle (oracle/block.py): its norms and activations against
torch's in float64, a block whose MLP and gates are switched off against the pinned layer,
and planted mistakes that have to show."""
import numpy as np
import pytest
import torch

import oracle.block as ob
import oracle.layer as ol

RNG = np.random.default_rng(77)


def test_norms_against_torch():
    v, w, c = RNG.standard_normal((3, 5, 8)), RNG.standard_normal(8), RNG.standard_normal(8)
    t = torch.from_numpy
    want = torch.nn.functional.layer_norm(t(v), (8,), t(w), t(c), 1e-3).numpy()
    assert np.allclose(ob.norm(v, w, c, True, 1e-3), want, rtol=0, atol=1e-13)
    want = torch.nn.functional.rms_norm(t(v), (8,), t(w), 1e-3).numpy()
    assert np.allclose(ob.norm(v, w, None, False, 1e-3), want, rtol=0, atol=1e-13)


def test_activations_against_torch():
    v = np.linspace(-6, 6, 101)
    F, t = torch.nn.functional, torch.from_numpy(v)
    for act, want in enumerate((t, F.relu(t), F.silu(t), F.gelu(t), F.gelu(t, approximate="tanh"))):
        assert np.allclose(ob.activation(v, act), want.numpy(), rtol=0, atol=1e-13)


def small():
    B, L, D, F, H, d = 2, 6, 8, 12, 2, 4
    n = RNG.standard_normal
    return dict(x=n((B, L, D)), Wq=n((D, H * d)), Wk=n((D, H * d)), Wv=n((D, H * d)),
                Wo=n((H * d, D)), beta=n(H), N=4, mode=1, H=H, H_kv=H, d=d, W_up=n((D, F)),
                W_down=n((F, D)), attn_norm=n(D), mlp_norm=n(D))


def test_switched_off_parts_leave_the_layer():
    p = small()
    p.update(mlp_gate=np.zeros((1, 8)), alpha=1.0)
    y, M, z = ob.block_forward(**p)
    a, M2, z2 = ol.layer_forward(ob.norm(p["x"], p["attn_norm"]), p["Wq"], p["Wk"], p["Wv"],
                                 p["Wo"], p["beta"], 4, 1, 2, 2, 4)
    assert np.allclose(y, p["x"] + a, rtol=0, atol=1e-12)
    assert np.array_equal(M, M2) and np.array_equal(z, z2)
    p.update(attn_gate=np.zeros((2, 8)), alpha=0.5)
    assert np.allclose(ob.block_forward(**p)[0], 0.25 * p["x"], rtol=0, atol=1e-13)


def test_gate_groups_are_batch_rows():
    u, gate = RNG.standard_normal((2, 3, 4)), RNG.standard_normal((2, 4))
    got = ob.gated(u, gate)
    for b in range(2):
        for l in range(3):
            assert np.allclose(got[b, l], u[b, l] * gate[b], rtol=0, atol=0)


@pytest.mark.parametrize("mistake", [dict(alpha=0.9), dict(act=3), dict(layer_norm=True),
                                     dict(attn_post_norm=np.ones(8)), dict(eps=1e-2),
                                     dict(b_up=np.full(12, 0.1))])
def test_planted_mistakes_show(mistake):
    p = small()
    assert not np.allclose(ob.block_forward(**p)[0], ob.block_forward(**{**p, **mistake})[0],
                           rtol=0, atol=1e-6)
