"""fp64 CPU oracle for one transformer block around the attention layer.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

  a = layer(norm(x; attn_norm))                   (oracle/layer.py)
  r = alpha x + attn_gate norm(a; attn_post_norm)
  f = act(norm(r; mlp_norm) W_up + b_up) W_down + b_down
  y = alpha r + mlp_gate norm(f; mlp_post_norm)

with norm(v; w, c) = v / sqrt(mean v^2 + eps) w, or (v - mean v) / sqrt(var v + eps) w + c,
over the last dimension; a post norm or a gate that is None is left out. Gates are
[groups, D_model], a batch row belonging to group (row * groups // rows).

Pinned in ``tests/test_oracle_block_pins.py``.
"""
from __future__ import annotations

import math

import numpy as np

from .layer import layer_forward, project


def norm(v, weight, bias=None, layer=False, eps=1e-5):
    v = np.asarray(v, dtype=np.float64)
    if layer:
        v = v - v.mean(-1, keepdims=True)
    n = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * weight
    return n if bias is None else n + bias


_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(v, act):
    """none, relu, silu, gelu, tanh gelu for act = 0..4."""
    if act == 1:
        return np.maximum(v, 0.0)
    if act == 2:
        return v / (1.0 + np.exp(-v))
    if act == 3:
        return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    if act == 4:
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def gated(u, gate):
    """u [B, L, D] times its rows' gates."""
    if gate is None:
        return u
    gate = np.asarray(gate, dtype=np.float64).reshape(-1, u.shape[-1])
    rows = u.reshape(-1, u.shape[-1])
    return (rows * np.repeat(gate, rows.shape[0] // gate.shape[0], axis=0)).reshape(u.shape)


def block_forward(x, Wq, Wk, Wv, Wo, beta, N, mode, H, H_kv, d, W_up, W_down, attn_norm,
                  mlp_norm, b_up=None, b_down=None, act=4, layer_norm=False, eps=1e-5, alpha=1.0,
                  attn_gate=None, mlp_gate=None, attn_post_norm=None, mlp_post_norm=None,
                  attn_norm_bias=None, mlp_norm_bias=None, attn_post_norm_bias=None,
                  mlp_post_norm_bias=None, M_in=None, z_in=None):
    """y [B, L, D_model] and the layer's final state (M, z)."""
    x = np.asarray(x, dtype=np.float64)
    nrm = lambda v, w, c: v if w is None else norm(v, w, c, layer_norm, eps)
    a, M, z = layer_forward(nrm(x, attn_norm, attn_norm_bias), Wq, Wk, Wv, Wo, beta, N, mode, H,
                            H_kv, d, M_in, z_in)
    r = alpha * x + gated(nrm(a, attn_post_norm, attn_post_norm_bias), attn_gate)
    m = project(nrm(r, mlp_norm, mlp_norm_bias), W_up) + (0.0 if b_up is None else b_up)
    f = project(activation(m, act), W_down) + (0.0 if b_down is None else b_down)
    return alpha * r + gated(nrm(f, mlp_post_norm, mlp_post_norm_bias), mlp_gate), M, z
