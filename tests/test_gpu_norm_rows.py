"""GPU tests of the norms: gates of an empty batch."""
import pytest
import torch

from test_gpu_norm import ia, normal  # noqa: F401

pytestmark = pytest.mark.gpu


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
