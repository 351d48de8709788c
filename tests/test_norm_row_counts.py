"""The check behind the sums over rows (test_gpu_norm_rows.counted), on the CPU: it passes a
sum that the worst fp32 rounding allows, and not one that leaves a row out or takes it twice."""
import pytest
import torch

from block_ref import F32
from test_gpu_norm_rows import MANY, counted, signs, whole


@pytest.mark.parametrize("dim", [136, 777])
def test_one_row_shows(dim, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)
    rows = 500
    n, d = signs(rows, dim, 1, torch.float32).double(), whole((rows, dim), 2).double()
    assert bool((n.sum(1) == 0).all()) and bool((n.abs().sum(1) == dim - dim % 2).all())
    factor = (dim / (dim - dim % 2)) ** 0.5
    most = max(r for _, r in MANY)
    want = (d * n).sum(0)
    counted(factor * want + 120 * F32 * rows, want, factor, most, "rounding")
    for bad in (want - d[7] * n[7], want + d[499] * n[499], torch.zeros_like(want)):
        with pytest.raises(AssertionError, match="off by"):
            counted(factor * bad, want, factor, most, "a row")
