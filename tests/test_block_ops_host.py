"""Host side of the operators around the attention layer that needs no GPU: which
neighbouring slices of one wide array a call may take, the scratch sizes of sizes that are
refused, empty gates, and the import without torch's CUDA build."""
import ctypes
import os
import subprocess
import sys

import pytest

SHAPE, CUDA, NOMEM, ALIAS = -2, -5, -6, -8
FAKE = 1 << 20  # aligned addresses that are never read
MB = 1 << 24
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ia():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import compressive_memory_transformer_b200 as m
    return m


def linear(ia, **kw):
    from compressive_memory_transformer_b200.block import LinearArgs
    a = dict(x=FAKE, W=FAKE + MB, y=FAKE + 2 * MB, M=128, K=64, N=128)
    a.update(kw)
    return ia.raw_call("infini_attn_linear", ctypes.byref(LinearArgs(**a)), None)


def grad(ia, **kw):
    """A gradient call that ends before any launch: with no alias for want of a device or,
    where there is one, of scratch (one byte is offered, act' needs more)."""
    from compressive_memory_transformer_b200 import Opts
    from compressive_memory_transformer_b200.block import LinearGradArgs
    a = dict(x=FAKE, W=FAKE + MB, preact=FAKE + 2 * MB, dy=FAKE + 3 * MB, dx=FAKE + 4 * MB,
             dW=FAKE + 5 * MB, dbias=FAKE + 6 * MB, M=128, K=64, N=128, act=2)
    a.update(kw)
    o = Opts()
    o.workspace, o.workspace_bytes = FAKE, 1
    st = ia.raw_call("infini_attn_linear_backward", ctypes.byref(LinearGradArgs(**a)),
                     ctypes.byref(o), None)
    assert st in (ALIAS, CUDA, NOMEM)
    return st


def overlaps(rows_a, cols_a, ld_a, a, rows_b, cols_b, ld_b, b):
    """Whether two matrices of 2-byte elements at byte addresses a and b share an element."""
    own = {a // 2 + i * ld_a + j for i in range(rows_a) for j in range(cols_a)}
    return any(b // 2 + i * ld_b + j in own for i in range(rows_b) for j in range(cols_b))


@pytest.mark.parametrize("first", [0, 8, 56, 64, 72, 128, 136, 192, 200, 256, 320, 376, 448])
@pytest.mark.parametrize("back", [0, 3])
def test_columns_of_one_wide_array(ia, first, back):
    """dx [128][64] from column 64 of an array 256 wide, dy [128][128] from any column, in the
    same rows or from three rows earlier on: an alias where elements are shared, only there."""
    dx, dy = FAKE + 2 * 64, FAKE + 2 * first - 2 * 256 * back
    want = overlaps(128, 64, 256, dx, 128, 128, 256, dy)
    got = grad(ia, x=FAKE + 7 * MB, dx=dx, dy=dy, lddx=256, lddy=256)
    assert (got == ALIAS) == want


def test_columns_beside_each_other(ia):
    """x, preact, dy and dx as columns of one array, W and dW of another."""
    at = lambda col: FAKE + 2 * col
    one = dict(x=at(0), preact=at(64), dy=at(192), dx=at(320), ldx=512, ldp=512, lddy=512,
               lddx=512)
    assert grad(ia, **one) != ALIAS
    assert grad(ia, **{**one, "dx": at(312)}) == ALIAS  # into dy
    assert grad(ia, **{**one, "dx": at(456)}) == ALIAS  # into the next row's x
    # another row stride: judged by the whole address range
    assert grad(ia, **{**one, "lddx": 520}) == ALIAS
    two = dict(ldw=256, lddw=256)
    assert grad(ia, dW=FAKE + MB + 256, **two) != ALIAS
    assert grad(ia, dW=FAKE + MB + 240, **two) == ALIAS


def test_shared_columns_are_refused(ia):
    """The forward's outputs in the columns of x, the residual or each other."""
    at = lambda col: FAKE + 2 * col
    ld = dict(x=at(0), ldx=512, ldr=512, ldy=512, ldp=512)
    for kw in (dict(residual=at(64), y=at(192), preact=at(312)),
               dict(residual=at(72), y=at(192), preact=at(320)),
               dict(residual=at(64), y=at(192), preact=at(392)),  # into the next row's x
               dict(residual=at(64), y=at(72), preact=at(320)),
               dict(y=at(192), ldy=520)):
        assert linear(ia, **{**ld, **kw}) == ALIAS


@pytest.mark.parametrize("kw", [
    dict(D_model=192), dict(D_model=8320), dict(D_ff=12), dict(mode=3), dict(mode=-1),
    dict(L=100), dict(d=64), dict(H=3, H_kv=2), dict(N=0), dict(B=0), dict(L=1 << 31)])
def test_block_scratch_of_unsupported_sizes_is_zero(ia, kw):
    a = dict(B=1, L=128, D_model=256, D_ff=512, H=2, H_kv=1, N=128, d=128, mode=0)
    assert ia.block_workspace_size(**a) > 0
    a.update(kw)
    assert ia.block_workspace_size(**a) == 0


def test_a_gate_row_per_token_of_no_tokens(ia):
    """`rows` gate groups are allowed, 0 rows too; with rows there has to be a group."""
    from compressive_memory_transformer_b200.block import ResidualNormArgs, ResidualNormGradArgs
    a = dict(x=FAKE, b=FAKE + MB, gate=FAKE + 2 * MB, pre_weight=FAKE + 4 * MB, r=FAKE + 5 * MB,
             h=FAKE + 6 * MB, rows=0, gate_groups=0, dim=128, kind=0, dtype=0, alpha=1.0, eps=1e-5)
    call = lambda: ia.raw_call("infini_attn_residual_norm", ctypes.byref(ResidualNormArgs(**a)),
                               None)
    assert call() == 0
    a["rows"] = 4
    assert call() == SHAPE
    g = ResidualNormGradArgs(dr=FAKE + 7 * MB, dgate=FAKE + 8 * MB)
    assert ia.raw_call("infini_attn_residual_norm_backward", ctypes.byref(ResidualNormArgs(**a)),
                       ctypes.byref(g), None, None) == SHAPE


def test_import_without_torchs_cuda_build(ia):
    """A torch built without CUDA lacks torch._C's CUDA functions: the package still imports
    (its host checks, sizes and error texts need no GPU)."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, n)\n"
            "import compressive_memory_transformer_b200 as ia\n"
            "assert ia.linear_backward_workspace_size(64, 64, 64) >= 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
