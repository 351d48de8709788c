"""Binding of the operators around the attention layer: the linear layer with bias,
activation and residual, the norms with a block's gate and the scaled residual stream,
their gradients, and the whole transformer block. Argument marshalling only, like the
rest of the package; the names are those of include/infini_attn.h.

Every call runs on the device of its tensors: on `stream`, or on that device's current
stream. Outputs and scratch that a call makes come from torch's allocator on the same
stream. Inputs made on another stream have to be ready (an event, a wait) by then.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import DTYPE_BF16, DTYPE_F32, LINEAR, Opts, _check, _lib

ACT_NONE = 0
ACT_RELU = 1
ACT_SILU = 2
ACT_GELU = 3
ACT_GELU_TANH = 4
NORM_RMS = 0
NORM_LAYER = 1

_vp, _i, _ll, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class LinearArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "W", "bias", "residual", "y", "preact")]
                + [(n, _ll) for n in ("ldx", "ldw", "ldr", "ldy", "ldp", "M")]
                + [(n, _i) for n in ("K", "N", "act")])


class LinearGradArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "W", "preact", "dy", "dx", "dW", "dbias")]
                + [(n, _ll) for n in ("ldx", "ldw", "ldp", "lddy", "lddx", "lddw", "M")]
                + [(n, _i) for n in ("K", "N", "act")])


class ResidualNormArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "b", "gate", "post_weight", "post_bias", "pre_weight",
                                    "pre_bias", "r", "h")]
                + [(n, _ll) for n in ("rows", "gate_groups")]
                + [(n, _i) for n in ("dim", "kind", "dtype")]
                + [(n, _f) for n in ("alpha", "eps")])


class ResidualNormGradArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dr", "dh", "dx", "db", "dgate", "dpost_weight", "dpost_bias",
                                   "dpre_weight", "dpre_bias")]


class BlockArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in (
        "x", "Wq", "Wk", "Wv", "Wo", "beta", "M_in", "z_in", "M_out", "z_out", "attn_norm",
        "attn_norm_bias", "attn_post_norm", "attn_post_norm_bias", "attn_gate", "mlp_norm",
        "mlp_norm_bias", "mlp_post_norm", "mlp_post_norm_bias", "mlp_gate", "W_up", "b_up",
        "W_down", "b_down", "y")]
                + [(n, _ll) for n in ("L", "gate_groups")]
                + [(n, _i) for n in ("B", "D_model", "D_ff", "H", "H_kv", "N", "d", "mode", "act",
                                     "kind")]
                + [(n, _f) for n in ("alpha", "eps")])


_size_t = ctypes.c_size_t
_P, _O = ctypes.POINTER, ctypes.POINTER(Opts)
SIGS = {
    "infini_attn_linear": (_i, [_P(LinearArgs), _vp]),
    "infini_attn_linear_backward": (_i, [_P(LinearGradArgs), _O, _vp]),
    "infini_attn_linear_backward_workspace_size": (_size_t, [_ll, _i, _i, _i]),
    "infini_attn_residual_norm": (_i, [_P(ResidualNormArgs), _vp]),
    "infini_attn_residual_norm_backward": (_i, [_P(ResidualNormArgs), _P(ResidualNormGradArgs),
                                                _O, _vp]),
    "infini_attn_residual_norm_backward_workspace_size": (_size_t, [_ll, _i, _ll, _i]),
    "infini_attn_norm": (_i, [_vp] * 4 + [_ll, _i, _i, _i, _f, _vp]),
    "infini_attn_norm_backward": (_i, [_vp] * 6 + [_ll, _i, _i, _i, _f, _O, _vp]),
    "infini_attn_block_forward": (_i, [_P(BlockArgs), _O, _vp]),
    "infini_attn_block_workspace_size": (_size_t, [_i, _ll] + [_i] * 7),
}
for _name, (_res, _args) in SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class _On:
    """The device and stream of one call. Entered, they are current, so that what the call
    allocates belongs to the stream that it runs on."""

    def __init__(self, device, stream):
        self.device, self.stream, self.undo = device, stream, []

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.undo.append(torch.cuda.device(self.device))
            self.undo[-1].__enter__()
        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        if self.stream.device != self.device:
            self.__exit__()
            raise ValueError("the stream is on another device than the tensors")
        self.undo.append(torch.cuda.stream(self.stream))
        self.undo[-1].__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        while self.undo:
            self.undo.pop().__exit__(None, None, None)
        return False


def _p(t):
    return None if t is None else t.data_ptr()


def _matrix(name, t, like, cols=None):
    """(rows, columns, row stride) of a bf16 matrix: 2-d with neighbouring columns, or any
    contiguous tensor seen as [rows, last dimension]."""
    if t.dtype != torch.bfloat16 or t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name} must be a bf16 tensor on the CUDA device of x")
    if t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1):
        r, c = t.shape
        # one row has no stride to keep to; repeated rows (stride 0) are no matrix in memory
        ld = t.stride(0) if r > 1 else c
        if ld < c:
            raise ValueError(f"{name} must not have overlapping rows")
    elif t.dim() >= 1 and t.is_contiguous():
        c = t.shape[-1]
        r, ld = (t.numel() // c if c else 0), c
    else:
        raise ValueError(f"{name} must be contiguous, or 2-d with contiguous rows")
    if cols is not None and c != cols:
        raise ValueError(f"{name} must have {cols} columns")
    return r, c, ld


def _vector(name, t, n, like):
    if t is not None and (t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous()
                          or t.device != like.device):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of {n} elements on the device "
                         "of x")


def _options(workspace, stage_events=None):
    o = Opts()
    if workspace is not None:
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    for i, ev in enumerate(stage_events or ()):
        o.stage_events[i] = None if ev is None else ev.cuda_event
    return o


def _scratch(workspace, size, like):
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=like.device) if size else None
    if workspace.device != like.device:
        raise ValueError("workspace must be on the device of x")
    return workspace


def infini_attn_linear(x, W, bias=None, act=ACT_NONE, residual=None, save_preact=False, out=None,
                       stream=None):
    """y = act(x W + bias) + residual: x [..., K], W [K, N], residual [..., N] bf16, bias [N]
    fp32; K and N multiples of 8. Returns y [..., N], and with save_preact (y, x W + bias),
    the second for the gradient of the activation. x, W, residual and out may be slices of
    wider 2-d tensors (row strides a multiple of 8); out may be residual itself."""
    M, K, ldx = _matrix("x", x, x)
    _, N, ldw = _matrix("W", W, x)
    if W.dim() != 2 or W.shape[0] != K:
        raise ValueError("W must be [K, N] with K the last dimension of x")
    _vector("bias", bias, N, x)
    shape = (*x.shape[:-1], N)
    a = LinearArgs(x=x.data_ptr(), W=W.data_ptr(), bias=_p(bias), ldx=ldx, ldw=ldw, M=M, K=K, N=N,
                   act=int(act))
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual must be {shape}")
        a.residual, a.ldr = residual.data_ptr(), _matrix("residual", residual, x)[2]
    if out is not None and out.shape != shape:
        raise ValueError(f"out must be {shape}")
    with _On(x.device, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
        a.y, a.ldy = out.data_ptr(), _matrix("out", out, x)[2]
        preact = None
        if save_preact:
            preact = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
            a.preact = preact.data_ptr()
        _check(_lib.infini_attn_linear(ctypes.byref(a), s))
    return (out, preact) if save_preact else out


def infini_attn_linear_backward(x, W, dy, act=ACT_NONE, preact=None, x_grad=True, W_grad=True,
                                bias_grad=True, workspace=None, stage_events=None, stream=None):
    """Gradient of infini_attn_linear: (dx, dW, dbias) for dy [..., N] and, unless act is
    ACT_NONE, the forward's preact. dx and dW are bf16 like x and W, dbias [N] fp32; what is
    not asked for is None. The residual's gradient is dy. workspace: optional uint8 CUDA tensor of
    at least linear_backward_workspace_size(...) bytes."""
    M, K, ldx = _matrix("x", x, x)
    _, N, ldw = _matrix("W", W, x)
    if W.dim() != 2 or W.shape[0] != K:
        raise ValueError("W must be [K, N] with K the last dimension of x")
    shape = (*x.shape[:-1], N)
    if dy.shape != shape:
        raise ValueError(f"dy must be {shape}")
    a = LinearGradArgs(x=x.data_ptr(), W=W.data_ptr(), dy=dy.data_ptr(), ldx=ldx, ldw=ldw,
                       lddy=_matrix("dy", dy, x)[2], M=M, K=K, N=N, act=int(act))
    if int(act) != ACT_NONE:
        if preact is None or preact.shape != shape:
            raise ValueError(f"preact must be {shape}")
        a.preact, a.ldp = preact.data_ptr(), _matrix("preact", preact, x)[2]
    dx = dW = dbias = None
    with _On(x.device, stream) as s:
        if x_grad:
            dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            a.dx = dx.data_ptr()
        if W_grad:
            dW = torch.empty(W.shape, dtype=W.dtype, device=x.device)
            a.dW = dW.data_ptr()
        if bias_grad:
            dbias = torch.empty((N,), dtype=torch.float32, device=x.device)
            a.dbias = dbias.data_ptr()
        if dx is None and dW is None and dbias is None:
            return dx, dW, dbias
        ws = _scratch(workspace, linear_backward_workspace_size(M, K, N, act), x)
        _check(_lib.infini_attn_linear_backward(ctypes.byref(a),
                                                ctypes.byref(_options(ws, stage_events)), s))
    return dx, dW, dbias


def linear_backward_workspace_size(M, K, N, act=ACT_NONE) -> int:
    return int(_lib.infini_attn_linear_backward_workspace_size(M, K, N, int(act)))


def _rows(name, t, like):
    if t is not None and (t.shape != like.shape or t.dtype != like.dtype
                          or t.device != like.device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor shaped and typed like x")


def _norm_args(x, b, gate, alpha, post_weight, post_bias, pre_weight, pre_bias, kind, eps):
    if x.dim() < 1 or not x.is_cuda or not x.is_contiguous() or x.dtype not in (torch.bfloat16,
                                                                                torch.float32):
        raise ValueError("x must be a contiguous bf16 or fp32 CUDA tensor [..., dim]")
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    _rows("b", b, x)
    for name, t in (("post_weight", post_weight), ("post_bias", post_bias),
                    ("pre_weight", pre_weight), ("pre_bias", pre_bias)):
        if t is not None:
            _vector(name, t, D, x)
    if b is None and (gate is not None or post_weight is not None):
        raise ValueError("a gate or a post norm needs b")
    if (pre_bias is not None and pre_weight is None) or (post_bias is not None
                                                         and post_weight is None):
        raise ValueError("a norm's bias needs its weight")
    groups = 0
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != D or gate.shape[0] == 0:
            raise ValueError("gate must be [dim] or [groups, dim]")
        groups = gate.shape[0] if gate.dim() == 2 else 1
        if rows % groups:
            raise ValueError("gate's groups must divide the rows")
        _vector("gate", gate, groups * D, x)
    return ResidualNormArgs(
        x=x.data_ptr(), b=_p(b), gate=_p(gate), post_weight=_p(post_weight),
        post_bias=_p(post_bias), pre_weight=_p(pre_weight), pre_bias=_p(pre_bias), rows=rows,
        gate_groups=groups, dim=D, kind=int(kind),
        dtype=DTYPE_BF16 if x.dtype == torch.bfloat16 else DTYPE_F32, alpha=alpha, eps=eps)


def infini_attn_residual_norm(x, b=None, gate=None, alpha=1.0, post_weight=None, post_bias=None,
                              pre_weight=None, pre_bias=None, kind=NORM_RMS, eps=1e-5, r_out=None,
                              h_out=None, stream=None):
    """r = alpha x + gate norm(b; post_weight, post_bias) and h = norm(r; pre_weight,
    pre_bias), in one pass: x (the residual stream) and b (a block's output) [..., dim] bf16 or
    fp32, gate [dim] or [groups, dim], weights and biases [dim] fp32. A norm is there when its
    weight is; h is None without pre_weight. r_out and h_out may be x or b themselves."""
    a = _norm_args(x, b, gate, alpha, post_weight, post_bias, pre_weight, pre_bias, kind, eps)
    _rows("r_out", r_out, x)
    _rows("h_out", h_out, x)
    with _On(x.device, stream) as s:
        r = torch.empty_like(x) if r_out is None else r_out
        a.r = r.data_ptr()
        h = None
        if pre_weight is not None:
            h = torch.empty_like(x) if h_out is None else h_out
            a.h = h.data_ptr()
        _check(_lib.infini_attn_residual_norm(ctypes.byref(a), s))
    return r, h


ResidualNormGrads = namedtuple("ResidualNormGrads",
                               "dx db dgate dpost_weight dpost_bias dpre_weight dpre_bias")


def infini_attn_residual_norm_backward(x, b, dr, dh, gate=None, alpha=1.0, post_weight=None,
                                       post_bias=None, pre_weight=None, pre_bias=None,
                                       kind=NORM_RMS, eps=1e-5, workspace=None, stream=None):
    """Gradient of infini_attn_residual_norm from its inputs and the gradients dr and dh of
    its outputs (either may be None: zero): a ResidualNormGrads with a gradient for every
    input that was given, None for the others."""
    a = _norm_args(x, b, gate, alpha, post_weight, post_bias, pre_weight, pre_bias, kind, eps)
    if dr is None and dh is None:
        raise ValueError("dr or dh must be given")
    if dh is not None and pre_weight is None:
        raise ValueError("dh needs pre_weight")
    _rows("dr", dr, x)
    _rows("dh", dh, x)
    with _On(x.device, stream) as s:
        given = dict(dx=x, db=b, dgate=gate, dpost_weight=post_weight, dpost_bias=post_bias,
                     dpre_weight=pre_weight, dpre_bias=pre_bias)
        out = {n: None if t is None else torch.empty_like(t) for n, t in given.items()}
        g = ResidualNormGradArgs(dr=_p(dr), dh=_p(dh), **{n: _p(t) for n, t in out.items()})
        ws = _scratch(workspace, residual_norm_backward_workspace_size(
            a.rows, a.dim, a.gate_groups, kind), x)
        _check(_lib.infini_attn_residual_norm_backward(ctypes.byref(a), ctypes.byref(g),
                                                       ctypes.byref(_options(ws)), s))
    return ResidualNormGrads(**out)


def residual_norm_backward_workspace_size(rows, dim, gate_groups=0, kind=NORM_RMS) -> int:
    return int(_lib.infini_attn_residual_norm_backward_workspace_size(rows, dim, gate_groups,
                                                                      int(kind)))


def infini_attn_norm(x, weight, bias=None, kind=NORM_RMS, eps=1e-5, out=None, stream=None):
    """h = norm(x; weight, bias) over the last dimension; x bf16 or fp32, weight and bias
    fp32. out may be x itself."""
    a = _norm_args(x, None, None, 1.0, None, None, weight, bias, kind, eps)
    if weight is None:
        raise ValueError("weight must be given")
    _rows("out", out, x)
    with _On(x.device, stream) as s:
        h = torch.empty_like(x) if out is None else out
        _check(_lib.infini_attn_norm(a.x, a.pre_weight, a.pre_bias, h.data_ptr(), a.rows, a.dim,
                                     a.kind, a.dtype, eps, s))
    return h


def infini_attn_norm_backward(x, weight, dh, bias=None, kind=NORM_RMS, eps=1e-5, workspace=None,
                              stream=None):
    """Gradient of infini_attn_norm: (dx, dweight, dbias), dbias None without a bias."""
    a = _norm_args(x, None, None, 1.0, None, None, weight, bias, kind, eps)
    if weight is None or dh is None:
        raise ValueError("weight and dh must be given")
    _rows("dh", dh, x)
    with _On(x.device, stream) as s:
        dx, dw = torch.empty_like(x), torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        ws = _scratch(workspace, residual_norm_backward_workspace_size(a.rows, a.dim, 0, kind), x)
        _check(_lib.infini_attn_norm_backward(a.x, a.pre_weight, dh.data_ptr(), dx.data_ptr(),
                                              dw.data_ptr(), _p(dbias), a.rows, a.dim, a.kind,
                                              a.dtype, eps, ctypes.byref(_options(ws)), s))
    return dx, dw, dbias


def infini_attn_block_forward(x, Wq, Wk, Wv, Wo, beta, N, mode, H, W_up, W_down, attn_norm,
                              mlp_norm, H_kv=None, b_up=None, b_down=None, act=ACT_GELU_TANH,
                              kind=NORM_RMS, eps=1e-5, alpha=1.0, attn_gate=None, mlp_gate=None,
                              attn_post_norm=None, mlp_post_norm=None, attn_norm_bias=None,
                              mlp_norm_bias=None, attn_post_norm_bias=None,
                              mlp_post_norm_bias=None, M_in=None, z_in=None, out=None,
                              state_out=True, workspace=None, stage_events=None, stream=None):
    """One transformer block: x [B, L, D_model] bf16 -> norm -> infini_attn_layer_forward ->
    (post norm, gate) + alpha x -> norm -> act(. W_up + b_up) W_down + b_down -> (post norm,
    gate) + alpha (.). Gates are [D_model] or [groups, D_model] fp32, norms' weights and
    biases [D_model] fp32, b_up and b_down fp32. Returns (y, M_out, z_out) with the layer's
    state (None when state_out is False)."""
    H_kv = H if H_kv is None else H_kv
    if x.dim() != 3 or x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 CUDA tensor [B, L, D_model]")
    B, L, D = x.shape
    if Wq.dim() != 2 or W_up.dim() != 2 or H < 1:
        raise ValueError("weights must be 2-d")
    d, D_ff = Wq.shape[1] // H, W_up.shape[1]
    for name, t, shape in (("Wq", Wq, (D, H * d)), ("Wk", Wk, (D, H_kv * d)),
                           ("Wv", Wv, (D, H_kv * d)), ("Wo", Wo, (H * d, D)),
                           ("W_up", W_up, (D, D_ff)), ("W_down", W_down, (D_ff, D))):
        if t.shape != shape or t.dtype != torch.bfloat16 or t.device != x.device or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor {shape} on the device of x")
    groups = 0
    for name, t in (("attn_gate", attn_gate), ("mlp_gate", mlp_gate)):
        if t is not None:
            n = t.shape[0] if t.dim() == 2 else 1
            if t.dim() not in (1, 2) or groups not in (0, n):
                raise ValueError("gates must be [D_model] or [groups, D_model], both alike")
            groups = n
            _vector(name, t, n * D, x)
    vectors = dict(attn_norm=attn_norm, attn_norm_bias=attn_norm_bias,
                   attn_post_norm=attn_post_norm, attn_post_norm_bias=attn_post_norm_bias,
                   mlp_norm=mlp_norm, mlp_norm_bias=mlp_norm_bias, mlp_post_norm=mlp_post_norm,
                   mlp_post_norm_bias=mlp_post_norm_bias)
    for name, t in vectors.items():
        _vector(name, t, D, x)
    _vector("b_up", b_up, D_ff, x)
    _vector("b_down", b_down, D, x)
    _vector("beta", beta, H, x)
    _vector("M_in", M_in, B * H_kv * d * d, x)
    _vector("z_in", z_in, B * H_kv * d, x)
    _rows("out", out, x)
    with _On(x.device, stream) as s:
        y = torch.empty_like(x) if out is None else out
        M_out = z_out = None
        if state_out:
            M_out = torch.empty((B, H_kv, d, d), device=x.device, dtype=torch.float32)
            z_out = torch.empty((B, H_kv, d), device=x.device, dtype=torch.float32)
        a = BlockArgs(x=x.data_ptr(), Wq=Wq.data_ptr(), Wk=Wk.data_ptr(), Wv=Wv.data_ptr(),
                      Wo=Wo.data_ptr(), beta=beta.data_ptr(), M_in=_p(M_in), z_in=_p(z_in),
                      M_out=_p(M_out), z_out=_p(z_out), attn_gate=_p(attn_gate),
                      mlp_gate=_p(mlp_gate), W_up=W_up.data_ptr(), b_up=_p(b_up),
                      W_down=W_down.data_ptr(), b_down=_p(b_down), y=y.data_ptr(), L=L,
                      gate_groups=groups, B=B, D_model=D, D_ff=D_ff, H=H, H_kv=H_kv, N=int(N),
                      d=d, mode=int(mode), act=int(act), kind=int(kind), alpha=alpha, eps=eps,
                      **{n: _p(t) for n, t in vectors.items()})
        ws = _scratch(workspace, block_workspace_size(B, L, D, D_ff, H, H_kv, N, d, mode), x)
        _check(_lib.infini_attn_block_forward(ctypes.byref(a),
                                              ctypes.byref(_options(ws, stage_events)), s))
    return y, M_out, z_out


def block_workspace_size(B, L, D_model, D_ff, H, H_kv, N, d=128, mode=LINEAR) -> int:
    return int(_lib.infini_attn_block_workspace_size(B, L, D_model, D_ff, H, H_kv, int(N), d,
                                                     int(mode)))
