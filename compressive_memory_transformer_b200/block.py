"""Binding of the operators around the attention layer: the linear layer with bias,
activation and residual, the norms with a block's gate and the scaled residual stream,
their gradients, and the whole transformer block. Argument marshalling only, like the
rest of the package; the names are those of include/infini_attn.h.

Every call runs on the device of its tensors: on `stream`, or on that device's current
stream. Outputs and scratch that a call makes come from torch's allocator on the same
stream. Inputs made on another stream have to be ready (an event, a wait) by then, and every
tensor of a call has to stay until the call's work on its stream is done.
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


def _on(dev, stream, call):
    """call(stream handle) with the device and the stream current, so that what it allocates
    belongs to the stream that it runs on. (The usual case, no stream given and the
    tensors' device already current, takes no context manager: they cost more than a small
    call's kernels. torch._C's functions are looked up here: a torch built without CUDA has
    none, and still imports this package.)"""
    if stream is None:
        if dev == torch._C._cuda_getDevice():
            return call(torch._C._cuda_getCurrentRawStream(dev))
        with torch.cuda.device(dev):
            return call(torch._C._cuda_getCurrentRawStream(dev))
    if stream.device_index != dev:
        raise ValueError("the stream is on another device than the tensors")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _p(t):
    return None if t is None else t.data_ptr()


def _matrix(name, t, dev, cols=None):
    """(rows, columns, row stride) of a bf16 matrix on device `dev`: 2-d with neighbouring
    columns, or any contiguous tensor seen as [rows, last dimension]."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a bf16 tensor on the CUDA device of x")
    shape = t.shape
    if len(shape) == 2 and (shape[1] <= 1 or t.stride(1) == 1):
        r, c = shape
        # one row has no stride to keep to; repeated rows (stride 0) are no matrix in memory
        ld = t.stride(0) if r > 1 else c
        if ld < c:
            raise ValueError(f"{name} must not have overlapping rows")
    elif len(shape) >= 1 and t.is_contiguous():
        c = shape[-1]
        r, ld = (t.numel() // c if c else 0), c
    else:
        raise ValueError(f"{name} must be contiguous, or 2-d with contiguous rows")
    if cols is not None and c != cols:
        raise ValueError(f"{name} must have {cols} columns")
    return r, c, ld


def _weight(W, dev, K):
    if W.dim() != 2 or W.shape[0] != K:
        raise ValueError("W must be [K, N] with K the last dimension of x")
    return _matrix("W", W, dev)


def _vector(name, t, n, dev):
    if t is not None and (t.dtype is not torch.float32 or t.numel() != n
                          or t.get_device() != dev or not t.is_contiguous()):
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
        return like.new_empty((size,), dtype=torch.uint8) if size else None
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of x")
    return workspace


def infini_attn_linear(x, W, bias=None, act=ACT_NONE, residual=None, save_preact=False, out=None,
                       stream=None):
    """y = act(x W + bias) + residual: x [..., K], W [K, N], residual [..., N] bf16, bias [N]
    fp32; K and N multiples of 8. Returns y [..., N], and with save_preact (y, x W + bias),
    the second for the gradient of the activation. x, W, residual and out may be slices of
    wider 2-d tensors (row strides a multiple of 8), out a slice of the same one as x or residual
    if it shares no column with them; out may be residual itself."""
    dev = x.get_device()
    M, K, ldx = _matrix("x", x, dev)
    _, N, ldw = _weight(W, dev, K)
    shape = x.shape[:-1] + (N,)
    a = LinearArgs(x=x.data_ptr(), W=W.data_ptr(), ldx=ldx, ldw=ldw, M=M, K=K, N=N, act=act)
    if bias is not None:
        _vector("bias", bias, N, dev)
        a.bias = bias.data_ptr()
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual must be {shape}")
        a.residual, a.ldr = residual.data_ptr(), _matrix("residual", residual, dev)[2]
    if out is not None:
        if out.shape != shape:
            raise ValueError(f"out must be {shape}")
        a.ldy = _matrix("out", out, dev)[2]

    def call(s):
        y = x.new_empty(shape) if out is None else out
        a.y = y.data_ptr()
        preact = None
        if save_preact:
            preact = x.new_empty(shape)
            a.preact = preact.data_ptr()
        _check(_lib.infini_attn_linear(ctypes.byref(a), s))
        return (y, preact) if save_preact else y

    return _on(dev, stream, call)


def infini_attn_linear_backward(x, W, dy, act=ACT_NONE, preact=None, x_grad=True, W_grad=True,
                                bias_grad=True, workspace=None, stage_events=None, stream=None):
    """Gradient of infini_attn_linear: (dx, dW, dbias) for dy [..., N] and, unless act is
    ACT_NONE, the forward's preact. dx and dW are bf16 like x and W, dbias [N] fp32; what is
    not asked for is None. The residual's gradient is dy. workspace: optional uint8 CUDA tensor of
    at least linear_backward_workspace_size(...) bytes."""
    dev = x.get_device()
    M, K, ldx = _matrix("x", x, dev)
    _, N, ldw = _weight(W, dev, K)
    shape = x.shape[:-1] + (N,)
    if dy.shape != shape:
        raise ValueError(f"dy must be {shape}")
    a = LinearGradArgs(x=x.data_ptr(), W=W.data_ptr(), dy=dy.data_ptr(), ldx=ldx, ldw=ldw,
                       lddy=_matrix("dy", dy, dev)[2], M=M, K=K, N=N, act=act)
    if act != ACT_NONE:
        if preact is None or preact.shape != shape:
            raise ValueError(f"preact must be {shape}")
        a.preact, a.ldp = preact.data_ptr(), _matrix("preact", preact, dev)[2]
    if not (x_grad or W_grad or bias_grad):
        return None, None, None

    def call(s):
        dx = dW = dbias = None
        if x_grad:
            dx = x.new_empty(x.shape)  # x may be a slice
            a.dx = dx.data_ptr()
        if W_grad:
            dW = W.new_empty((K, N))
            a.dW = dW.data_ptr()
        if bias_grad:
            dbias = x.new_empty((N,), dtype=torch.float32)
            a.dbias = dbias.data_ptr()
        ws = _scratch(workspace, linear_backward_workspace_size(M, K, N, act), x)
        _check(_lib.infini_attn_linear_backward(ctypes.byref(a),
                                                ctypes.byref(_options(ws, stage_events)), s))
        return dx, dW, dbias

    return _on(dev, stream, call)


def linear_backward_workspace_size(M, K, N, act=ACT_NONE) -> int:
    return int(_lib.infini_attn_linear_backward_workspace_size(M, K, N, int(act)))


def _rows(name, t, x):
    if t is not None and (t.shape != x.shape or t.dtype is not x.dtype
                          or t.get_device() != x.get_device() or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor shaped and typed like x")


def _norm_args(x, b, gate, alpha, post_weight, post_bias, pre_weight, pre_bias, kind, eps):
    dev, shape, dtype = x.get_device(), x.shape, x.dtype
    if dev < 0 or len(shape) < 1 or not x.is_contiguous() or (dtype is not torch.bfloat16
                                                              and dtype is not torch.float32):
        raise ValueError("x must be a contiguous bf16 or fp32 CUDA tensor [..., dim]")
    D = shape[-1]
    rows = x.numel() // D if D else 0
    a = ResidualNormArgs(x=x.data_ptr(), rows=rows, dim=D, kind=kind, alpha=alpha, eps=eps,
                         dtype=DTYPE_BF16 if dtype is torch.bfloat16 else DTYPE_F32)
    if b is not None:
        _rows("b", b, x)
        a.b = b.data_ptr()
    elif gate is not None or post_weight is not None:
        raise ValueError("a gate or a post norm needs b")
    if pre_weight is not None:
        _vector("pre_weight", pre_weight, D, dev)
        a.pre_weight = pre_weight.data_ptr()
    if post_weight is not None:
        _vector("post_weight", post_weight, D, dev)
        a.post_weight = post_weight.data_ptr()
    if pre_bias is not None or post_bias is not None:
        if (pre_bias is not None and pre_weight is None) or (post_bias is not None
                                                             and post_weight is None):
            raise ValueError("a norm's bias needs its weight")
        _vector("pre_bias", pre_bias, D, dev)
        _vector("post_bias", post_bias, D, dev)
        a.pre_bias, a.post_bias = _p(pre_bias), _p(post_bias)
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != D:
            raise ValueError("gate must be [dim] or [groups, dim]")
        groups = gate.shape[0] if gate.dim() == 2 else 1
        if rows % groups if groups else rows:  # no groups: a row per token of no tokens
            raise ValueError("gate's groups must divide the rows")
        _vector("gate", gate, groups * D, dev)
        a.gate, a.gate_groups = gate.data_ptr(), groups
    return a


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

    def call(s):
        r = torch.empty_like(x) if r_out is None else r_out
        a.r = r.data_ptr()
        h = None
        if pre_weight is not None:
            h = torch.empty_like(x) if h_out is None else h_out
            a.h = h.data_ptr()
        _check(_lib.infini_attn_residual_norm(ctypes.byref(a), s))
        return r, h

    return _on(x.get_device(), stream, call)


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

    def call(s):
        out = [None if t is None else torch.empty_like(t)
               for t in (x, b, gate, post_weight, post_bias, pre_weight, pre_bias)]
        g = ResidualNormGradArgs(_p(dr), _p(dh), *[None if t is None else t.data_ptr()
                                                   for t in out])
        ws = _scratch(workspace, residual_norm_backward_workspace_size(
            a.rows, a.dim, a.gate_groups, kind), x)
        _check(_lib.infini_attn_residual_norm_backward(ctypes.byref(a), ctypes.byref(g),
                                                       ctypes.byref(_options(ws)), s))
        return ResidualNormGrads(*out)

    return _on(x.get_device(), stream, call)


def residual_norm_backward_workspace_size(rows, dim, gate_groups=0, kind=NORM_RMS) -> int:
    return int(_lib.infini_attn_residual_norm_backward_workspace_size(rows, dim, gate_groups,
                                                                      int(kind)))


def infini_attn_norm(x, weight, bias=None, kind=NORM_RMS, eps=1e-5, out=None, stream=None):
    """h = norm(x; weight, bias) over the last dimension; x bf16 or fp32, weight and bias
    fp32. out may be x itself."""
    if weight is None:
        raise ValueError("weight must be given")
    a = _norm_args(x, None, None, 1.0, None, None, weight, bias, kind, eps)
    _rows("out", out, x)

    def call(s):
        h = torch.empty_like(x) if out is None else out
        _check(_lib.infini_attn_norm(a.x, a.pre_weight, a.pre_bias, h.data_ptr(), a.rows, a.dim,
                                     a.kind, a.dtype, eps, s))
        return h

    return _on(x.get_device(), stream, call)


def infini_attn_norm_backward(x, weight, dh, bias=None, kind=NORM_RMS, eps=1e-5, workspace=None,
                              stream=None):
    """Gradient of infini_attn_norm: (dx, dweight, dbias), dbias None without a bias."""
    if weight is None or dh is None:
        raise ValueError("weight and dh must be given")
    a = _norm_args(x, None, None, 1.0, None, None, weight, bias, kind, eps)
    _rows("dh", dh, x)

    def call(s):
        dx, dw = torch.empty_like(x), torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        ws = _scratch(workspace, residual_norm_backward_workspace_size(a.rows, a.dim, 0, kind), x)
        _check(_lib.infini_attn_norm_backward(a.x, a.pre_weight, dh.data_ptr(), dx.data_ptr(),
                                              dw.data_ptr(), _p(dbias), a.rows, a.dim, a.kind,
                                              a.dtype, eps, ctypes.byref(_options(ws)), s))
        return dx, dw, dbias

    return _on(x.get_device(), stream, call)


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
    H_kv, dev = H if H_kv is None else H_kv, x.get_device()
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
            if t.dim() not in (1, 2) or n == 0 or groups not in (0, n):
                raise ValueError("gates must be [D_model] or [groups, D_model], both alike")
            groups = n
            _vector(name, t, n * D, dev)
    vectors = dict(attn_norm=attn_norm, attn_norm_bias=attn_norm_bias,
                   attn_post_norm=attn_post_norm, attn_post_norm_bias=attn_post_norm_bias,
                   mlp_norm=mlp_norm, mlp_norm_bias=mlp_norm_bias, mlp_post_norm=mlp_post_norm,
                   mlp_post_norm_bias=mlp_post_norm_bias)
    for name, t in vectors.items():
        _vector(name, t, D, dev)
    _vector("b_up", b_up, D_ff, dev)
    _vector("b_down", b_down, D, dev)
    _vector("beta", beta, H, dev)
    _vector("M_in", M_in, B * H_kv * d * d, dev)
    _vector("z_in", z_in, B * H_kv * d, dev)
    _rows("out", out, x)

    def call(s):
        y = x.new_empty(x.shape) if out is None else out
        M_out = z_out = None
        if state_out:
            M_out = x.new_empty((B, H_kv, d, d), dtype=torch.float32)
            z_out = x.new_empty((B, H_kv, d), dtype=torch.float32)
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

    return _on(dev, stream, call)


def block_workspace_size(B, L, D_model, D_ff, H, H_kv, N, d=128, mode=LINEAR) -> int:
    return int(_lib.infini_attn_block_workspace_size(B, L, D_model, D_ff, H, H_kv, int(N), d,
                                                     int(mode)))
