"""64-bit references of the operators around the attention layer, on the CPU or the GPU in
float64, with bounds on how far a result in fewer bits may be off.

Every bound is a sum of: half a rounding step of the result (bf16 2^-8, fp32 2^-24,
relative); the rounding errors of fp32 sums, at most (terms) 2^-24 times the sum of the
terms' magnitudes (2^-23 where the tensor cores sum, which may truncate instead of
rounding); and, where an operand was rounded to bf16 on the way, 2^-8 times the sum of the
magnitudes it enters. SPECIAL covers the exponentials, error functions, divisions and
square roots in fp32, whose errors are a few units of 2^-23.
"""
import math

import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24
TENSOR = 2.0 ** -23
SPECIAL = 2.0 ** -20


def half_step(dtype):
    return BF16 if dtype == torch.bfloat16 else F32


def act(v, a):
    if a == 1:
        return torch.relu(v)
    if a == 2:
        return v * torch.sigmoid(v)
    if a == 3:
        return v * torch.erfc(-v / math.sqrt(2)) / 2
    if a == 4:
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v.clone()


def act_grad(v, a):
    if a == 0:
        return torch.ones_like(v)
    z = v.detach().clone().requires_grad_()
    return torch.autograd.grad(act(z, a).sum(), z)[0]


def linear(x, W, bias, a, res):
    """(y, pre) and their bounds before the final rounding."""
    x, W = x.double(), W.double()
    pre = x @ W
    mag = x.abs() @ W.abs()
    e = (x.shape[1] + 2) * TENSOR * mag
    if bias is not None:
        pre = pre + bias.double()
        e = e + 2 * F32 * (mag + bias.double().abs())
    y = act(pre, a)
    # no activation here has a slope above 1.13
    ey = 1.13 * e + (SPECIAL * (pre.abs() + y.abs()) if a else 0)
    if res is not None:
        y = y + res.double()
        ey = ey + 2 * F32 * (y.abs() + res.double().abs())
    return y, ey, pre, e


def linear_backward(x, W, pre, dy, a):
    """(dx, dW, dbias) and their bounds before the final rounding."""
    x, W, dy = x.double(), W.double(), dy.double()
    d = dy if a == 0 else dy * act_grad(pre.double(), a)
    # the derivative's own terms are at most 1.13 (1 + |v|) where they nearly cancel
    ed = torch.zeros_like(d) if a == 0 else SPECIAL * dy.abs() * (1 + pre.double().abs())
    rounded = ed if a == 0 else 1.01 * ed + BF16 * d.abs()
    M, N = d.shape
    dx, dW, db = d @ W.T, x.T @ d, d.sum(0)
    edx = rounded @ W.abs().T + (N + 2) * TENSOR * (1.01 * d.abs() @ W.abs().T)
    edW = x.abs().T @ rounded + (M + 2) * TENSOR * (x.abs().T @ (1.01 * d.abs()))
    edb = ed.sum(0) + (M + 2) * F32 * (d.abs() + ed).sum(0)
    return (dx, edx), (dW, edW), (db, edb)


def within(got, ref, err, step, what=""):
    """|got - ref| <= err + the result's rounding, everywhere."""
    assert got.shape == ref.shape, what
    bound = 1.01 * err + step * ref.abs() + 1e-38
    off = (got.double() - ref).abs()
    assert bool(torch.isfinite(got.double()).all()), f"{what}: not finite"
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


# Norms. Statistics of a row are sums over at most 8192 values in a tree whose longest path
# is 8 + 5 + 32 additions; with the divisions and the square root their relative error stays
# below 64 units. A result's bound is UNITS units of its terms' magnitudes, to which a layer
# norm's v - mean adds |v| + mean |v| in place of the difference itself.
UNITS = 128 * F32


def normed(v, kind, eps):
    """n(v), 1 / divisor, and the magnitude that n(v)'s rounding errors are relative to."""
    mean_abs = v.abs().mean(-1, keepdim=True)
    c = v - v.mean(-1, keepdim=True) if kind else v
    inv = 1 / (c.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n = c * inv
    mag = n.abs() + (v.abs() + mean_abs) * inv if kind else n.abs()
    return n, inv, mag


def residual_norm(x, b, gate, alpha, pw, pb, w, c, kind, eps):
    """(r, h) in float64 with bounds before the final rounding. All arguments float64."""
    r, er = alpha * x, UNITS * abs(alpha) * x.abs()
    if b is not None:
        u, eu = b, torch.zeros_like(b)
        if pw is not None:
            n, _, mag = normed(b, kind, eps)
            u, eu = n * pw, UNITS * mag * pw.abs()
            if pb is not None:
                u, eu = u + pb, eu + UNITS * pb.abs()
        if gate is not None:
            g = gate.reshape(-1, x.shape[1]).repeat_interleave(
                x.shape[0] // gate.reshape(-1, x.shape[1]).shape[0], 0)
            u, eu = u * g, eu * g.abs()
        r, er = r + u, er + eu + UNITS * u.abs()
    if w is None:
        return r, er, None, None
    n, inv, mag = normed(r, kind, eps)
    # r's own error reaches h directly, through the mean and through the divisor
    rms = er.pow(2).mean(-1, keepdim=True).sqrt()
    eh = w.abs() * (UNITS * mag + inv * (er + er.mean(-1, keepdim=True) + n.abs() * rms))
    h = n * w
    if c is not None:
        h, eh = h + c, eh + UNITS * c.abs()
    return r, er, h, eh


def residual_norm_grads(x, b, gate, alpha, pw, pb, w, c, kind, eps, dr, dh):
    """The gradients by differentiation in float64, in the order of the arguments; None for
    an argument that is None."""
    args = [None if t is None else t.detach().clone().requires_grad_()
            for t in (x, b, gate, pw, pb, w, c)]
    x, b, gate, pw, pb, w, c = args
    r, _, h, _ = residual_norm(x, b, gate, alpha, pw, pb, w, c, kind, eps)
    loss = 0
    if dr is not None:
        loss = loss + (r * dr).sum()
    if dh is not None:
        loss = loss + (h * dh).sum()
    given = [t for t in args if t is not None]
    got = iter(torch.autograd.grad(loss, given, allow_unused=True))
    return [None if t is None else next(got) for t in args]


def residual_norm_grad_sizes(x, b, gate, alpha, pw, pb, w, c, kind, eps, dr, dh):
    """Magnitudes of the terms of each gradient, which their rounding errors are relative
    to: the formulas with every term replaced by its absolute value."""
    m = lambda t: t.mean(-1, keepdim=True)
    rows = x.shape[0]
    u, bn_mag = None, None
    r_mag = abs(alpha) * x.abs()
    if b is not None:
        u, u_mag = b, b.abs()
        if pw is not None:
            bn, b_inv, bn_mag = normed(b, kind, eps)
            u, u_mag = bn * pw, bn_mag * pw.abs()
            if pb is not None:
                u, u_mag = u + pb, u_mag + pb.abs()
        if gate is not None:
            G = gate.reshape(-1, x.shape[1])
            g = G.repeat_interleave(rows // G.shape[0], 0)
        else:
            g = torch.ones_like(x)
        r_mag = r_mag + u_mag * g.abs()
        r = alpha * x + g * u
    else:
        r = alpha * x
    d = torch.zeros_like(x) if dr is None else dr.abs()
    dw = dc = None
    if w is not None and dh is not None:
        _, inv, _ = normed(r, kind, eps)
        rn = (r_mag + m(r_mag)) * inv  # what n(r)'s errors are relative to
        t = dh.abs() * w.abs()
        d = d + inv * (t + m(t) + rn * m(t * rn) * (2 + rn.pow(2).mean(-1, keepdim=True)))
        dw, dc = (dh.abs() * rn * (1 + m(rn))).sum(0), dh.abs().sum(0)
    elif w is not None:
        dw = dc = torch.zeros_like(w)
    dx = abs(alpha) * d
    if b is None:
        return dx, None, None, None, None, dw, dc
    dg = None
    if gate is not None:
        dg = (d * u_mag).reshape(G.shape[0], -1, x.shape[1]).sum(1).reshape(gate.shape)
        d = d * g.abs()
    if pw is None:
        return dx, d, dg, None, None, dw, dc
    dpw, dpb = (d * bn_mag).sum(0), d.sum(0)
    t = d * pw.abs()
    db = b_inv * (t + m(t) + bn_mag * m(t * bn_mag) * 2)
    return dx, db, dg, dpw, dpb, dw, dc
