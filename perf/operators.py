"""The operators around an attention layer, as measurable cases: the matrix product
with bias, activation and residual in its epilogue (and its gradient), and the norms
before and after a block, fused with the block's gate and the residual scale (and
their gradient).

linear            y = act(x W + bias) + residual; a training forward also returns the
                  pre-activation x W + bias
linear_backward   from x, W, the pre-activation and dy: dx, dW, dbias
residual_norm     r = alpha x + gate * post(b), h = pre(r), with post and pre each a
                  root-mean-square or a layer norm (or absent): the norm after a block
                  whose output is b, its gate, the scaled residual stream and the norm
                  before the next block, in one pass
residual_norm_backward   its gradients: x, b, the gate, every norm's weight and bias

listed() and draw() give cases, prepare() the inputs, run() one pass: in plain torch
operations in 32 bits, or (own = True) by this package's kernels. exact() is the same
from the definitions in 64 bits, the gradients by differentiation.
"""
import math

import torch

own = False

NONE, RELU, SILU, GELU, GELU_TANH = "none", "relu", "silu", "gelu", "gelu_tanh"


def listed():
    return [
        # one new token through the up projection of an MLP of width 1024: latency
        _linear("linear one token", 1, 1024, 4096, GELU_TANH),
        # 33 streams decoding at once, the down projection back onto the residual stream
        _linear("linear 33 tokens, residual", 33, 4096, 1024, NONE, res=True),
        # a ragged batch of prompts, widths that are no multiple of a tile, no bias
        _linear("linear ragged 5003 rows", 5003, 1160, 2056, SILU, bias=False),
        # the training forward of the up projection, 4 sequences of 32768 tokens
        _linear("linear up 131072 rows", 131072, 1024, 4096, GELU_TANH, pre=True),
        # the down projection of 32768 tokens with the residual added in the epilogue
        _linear("linear down 32768 rows", 32768, 4096, 1024, NONE, res=True),
        # a small training batch with odd row count
        _linear_bwd("linear backward 641 rows", 641, 512, 1408, GELU),
        # the up projection's gradient for 16384 tokens
        _linear_bwd("linear backward 16384 rows", 16384, 1024, 4096, GELU_TANH),
        # one token's residual stream between two blocks: latency
        _norm("residual norm one token", 1, 1024, "rms", "bf16", groups=0, post=True),
        # the residual stream of 4 sequences of 32768 tokens, gated per sequence
        _norm("residual norm 131072 rows", 131072, 1024, "rms", "bf16", groups=4, post=True),
        # an odd width in 32 bits, layer norms, no norm after the block
        _norm("residual norm odd width f32", 4099, 777, "layer", "f32", groups=1, post=False),
        # the gradient of a small odd batch, layer norms with biases
        _norm_bwd("residual norm backward 515 rows", 515, 640, "layer", "f32", groups=5, post=True),
        # the gradient over 32768 tokens of a model of width 4096
        _norm_bwd("residual norm backward 32768 rows", 32768, 4096, "rms", "bf16", groups=1,
                  post=True),
    ]


def _linear(name, M, K, N, act, bias=True, res=False, pre=False):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "act": act, "bias": bias,
            "res": res, "pre": pre}


def _linear_bwd(name, M, K, N, act, bias=True):
    return {"name": name, "op": "linear_backward", "M": M, "K": K, "N": N, "act": act,
            "bias": bias}


def _norm(name, rows, dim, kind, dtype, groups, post, alpha=0.75):
    return {"name": name, "op": "residual_norm", "rows": rows, "dim": dim, "kind": kind,
            "dtype": dtype, "groups": groups, "post": post, "alpha": alpha}


def _norm_bwd(name, rows, dim, kind, dtype, groups, post, alpha=0.75):
    return dict(_norm(name, rows, dim, kind, dtype, groups, post, alpha),
                op="residual_norm_backward")


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "residual_norm",
                     "residual_norm_backward"])
    if op == "linear":
        # few rows (a decoding batch) as often as many (prompts, training)
        M = _log(rng, 1, 128) if rng.random() < 0.4 else _log(rng, 128, 32768)
        c = _linear("", M, 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512),
                    rng.choice([NONE, RELU, SILU, GELU, GELU_TANH]), rng.random() < 0.7,
                    rng.random() < 0.4, rng.random() < 0.3)
    elif op == "linear_backward":
        c = _linear_bwd("", _log(rng, 1, 8192), 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512),
                        rng.choice([NONE, RELU, SILU, GELU, GELU_TANH]), rng.random() < 0.7)
    else:
        dim = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            dim = dim // 8 * 8
        rows = _log(rng, 1, max(2, min(131072, (1 << 27) // dim)))
        groups = rng.choice([0, 1, 1, 2, 8])
        if groups > 1:
            rows = max(1, rows // groups) * groups
        make = _norm if op == "residual_norm" else _norm_bwd
        c = make("", rows, dim, rng.choice(["rms", "layer"]),
                 rng.choice(["bf16", "bf16", "f32"]), groups, rng.random() < 0.6,
                 rng.choice([1.0, 0.5]))
    del c["name"]
    return c


def work(case):
    if "linear" in case["op"]:
        M, K, N = case["M"], case["K"], case["N"]
        vec = 4 * N if case["bias"] else 0
        if case["op"] == "linear":
            outs = 1 + int(case["res"]) + int(case["pre"])
            return {"bytes": 2 * (M * K + K * N + outs * M * N) + vec, "flops": 2 * M * N * K}
        pre = 0 if case["act"] == NONE else 1
        return {"bytes": 2 * (2 * M * K + 2 * K * N + (1 + pre) * M * N) + vec,
                "flops": 4 * M * N * K}
    R, D = case["rows"], case["dim"]
    e = 2 if case["dtype"] == "bf16" else 4
    vecs = case["groups"] + (2 if case["kind"] == "layer" else 1) * (1 + int(case["post"]))
    if case["op"] == "residual_norm":  # x, b -> r, h
        return {"bytes": 4 * e * R * D + 4 * vecs * D, "flops": 12 * R * D}
    # x, b, dr, dh -> dx, db and the vectors' gradients
    return {"bytes": 6 * e * R * D + 8 * vecs * D, "flops": 30 * R * D}


EPS = 1e-5


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.bfloat16):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(shift).to(dtype)

    s = {"case": dict(case)}
    if "linear" in case["op"]:
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = normal(M, K)
        s["W"] = normal(K, N, scale=K ** -0.5)
        s["bias"] = normal(N, scale=0.3, dtype=torch.float32) if case["bias"] else None
        if case["op"] == "linear":
            s["res"] = normal(M, N) if case["res"] else None
        else:
            # what the forward kept, and a gradient of the size that a mean over the rows gives
            s["pre"] = None if case["act"] == NONE else normal(M, N)
            s["dy"] = normal(M, N, scale=1.0 / M)
        return s
    R, D, f32 = case["rows"], case["dim"], torch.float32
    t = torch.bfloat16 if case["dtype"] == "bf16" else f32
    # a residual stream with an offset and a block's output of another size
    s["x"] = normal(R, D, scale=2.0, shift=0.25, dtype=t)
    s["b"] = normal(R, D, scale=0.7, shift=-0.1, dtype=t)
    s["pre_w"] = normal(D, scale=0.1, shift=1.0, dtype=f32)
    s["post_w"] = normal(D, scale=0.1, shift=0.8, dtype=f32) if case["post"] else None
    layer = case["kind"] == "layer"
    s["pre_b"] = normal(D, scale=0.1, dtype=f32) if layer else None
    s["post_b"] = normal(D, scale=0.1, dtype=f32) if layer and case["post"] else None
    G = case["groups"]
    s["gate"] = normal(G, D, scale=0.3, shift=0.5, dtype=f32) if G else None
    if case["op"] == "residual_norm_backward":
        s["dr"] = normal(R, D, scale=0.5, dtype=t)
        s["dh"] = normal(R, D, dtype=t)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return _PLAIN[op](state)


# ---- the plain forms -----------------------------------------------------------------

def _act(v, act):
    if act == RELU:
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == SILU:
        return v / (1 + torch.exp(-v))
    if act == GELU:
        return 0.5 * v * (1 + torch.erf(v * 0.7071067811865476))
    if act == GELU_TANH:
        return 0.5 * v * (1 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    return v


def _act_grad(v, act):
    if act == RELU:
        return (v > 0).to(v.dtype)
    if act == SILU:
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if act == GELU:
        cdf = 0.5 * (1 + torch.erf(v * 0.7071067811865476))
        return cdf + v * 0.3989422804014327 * torch.exp(-0.5 * v * v)
    t = torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * v * v)


def _plain_linear(s):
    c = s["case"]
    pre = s["x"].float() @ s["W"].float()
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = _act(pre, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    if c["pre"]:
        return y.to(torch.bfloat16), pre.to(torch.bfloat16)
    return (y.to(torch.bfloat16),)


def _plain_linear_backward(s):
    c = s["case"]
    d = s["dy"].float()
    if s["pre"] is not None:
        d = d * _act_grad(s["pre"].float(), c["act"])
    dx = (d @ s["W"].float().t()).to(torch.bfloat16)
    dW = (s["x"].float().t() @ d).to(torch.bfloat16)
    return (dx, dW, d.sum(0)) if c["bias"] else (dx, dW)


def _normed(v, layer):
    """(v - mean) / sd and 1 / sd for a layer norm, v / rms and 1 / rms otherwise."""
    if layer:
        v = v - v.mean(1, keepdim=True)
    inv = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * inv, inv


def _scaled(vn, w, b):
    return vn * w if b is None else vn * w + b


def _gate_rows(gate, u):
    """gate * u, row r by the gate's row r / (rows / groups)."""
    return (u.view(gate.shape[0], -1, u.shape[1]) * gate[:, None, :]).view_as(u)


def _plain_residual_norm(s):
    layer, t = s["case"]["kind"] == "layer", s["x"].dtype
    u = s["b"].float()
    if s["post_w"] is not None:
        u = _scaled(_normed(u, layer)[0], s["post_w"], s["post_b"])
    if s["gate"] is not None:
        u = _gate_rows(s["gate"], u)
    r = s["case"]["alpha"] * s["x"].float() + u
    h = _scaled(_normed(r, layer)[0], s["pre_w"], s["pre_b"])
    return r.to(t), h.to(t)


def _norm_grad(d, vn, inv, layer):
    """The gradient of v from that of _normed(v)."""
    d = d - vn * (d * vn).mean(1, keepdim=True)
    if layer:
        d = d - d.mean(1, keepdim=True)
    return d * inv


def _plain_residual_norm_backward(s):
    layer, t, G = s["case"]["kind"] == "layer", s["x"].dtype, s["case"]["groups"]
    u = s["b"].float()
    if s["post_w"] is not None:
        bn, binv = _normed(u, layer)
        u = _scaled(bn, s["post_w"], s["post_b"])
    r = s["case"]["alpha"] * s["x"].float() + (u if s["gate"] is None else _gate_rows(s["gate"], u))
    rn, rinv = _normed(r, layer)
    dh = s["dh"].float()
    out = {"pre_w": (dh * rn).sum(0)}
    if layer:
        out["pre_b"] = dh.sum(0)
    d = s["dr"].float() + _norm_grad(dh * s["pre_w"], rn, rinv, layer)
    out["x"] = (s["case"]["alpha"] * d).to(t)
    if s["gate"] is not None:
        out["gate"] = (d * u).view(G, -1, d.shape[1]).sum(1)
        d = _gate_rows(s["gate"], d)
    if s["post_w"] is not None:
        out["post_w"] = (d * bn).sum(0)
        if layer:
            out["post_b"] = d.sum(0)
        d = _norm_grad(d * s["post_w"], bn, binv, layer)
    out["b"] = d.to(t)
    return out


_PLAIN = {"linear": _plain_linear, "linear_backward": _plain_linear_backward,
          "residual_norm": _plain_residual_norm,
          "residual_norm_backward": _plain_residual_norm_backward}


# ---- by the package's kernels ---------------------------------------------------------

def _own(op, s):
    import compressive_memory_transformer_b200 as ia
    c = s["case"]
    if "linear" in op:
        act = {NONE: ia.ACT_NONE, RELU: ia.ACT_RELU, SILU: ia.ACT_SILU, GELU: ia.ACT_GELU,
               GELU_TANH: ia.ACT_GELU_TANH}[c["act"]]
        if op == "linear":
            y = ia.infini_attn_linear(s["x"], s["W"], bias=s["bias"], act=act, residual=s["res"],
                                      save_preact=c["pre"])
            return y if c["pre"] else (y,)
        dx, dW, dbias = ia.infini_attn_linear_backward(s["x"], s["W"], s["dy"], act=act,
                                                       preact=s["pre"], bias_grad=c["bias"])
        return (dx, dW, dbias) if c["bias"] else (dx, dW)
    kind = ia.NORM_LAYER if c["kind"] == "layer" else ia.NORM_RMS
    given = dict(gate=s["gate"], alpha=c["alpha"], post_weight=s["post_w"], post_bias=s["post_b"],
                 pre_weight=s["pre_w"], pre_bias=s["pre_b"], kind=kind, eps=EPS)
    if op == "residual_norm":
        return ia.infini_attn_residual_norm(s["x"], s["b"], **given)
    g = ia.infini_attn_residual_norm_backward(s["x"], s["b"], s["dr"], s["dh"], **given)
    out = {"x": g.dx, "b": g.db, "pre_w": g.dpre_weight}
    if s["pre_b"] is not None:
        out["pre_b"] = g.dpre_bias
    if s["gate"] is not None:
        out["gate"] = g.dgate
    if s["post_w"] is not None:
        out["post_w"] = g.dpost_weight
    if s["post_b"] is not None:
        out["post_b"] = g.dpost_bias
    return out


# ---- from the definitions, in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor)}
    grads = case["op"].endswith("_backward")
    if "linear" in case["op"]:
        if not grads:
            z = torch.addmm(v["bias"], v["x"], v["W"]) if "bias" in v else torch.mm(v["x"], v["W"])
            y = _exact_act(z, case["act"])
            if "res" in v:
                y = y + v["res"]
            return (y, z) if case["pre"] else (y,)
        d = v["dy"]
        if "pre" in v:
            z = v["pre"].requires_grad_()
            d, = torch.autograd.grad(_exact_act(z, case["act"]), z, v["dy"])
        dx, dW = torch.mm(d, v["W"].T), torch.mm(v["x"].T, d)
        return (dx, dW, torch.ones(d.shape[0], dtype=d.dtype, device=d.device) @ d) \
            if case["bias"] else (dx, dW)
    names = [n for n in ("x", "b", "pre_w", "pre_b", "gate", "post_w", "post_b") if n in v]
    with torch.set_grad_enabled(grads):
        if grads:
            for n in names:
                v[n].requires_grad_()
        u = _exact_norm(v["b"], case["kind"], v["post_w"], v.get("post_b")) if case["post"] else v["b"]
        if "gate" in v:
            u = u * v["gate"].repeat_interleave(case["rows"] // case["groups"], 0)
        r = v["x"] * case["alpha"] + u
        h = _exact_norm(r, case["kind"], v["pre_w"], v.get("pre_b"))
        if not grads:
            return r, h
        got = torch.autograd.grad([r, h], [v[n] for n in names], [v["dr"], v["dh"]])
    return dict(zip(names, got))


def _exact_act(z, act):
    if act == RELU:
        return z.clamp(min=0)
    if act == SILU:
        return z * torch.sigmoid(z)
    if act == GELU:
        return z * torch.erfc(-z / math.sqrt(2)) / 2
    if act == GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _exact_norm(v, kind, w, b):
    if kind == "layer":
        var, mean = torch.var_mean(v, 1, keepdim=True, correction=0)
        v, ms = v - mean, var
    else:
        ms = v.pow(2).sum(1, keepdim=True) / v.shape[1]
    y = v / (ms + EPS).sqrt() * w
    return y if b is None else y + b
