"""Measured cases of the dense operators next to the sparse convolution:
layer norm, linear with a fused epilogue, and the gated feed-forward block,
each forward and backward.

``run`` computes a case in plain torch operations in 32 bits, or, where
``own`` is true, through the package's entry points. ``exact`` is the
definition in 64 bits. Rows are voxel sites (209,715 sites: a 128^3 grid at
10 % occupancy, the package's benchmark), channel widths those of its layers.
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-5


def _ln(name, way, rows, cin, dtype, pad=0):
    return {"name": name, "op": "layer_norm", "way": way, "rows": rows, "cin": cin, "dtype": dtype, "pad": pad}


def _linear(name, way, rows, cin, cout, dtype, act, residual=False, keep=False, pad=0):
    return {"name": name, "op": "linear", "way": way, "rows": rows, "cin": cin, "cout": cout, "dtype": dtype,
            "act": act, "residual": residual, "keep": keep, "pad": pad}


def _ffn(name, way, rows, cin, hidden, dtype, act, residual=False, keep=False, pad=0):
    return {"name": name, "op": "gated_ffn", "way": way, "rows": rows, "cin": cin, "cout": cin, "hidden": hidden,
            "dtype": dtype, "act": act, "residual": residual, "keep": keep, "pad": pad}


def listed():
    return [
        # one conditioning vector normalised: latency alone
        _ln("ln_forward_1x1024", "forward", 1, 1024, "fp16"),
        # the norm after a convolution on the benchmark's sites, inference
        _ln("ln_forward_209715x128", "forward", 209715, 128, "fp16"),
        # the same layer's gradients in training
        _ln("ln_backward_209715x128", "backward", 209715, 128, "bf16"),
        # an odd width in 32 bits, rows that are a slice of wider ones
        _ln("ln_backward_20011x515", "backward", 20011, 515, "fp32", pad=3),
        # the projection of one timestep or conditioning vector
        _linear("linear_forward_1_256_1024", "forward", 1, 256, 1024, "fp16", "silu"),
        # the first half of a point-wise block in training: pre-activations kept
        _linear("linear_forward_209715_128_512", "forward", 209715, 128, 512, "bf16", "gelu_tanh", keep=True),
        # a head onto an odd number of outputs, odd inputs, rows of a wider tensor
        _linear("linear_forward_12347_195_77", "forward", 12347, 195, 77, "fp16", "relu", residual=True, pad=5),
        # gradients of a point-wise layer in training
        _linear("linear_backward_100003_256_1024", "backward", 100003, 256, 1024, "bf16", "silu"),
        # the gated block on one vector
        _ffn("ffn_forward_1_512_2048", "forward", 1, 512, 2048, "fp16", "silu"),
        # the gated block of the benchmark's layer width on its sites, inference with the skip connection
        _ffn("ffn_forward_209715_128_512", "forward", 209715, 128, 512, "fp16", "silu", residual=True),
        # the largest: the gated block's gradients at 256 channels on the benchmark's sites
        _ffn("ffn_backward_209715_256_1024", "backward", 209715, 256, 1024, "bf16", "silu"),
        # a small set of sites with odd widths, training
        _ffn("ffn_backward_4099_100_267", "backward", 4099, 100, 267, "fp16", "gelu"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], uniform in its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A channel count: mostly a multiple of 8, sometimes any number."""
    w = _spread(rng, low, high)
    return w if rng.random() < 0.3 else max(8, 8 * (w // 8))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e15)


def draw(rng: random.Random):
    most = max(_cost(c) for c in listed())
    op = rng.choice(["layer_norm", "linear", "gated_ffn"])
    way = rng.choice(["forward", "backward"])
    pad = rng.choice([0, 0, 8, 3])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    residual = way == "forward" and rng.random() < 0.5
    keep = way == "forward" and rng.random() < 0.5
    rows = _spread(rng, 1, 209715)
    if op == "layer_norm":
        case = _ln("", way, rows, _width(rng, 8, 2048), rng.choice(["fp16", "bf16", "fp32"]), pad)
    elif op == "linear":
        case = _linear("", way, rows, _width(rng, 8, 1024), _width(rng, 8, 2048), rng.choice(["fp16", "bf16"]),
                       rng.choice([act, "none"]), residual, keep, pad)
    else:
        case = _ffn("", way, rows, _width(rng, 16, 512), _width(rng, 32, 2048), rng.choice(["fp16", "bf16"]),
                    act, residual, keep, pad)
    del case["name"]
    while _cost(case) > most:
        case["rows"] = max(1, case["rows"] // 2)
    return case


def work(case):
    n, c = case["rows"], case["cin"]
    s = 4 if case["dtype"] == "fp32" else 2
    back = case["way"] == "backward"
    if case["op"] == "layer_norm":
        if back:  # x, dy -> dx; mean, rstd; gamma -> dgamma, dbeta
            return {"bytes": 3 * n * c * s + 8 * n + 12 * c, "flops": 12 * n * c}
        return {"bytes": 2 * n * c * s + 8 * n + 8 * c, "flops": 8 * n * c}
    m = case["cout"]
    if case["op"] == "linear":
        if back:  # dy, z, x, W -> dx, dW, db
            z = 0 if case["act"] == "none" else n * m
            return {"bytes": s * (n * m + z + 2 * n * c + 2 * c * m) + 4 * m, "flops": 4 * n * c * m}
        extra = n * m * (int(case["residual"]) + int(case["keep"]))
        return {"bytes": s * (n * c + c * m + n * m + extra) + 4 * m, "flops": 2 * n * c * m}
    f = case["hidden"]
    if back:  # dy, [g|u], x, both weights -> dx and both weights' and biases' gradients; h counts neither way
        return {"bytes": s * (3 * n * c + 2 * n * f + 6 * c * f) + 4 * (2 * f + c), "flops": 12 * n * c * f}
    extra = n * c * int(case["residual"]) + 2 * n * f * int(case["keep"])
    return {"bytes": s * (2 * n * c + 3 * c * f + extra) + 4 * (2 * f + c), "flops": 6 * n * c * f}


def prepare(case, seed):
    """The inputs of a case: normalised features with channel means of their
    own before a norm, weights of variance 1 / fan-in, pre-activations near
    N(0, 1), gradients of unit size."""
    dev = torch.device("cuda")
    dt = _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * scale + shift).to(dtype)

    def rows(n, c):  # rows of a tensor `pad` columns wider
        return normal(n, c + case["pad"])[:, :c]

    n, c = case["rows"], case["cin"]
    back = case["way"] == "backward"
    s = {"case": case}
    if case["op"] == "layer_norm":
        x = torch.randn((n, c + case["pad"]), generator=gen, device=dev)
        x = x * (0.5 + torch.rand((c + case["pad"],), generator=gen, device=dev)) + 0.5
        s["x"] = x.to(dt)[:, :c]
        s["weight"] = normal(c, scale=0.2, shift=1.0, dtype=torch.float32)
        if back:
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + _EPS)
            s["grad"] = rows(n, c)
        else:
            s["bias"] = normal(c, scale=0.2, dtype=torch.float32)
        return s
    m = case["cout"]
    s["x"] = rows(n, c)
    if case["op"] == "linear":
        s["W"] = normal(c, m, scale=c ** -0.5)
        if back:
            s["grad"] = rows(n, m)
            s["pre"] = normal(n, m) if case["act"] != "none" else None
        else:
            s["bias"] = normal(m, scale=0.2, dtype=torch.float32)
            s["residual"] = rows(n, m) if case["residual"] else None
        return s
    f = case["hidden"]
    s["W_in"] = normal(c, 2 * f, scale=c ** -0.5)
    s["W_out"] = normal(f, m, scale=f ** -0.5)
    if back:
        s["grad"] = rows(n, m)
        s["pre"] = normal(n, 2 * f)
    else:
        s["b_in"] = normal(2 * f, scale=0.2, dtype=torch.float32)
        s["b_out"] = normal(m, scale=0.2, dtype=torch.float32)
        s["residual"] = rows(n, m) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# the plain form, in 32 bits
# ---------------------------------------------------------------------------

_K = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_K * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 * _K)
    if act == "gelu_tanh":
        t = torch.tanh(_K * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _K * (1 + 0.134145 * z * z)
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    dt, act = _TYPES[case["dtype"]], case.get("act")
    back = case["way"] == "backward"
    x = s["x"].float()
    if case["op"] == "layer_norm":
        if back:
            dy = s["grad"].float()
            xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
            d = dy * s["weight"]
            dx = s["rstd"][:, None] * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
            return dx.to(dt), (dy * xh).sum(0), dy.sum(0)
        m = x.mean(1)
        r = torch.rsqrt((x - m[:, None]).square().mean(1) + _EPS)
        return ((x - m[:, None]) * r[:, None] * s["weight"] + s["bias"]).to(dt), m, r
    if case["op"] == "linear":
        W = s["W"].float()
        if back:
            dz = s["grad"].float()
            if s["pre"] is not None:
                dz = dz * _act_grad(s["pre"].float(), act)
            return (dz @ W.t()).to(dt), (x.t() @ dz).to(dt), dz.sum(0)
        z = x @ W + s["bias"]
        out = _act(z, act)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return (out.to(dt), z.to(dt)) if case["keep"] else out.to(dt)
    W_in, W_out, f = s["W_in"].float(), s["W_out"].float(), case["hidden"]
    if back:
        dy, z = s["grad"].float(), s["pre"].float()
        g, u = z[:, :f], z[:, f:]
        a = _act(g, act)
        dh = dy @ W_out.t()
        dz = torch.cat([dh * u * _act_grad(g, act), dh * a], 1)
        return ((dz @ W_in.t()).to(dt), (x.t() @ dz).to(dt), dz.sum(0), ((a * u).t() @ dy).to(dt), dy.sum(0))
    z = x @ W_in + s["b_in"]
    out = (_act(z[:, :f], act) * z[:, f:]) @ W_out + s["b_out"]
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return (out.to(dt), z.to(dt)) if case["keep"] else out.to(dt)


def _own(s):
    import submanifold_sparse_convolution_hash_amd as sc

    case = s["case"]
    back = case["way"] == "backward"
    if case["op"] == "layer_norm":
        if back:
            return sc.layer_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["weight"])
        return sc.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS, return_stats=True)
    if case["op"] == "linear":
        if back:
            return sc.linear_backward(s["grad"], s["x"], s["W"], s["pre"], act=case["act"])
        return sc.linear(s["x"], s["W"], s["bias"], act=case["act"], residual=s["residual"], return_pre=case["keep"])
    if back:
        return sc.gated_ffn_backward(s["grad"], s["x"], s["W_in"], s["W_out"], s["pre"], act=case["act"])
    return sc.gated_ffn(s["x"], s["W_in"], s["b_in"], s["W_out"], s["b_out"], act=case["act"],
                        residual=s["residual"], return_pre=case["keep"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------


def _value_and_slope(z, act):
    """An activation and its derivative, from Phi(z) = erfc(-z / sqrt 2) / 2,
    the logistic function and tanh as 1 - 2 / (1 + e^2t)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = torch.where(z > 0, 1.0, 0.0).double()
        return z * on, on
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * torch.sigmoid(-z)
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)  # gelu_tanh: z sigmoid(2 t), 2 t = k (z + 0.044715 z^3)
    q = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * q, q + z * q * (1 - q) * k * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    back = case["way"] == "backward"
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    x = d["x"]
    if case["op"] == "layer_norm":
        c = case["cin"]
        if not back:
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            std = (var + _EPS).sqrt()
            return torch.addcmul(d["bias"], (x - mean) / std, d["weight"]), mean[:, 0], 1 / std[:, 0]
        r, dy = d["rstd"].unsqueeze(1), d["grad"]
        xh = (x - d["mean"].unsqueeze(1)) * r
        t = dy * d["weight"]
        dx = r * (c * t - t.sum(1, keepdim=True) - xh * (t * xh).sum(1, keepdim=True)) / c
        return dx, torch.einsum("nc,nc->c", dy, xh), dy.sum(0)
    if case["op"] == "linear":
        if back:
            dz = d["grad"]
            if "pre" in d:
                dz = dz * _value_and_slope(d["pre"], case["act"])[1]
            return torch.mm(dz, d["W"].T), torch.mm(x.T, dz), dz.sum(0)
        z = torch.addmm(d["bias"], x, d["W"])
        out = _value_and_slope(z, case["act"])[0]
        if "residual" in d:
            out = out + d["residual"]
        return (out, z) if case["keep"] else out
    if back:
        g, u = d["pre"].chunk(2, 1)
        a, slope = _value_and_slope(g, case["act"])
        dh = torch.mm(d["grad"], d["W_out"].T)
        dg, du = dh * u * slope, dh * a
        w_g, w_u = d["W_in"].chunk(2, 1)
        return (dg @ w_g.T + du @ w_u.T, torch.cat([x.T @ dg, x.T @ du], 1), torch.cat([dg.sum(0), du.sum(0)]),
                torch.mm((a * u).T, d["grad"]), d["grad"].sum(0))
    z = torch.addmm(d["b_in"], x, d["W_in"])
    g, u = z.chunk(2, 1)
    out = torch.addmm(d["b_out"], _value_and_slope(g, case["act"])[0] * u, d["W_out"])
    if "residual" in d:
        out = out + d["residual"]
    return (out, z) if case["keep"] else out
