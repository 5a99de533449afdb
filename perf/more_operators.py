"""Measured cases of the operators that work on the rows of items packed one
after the other: group norm with an activation, rotary positions, and
attention among the rows of an item, each forward and backward.

``run`` computes a case in plain torch operations in 32 bits (the rows of the
items padded to the longest), or, where ``own`` is true, through the package's
entry points. ``exact`` is the definition in 64 bits, item by item. Rows are
voxel sites (209,715 sites: a 128^3 grid at 10 % occupancy, the package's
benchmark) or tokens.
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-5


def _gn(name, way, rows, cin, groups, items, dtype, act, ragged=False, pad=0):
    return {"name": name, "op": "group_norm", "way": way, "rows": rows, "cin": cin, "groups": groups, "items": items,
            "dtype": dtype, "act": act, "ragged": ragged, "pad": pad}


def _rotary(name, way, rows, heads, dim, axes, part, reach, dtype, interleaved=False, scaling="none", factor=1.0,
            pad=0):
    """``part`` columns of each head are rotated, ``reach`` bounds the positions, rows are ``pad`` heads wider."""
    return {"name": name, "op": "rotary", "way": way, "rows": rows, "heads": heads, "dim": dim, "axes": axes,
            "part": part, "reach": reach, "dtype": dtype, "interleaved": interleaved, "scaling": scaling,
            "factor": factor, "pad": pad}


def _attn(name, way, rows, items, heads, kv_heads, dim, dtype, causal, keys=0, ragged=False):
    """``keys`` 0: the queries' own rows are the keys."""
    return {"name": name, "op": "attention", "way": way, "rows": rows, "items": items, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "causal": causal, "keys": keys, "ragged": ragged}


def listed():
    return [
        # a norm on the few rows of a coarse level, two items: latency alone
        _gn("gn_forward_64x256", "forward", 64, 256, 32, 2, "fp16", "silu"),
        # the norm in front of a convolution on the benchmark's sites, inference
        _gn("gn_forward_209715x128", "forward", 209715, 128, 32, 1, "fp16", "silu"),
        # its gradients in training, four items of a batch
        _gn("gn_backward_209715x128", "backward", 209715, 128, 32, 4, "bf16", "silu", ragged=True),
        # groups of five channels in 32 bits, ragged items (an empty one among them), rows that are a slice of wider ones
        _gn("gn_backward_20011x60", "backward", 20011, 60, 12, 7, "fp32", "gelu", ragged=True, pad=3),
        # the new tokens of eight sequences, far positions of a scaled long context: latency alone
        _rotary("rotary_forward_8x20x128", "forward", 8, 20, 128, 1, 128, 131072, "bf16", scaling="parts", factor=8.0,
                pad=4),
        # queries and keys of the benchmark's sites by their three coordinates
        _rotary("rotary_forward_209715x8x64", "forward", 209715, 8, 64, 3, 60, 512, "fp16", interleaved=True, pad=4),
        # gradients where a part of an odd number of heads is rotated, in 32 bits
        _rotary("rotary_backward_20011x5x80", "backward", 20011, 5, 80, 1, 48, 1048576, "fp32", scaling="linear",
                factor=4.0),
        # one new token for each of eight sequences over their caches: serving
        _attn("attn_forward_8_on_32768", "forward", 8, 8, 16, 4, 64, "bf16", True, keys=32768, ragged=True),
        # prompts of different lengths packed together, grouped heads
        _attn("attn_forward_8192_causal", "forward", 8192, 4, 16, 4, 128, "bf16", True, ragged=True),
        # full attention among the sites of two items, an odd number of rows
        _attn("attn_forward_20011", "forward", 20011, 2, 12, 12, 64, "fp16", False),
        # gradients of a cross attention: many sites on a few rows of conditioning, a width between the powers of two
        _attn("attn_backward_12347_on_308", "backward", 12347, 4, 10, 10, 72, "fp16", False, keys=308),
        # the largest: gradients of the prompts in training
        _attn("attn_backward_16384_causal", "backward", 16384, 4, 16, 4, 128, "bf16", True, ragged=True),
    ]


def _lengths(total, items, ragged, salt=0):
    """Rows of each item: near equal, or ragged by up to a factor of five with,
    from five items on, an empty one and one of a single row."""
    if not ragged:
        return [(total * (i + 1)) // items - (total * i) // items for i in range(items)]
    rng = random.Random(total * 1000 + items * 10 + salt)
    w = [rng.uniform(0.2, 1.0) for _ in range(items)]
    cut = [0]
    for i in range(items):
        cut.append(total if i == items - 1 else round(total * sum(w[:i + 1]) / sum(w)))
    n = [b - a for a, b in zip(cut, cut[1:])]
    if items >= 5:
        n[0], n[1] = n[0] + n[1], 0
        n[2], n[3] = (1, n[3] + n[2] - 1) if n[2] else (0, n[3])
    return n


def _both_lengths(case):
    """Rows and keys of each item of an attention case."""
    if case["keys"] == 0:
        n = _lengths(case["rows"], case["items"], case["ragged"])
        return n, n
    one_each = case["rows"] == case["items"]
    return (_lengths(case["rows"], case["items"], case["ragged"] and not one_each),
            _lengths(case["keys"], case["items"], case["ragged"], 1))


def _pairs(case):
    """Query-key pairs that attend, over the items."""
    total = 0
    for lq, lk in zip(*_both_lengths(case)):
        if not case["causal"]:
            total += lq * lk
        elif lk >= lq:
            total += lq * (lk - lq) + lq * (lq + 1) // 2
        else:
            total += lk * (lk + 1) // 2
    return total


def _spread(rng, low, high):
    """A whole number of [low, high], uniform in its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _padded_scores(case):
    lq, lk = _both_lengths(case)
    return case["items"] * case["heads"] * max(lq) * max(lk)


def draw(rng: random.Random):
    op = rng.choice(["group_norm", "rotary", "attention"])
    way = rng.choice(["forward", "backward"])
    if op == "group_norm":
        rows = _spread(rng, 1, 209715)
        groups = rng.choice([1, 4, 8, 16, 32, 32, 12])
        most = 2048 if rows < 13000 else 128
        per = _spread(rng, 1, most // groups) if rng.random() < 0.4 else 2 ** rng.randint(0, int(math.log2(most // groups)))
        items = min(rows, rng.choice([1, 1, 2, 4, 7, 16]))
        case = _gn("", way, rows, groups * per, groups, items, rng.choice(["fp16", "bf16", "fp32"]),
                   rng.choice(["none", "silu", "silu", "gelu", "relu"]), rng.random() < 0.6, rng.choice([0, 0, 8, 3]))
    elif op == "rotary":
        axes = rng.choice([1, 1, 3])
        dim = rng.choice([32, 64, 80, 96, 128])
        part = dim if rng.random() < 0.5 else 2 * rng.randint(4, dim // 2)
        part -= part % (2 * axes)
        scaling = rng.choice(["none", "linear", "base", "parts"]) if axes == 1 else "none"
        reach = _spread(rng, 64, 1 << 20) if axes == 1 else _spread(rng, 16, 1024)
        heads = rng.randint(1, 24)
        rows = _spread(rng, 1, max(1, 209715 * 8 * 64 // (heads * dim)))
        case = _rotary("", way, rows, heads, dim, axes, part, reach, rng.choice(["fp16", "bf16", "fp32"]),
                       rng.random() < 0.5, scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                       rng.choice([0, 0, 2, 5]))
    else:
        group, kv_heads = rng.choice([1, 1, 2, 4, 8]), rng.randint(1, 8)
        dim = rng.choice([32, 64, 64, 128, 128, 8 * rng.randint(2, 16)])
        dtype, causal, ragged = rng.choice(["fp16", "bf16"]), rng.random() < 0.5, rng.random() < 0.6
        items = rng.choice([1, 2, 3, 5, 8])
        kind = rng.choice(["self", "self", "cross", "tokens"])
        if kind == "tokens":
            way, rows, keys, causal = "forward", items, items * _spread(rng, 16, 8192), True
        elif kind == "cross":
            rows, keys, causal = max(items, _spread(rng, 16, 12347)), items * _spread(rng, 8, 512), False
        else:
            rows, keys = max(items, _spread(rng, 16, 16384)), 0
        case = _attn("", way, rows, items, group * kv_heads, kv_heads, dim, dtype, causal, keys, ragged)
        largest = listed()[-1]
        while work(case)["flops"] > work(largest)["flops"] or _padded_scores(case) > _padded_scores(largest):
            case["rows"] = max(items, case["rows"] * 2 // 3)
    del case["name"]
    return case


def work(case):
    n, back = case["rows"], case["way"] == "backward"
    s = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "group_norm":
        c, stats = case["cin"], 8 * case["items"] * case["groups"]
        if back:  # x, dy -> dx; mean, rstd; weight, bias -> their gradients
            return {"bytes": 3 * n * c * s + stats + 16 * c, "flops": 20 * n * c}
        return {"bytes": 2 * n * c * s + stats + 8 * c, "flops": 12 * n * c}
    if case["op"] == "rotary":
        return {"bytes": 2 * n * case["heads"] * case["dim"] * s + 4 * n * case["axes"],
                "flops": 3 * n * case["heads"] * case["part"]}
    h, d = case["heads"], case["dim"]
    keys = case["keys"] or n
    q, kv = n * h * d * s, keys * case["kv_heads"] * d * s
    if back:  # q, o, do, lse, k, v -> dq, dk, dv
        return {"bytes": 4 * q + 4 * kv + 4 * n * h, "flops": 10 * h * d * _pairs(case)}
    return {"bytes": 2 * q + 2 * kv + 4 * n * h, "flops": 4 * h * d * _pairs(case)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _offsets(lengths, dev):
    return torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)


def _frequencies(case):
    """Radians per position of the pairs of one axis, in 64 bits."""
    pairs = case["part"] // (2 * case["axes"])
    e = torch.arange(pairs, dtype=torch.float64) / pairs
    base, factor = 10000.0, case["factor"]
    if case["scaling"] == "base":
        base *= factor ** (pairs / max(1, pairs - 1))
    f = base ** -e
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":  # pairs of few turns over 4096 positions are stretched, those of many kept
        keep = ((4096 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f


def prepare(case, seed):
    """The inputs of a case: features with channel means and widths of their own
    before a norm, sites' coordinates or far positions, queries and keys with
    logits of a few units, gradients of unit size; queries, keys and values are
    columns of one projection."""
    dev = torch.device("cuda")
    dt = _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * scale + shift).to(dtype)

    n, back = case["rows"], case["way"] == "backward"
    s = {"case": case}
    if case["op"] == "group_norm":
        c, g = case["cin"], case["groups"]
        wide = c + case["pad"]
        lengths = _lengths(n, case["items"], case["ragged"])
        s["offsets"] = _offsets(lengths, dev) if case["items"] > 1 else None
        s["most"] = max(lengths)
        x = torch.randn((n, wide), generator=gen, device=dev) * (0.5 + torch.rand((wide,), generator=gen, device=dev))
        s["x"] = (x + normal(wide, shift=0.5, scale=0.5, dtype=torch.float32)).to(dt)[:, :c]
        s["weight"] = normal(c, scale=0.2, shift=1.0, dtype=torch.float32)
        s["bias"] = normal(c, scale=0.2, dtype=torch.float32)
        if back:
            s["grad"] = normal(n, wide)[:, :c]
            s["mean"], s["rstd"] = _group_stats(s, _pad(s["x"].float(), s["offsets"], s["most"]))
        return s
    if case["op"] == "rotary":
        h, d = case["heads"], case["dim"]
        s["x"] = normal(n, h + case["pad"], d)[:, :h]
        at = torch.randint(0, case["reach"], (n, case["axes"]), generator=gen, device=dev, dtype=torch.int32)
        s["positions"] = at[:, 0] if case["axes"] == 1 else at
        s["freqs"] = _frequencies(case).to(dev)
        return s
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    lq, lk = _both_lengths(case)
    s["offsets"], s["most_q"], s["most_k"] = _offsets(lq, dev), max(lq), max(lk)
    if case["keys"] == 0:
        s["k_offsets"] = None
        s["q"], s["k"], s["v"] = normal(n, h + 2 * hk, d, scale=1.2).split([h, hk, hk], 1)
    else:
        s["k_offsets"] = _offsets(lk, dev)
        s["q"] = normal(n, h, d, scale=1.2)
        s["k"], s["v"] = normal(case["keys"], 2 * hk, d, scale=1.2).split([hk, hk], 1)
    s["scale"] = d ** -0.5
    if back:
        s["out"], s["lse"] = _attention(s)
        s["grad"] = normal(n, h, d)
    return s


# ---------------------------------------------------------------------------
# the plain form, in 32 bits
# ---------------------------------------------------------------------------


def _pad(t, offsets, most):
    """The rows of each item, [items, most, ...], zeros behind its last."""
    if offsets is None:
        return t[None]
    at, real = _places(offsets, most)
    return t[at.clamp(max=max(0, t.shape[0] - 1))] * real.view(*real.shape, *([1] * (t.dim() - 1)))


def _places(offsets, most):
    """Row of each place of the padded items, and whether it is a real one."""
    at = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return at, at < offsets[1:, None]


def _pack(t, offsets, rows):
    """The rows of padded items, one after the other again."""
    if offsets is None:
        return t[0]
    at, real = _places(offsets, t.shape[1])
    out = t.new_zeros((rows + 1, *t.shape[2:]))
    out[torch.where(real, at, rows)] = t
    return out[:rows]


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -(0.5 ** 0.5))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -(0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _real(s, x):
    """1 for the places of real rows [items, most, 1, 1], and each item's number of values per group."""
    g, c = s["case"]["groups"], s["case"]["cin"]
    if s["offsets"] is None:
        return torch.ones((1, 1, 1, 1), device=x.device), torch.tensor([[float(x.shape[1] * (c // g))]], device=x.device)
    real = _places(s["offsets"], x.shape[1])[1][:, :, None, None].float()
    return real, (s["offsets"].diff().clamp(min=1) * (c // g)).float()[:, None]


def _group_stats(s, x):
    """Mean and 1 / deviation of each item's groups, of padded rows [items, most, C]."""
    g = s["case"]["groups"]
    x = x.unflatten(2, (g, -1))
    real, count = _real(s, x)
    mean = x.sum((1, 3)) / count
    var = ((x - mean[:, None, :, None]) * real).square().sum((1, 3)) / count
    return mean, torch.rsqrt(var + _EPS)


def _group_norm(s):
    case, dt = s["case"], s["x"].dtype
    n, g, back = case["rows"], case["groups"], case["way"] == "backward"
    x = _pad(s["x"].float(), s["offsets"], s["most"])
    mean, rstd = (s["mean"], s["rstd"]) if back else _group_stats(s, x)
    m, r = mean[:, None, :, None], rstd[:, None, :, None]
    w, b = s["weight"].view(g, -1), s["bias"].view(g, -1)
    xh = (x.unflatten(2, (g, -1)) - m) * r
    z = xh * w + b
    if not back:
        return _pack(_act(z, case["act"]).flatten(2), s["offsets"], n).to(dt), mean, rstd
    _, count = _real(s, x)
    dz = _pad(s["grad"].float(), s["offsets"], s["most"]).unflatten(2, (g, -1)) * _act_grad(z, case["act"])
    d = dz * w
    s1 = (d.sum((1, 3)) / count)[:, None, :, None]
    s2 = ((d * xh).sum((1, 3)) / count)[:, None, :, None]
    dx = r * (d - s1 - xh * s2)
    return _pack(dx.flatten(2), s["offsets"], n).to(dt), (dz * xh).sum((0, 1)).flatten(), dz.sum((0, 1)).flatten()


def _rotate(s):
    case, x = s["case"], s["x"]
    part, pairs = case["part"], case["part"] // 2
    at = s["positions"].view(case["rows"], case["axes"]).double()
    angle = (at[:, :, None] * s["freqs"]).flatten(1)  # 64 bits: far positions
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["way"] == "backward":
        sin = -sin
    t = x.float()
    if case["interleaved"]:
        a, b = t[..., 0:part:2], t[..., 1:part:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = t[..., :pairs], t[..., pairs:part]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, t[..., part:]], -1).to(x.dtype)


def _heads(s):
    """q, k, v as padded 32-bit [items, heads, most, dim], keys and values repeated for their group, and the mask."""
    k_off = s["offsets"] if s["k_offsets"] is None else s["k_offsets"]
    group = s["case"]["heads"] // s["case"]["kv_heads"]
    q = _pad(s["q"].float(), s["offsets"], s["most_q"]).transpose(1, 2)
    k = _pad(s["k"].float(), k_off, s["most_k"]).transpose(1, 2).repeat_interleave(group, 1)
    v = _pad(s["v"].float(), k_off, s["most_k"]).transpose(1, 2).repeat_interleave(group, 1)
    lq, lk = s["offsets"].diff()[:, None, None], k_off.diff()[:, None, None]
    i = torch.arange(s["most_q"], device=q.device)[None, :, None]
    j = torch.arange(s["most_k"], device=q.device)[None, None, :]
    seen = (j < lk) & (i < lq)
    if s["case"]["causal"]:
        seen = seen & (j <= i + lk - lq)
    return q, k, v, seen[:, None], k_off


def _attention(s):
    q, k, v, seen, _ = _heads(s)
    z = (q @ k.transpose(2, 3).contiguous()) * s["scale"]
    z = z.masked_fill_(~seen, -math.inf)
    top = z.amax(3, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(3, keepdim=True)
    out = (p @ v.contiguous()) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    n = s["case"]["rows"]
    return (_pack(out.transpose(1, 2), s["offsets"], n).to(s["q"].dtype), _pack(lse.transpose(1, 2), s["offsets"], n))


def _attention_backward(s):
    q, k, v, seen, k_off = _heads(s)
    case, dt = s["case"], s["q"].dtype
    do = _pad(s["grad"].float(), s["offsets"], s["most_q"]).transpose(1, 2).contiguous()
    p = (q @ k.transpose(2, 3).contiguous()) * s["scale"]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(3, keepdim=True)
    p = torch.exp(p - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    dp = do @ v.transpose(2, 3).contiguous()
    ds = p * (dp - (p * dp).sum(3, keepdim=True)) * s["scale"]
    del dp
    dq = ds @ k.contiguous()
    group = (case["kv_heads"], case["heads"] // case["kv_heads"])
    dk = (ds.transpose(2, 3).contiguous() @ q.contiguous()).unflatten(1, group).sum(2)
    dv = (p.transpose(2, 3).contiguous() @ do).unflatten(1, group).sum(2)
    keys = case["keys"] or case["rows"]
    return (_pack(dq.transpose(1, 2), s["offsets"], case["rows"]).to(dt),
            _pack(dk.transpose(1, 2), k_off, keys).to(dt), _pack(dv.transpose(1, 2), k_off, keys).to(dt))


def _plain(s):
    if s["case"]["op"] == "group_norm":
        return _group_norm(s)
    if s["case"]["op"] == "rotary":
        return _rotate(s)
    return _attention_backward(s) if s["case"]["way"] == "backward" else _attention(s)


# ---------------------------------------------------------------------------
# the package's entry points
# ---------------------------------------------------------------------------


def _own(s):
    import submanifold_sparse_convolution_hash_amd as sc

    case = s["case"]
    back = case["way"] == "backward"
    if case["op"] == "group_norm":
        if back:
            return sc.group_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["weight"], s["bias"],
                                          act=case["act"], offsets=s["offsets"])
        return sc.group_norm(s["x"], case["groups"], s["weight"], s["bias"], eps=_EPS, act=case["act"],
                             offsets=s["offsets"], return_stats=True)
    if case["op"] == "rotary":
        return sc.rotary(s["x"], s["positions"], s["freqs"], interleaved=case["interleaved"], inverse=back)
    if back:
        return sc.attention_backward(s["grad"], s["q"], s["k"], s["v"], s["out"], s["lse"], offsets=s["offsets"],
                                     k_offsets=s["k_offsets"], causal=case["causal"], scale=s["scale"])
    return sc.attention(s["q"], s["k"], s["v"], offsets=s["offsets"], k_offsets=s["k_offsets"], causal=case["causal"],
                        scale=s["scale"], return_lse=True)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------


def _slope(z, act):
    """An activation and its derivative, from the logistic function and the normal distribution's."""
    if act == "relu":
        on = torch.where(z > 0, 1.0, 0.0).double()
        return z * on, on
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * torch.sigmoid(-z)
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def _exact_group_norm(s):
    case = s["case"]
    n, c, g = case["rows"], case["cin"], case["groups"]
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    lengths = _lengths(n, case["items"], case["ragged"])
    back = case["way"] == "backward"
    rows, means, rstds, dw, db = [], [], [], torch.zeros_like(w), torch.zeros_like(b)
    start = 0
    for i, length in enumerate(lengths):
        t = x[start:start + length].reshape(length, g, c // g)
        if back:
            mean, std = s["mean"][i].double(), 1 / s["rstd"][i].double()
        elif length == 0:
            mean, std = x.new_zeros(g), x.new_full((g,), math.sqrt(_EPS))
        else:
            var, mean = torch.var_mean(t, (0, 2), correction=0)
            std = (var + _EPS).sqrt()
        xh = ((t - mean[:, None]) / std[:, None]).reshape(length, c)
        y, slope = _slope(torch.addcmul(b, xh, w), case["act"])
        if back:
            dz = s["grad"][start:start + length].double() * slope
            dw, db = dw + torch.einsum("nc,nc->c", dz, xh), db + dz.sum(0)
            d, k = (dz * w).view(length, g, c // g), xh.view(length, g, c // g)
            count = max(1, length * (c // g))
            first, second = torch.einsum("ngc->g", d) / count, torch.einsum("ngc,ngc->g", d, k) / count
            y = ((d - first[:, None] - k * second[:, None]) / std[:, None]).reshape(length, c)
        rows.append(y)
        means.append(mean)
        rstds.append(1 / std)
        start += length
    return (torch.cat(rows), dw, db) if back else (torch.cat(rows), torch.stack(means), torch.stack(rstds))


def _exact_rotary(s):
    case, x = s["case"], s["x"].double()
    turn = torch.einsum("na,f->naf", s["positions"].view(case["rows"], -1).double(), s["freqs"]).flatten(1)
    unit = torch.polar(torch.ones_like(turn), -turn if case["way"] == "backward" else turn)[:, None]
    part, half = case["part"], case["part"] // 2
    if case["interleaved"]:
        first, second = x[..., :part].unflatten(-1, (half, 2)).unbind(-1)
    else:
        first, second = x[..., :part].unflatten(-1, (2, half)).unbind(-2)
    turned = torch.view_as_real(torch.complex(first.contiguous(), second.contiguous()) * unit)
    return torch.cat([turned.flatten(-2) if case["interleaved"] else turned.transpose(-1, -2).flatten(-2), x[..., part:]], -1)


def _exact_attention(s):
    case = s["case"]
    back, group = case["way"] == "backward", case["heads"] // case["kv_heads"]
    q, k, v = (s[t].double().permute(1, 0, 2).contiguous() for t in "qkv")
    out, lse = torch.zeros_like(q), q.new_full(q.shape[:2], -math.inf)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    grad = s["grad"].double().permute(1, 0, 2).contiguous() if back else None
    at, kat = 0, 0
    for lq, lk in zip(*_both_lengths(case)):
        rows, cols = slice(at, at + lq), slice(kat, kat + lk)
        at, kat = at + lq, kat + lk
        if lq == 0 or lk == 0:
            continue
        hidden = torch.ones((lq, lk), dtype=torch.bool, device=q.device).triu(lk - lq + 1) if case["causal"] else None
        for h in range(case["heads"]):
            kh, vh = k[h // group, cols], v[h // group, cols]
            z = torch.mm(q[h, rows], kh.T) * s["scale"]
            if hidden is not None:
                z[hidden] = -math.inf
            lse[h, rows] = torch.logsumexp(z, 1)
            p = torch.nan_to_num(torch.softmax(z, 1))  # a row that sees nothing: zeros
            if not back:
                out[h, rows] = torch.mm(p, vh)
                continue
            dp = torch.mm(grad[h, rows], vh.T)
            ds = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None]) * s["scale"]
            dq[h, rows] = torch.mm(ds, kh)
            dk[h // group, cols] += torch.mm(ds.T, q[h, rows])
            dv[h // group, cols] += torch.mm(p.T, grad[h, rows])
    if back:
        return tuple(t.permute(1, 0, 2).contiguous() for t in (dq, dk, dv))
    return out.permute(1, 0, 2).contiguous(), lse.T.contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    return {"group_norm": _exact_group_norm, "rotary": _exact_rotary, "attention": _exact_attention}[case["op"]](s)
