"""Measured cases of the norms around the layer and of experts with 4-bit weights and group scales.

Four operators, each through its public call:

* ``norm``:    semmoe_norm -- the norm before the layer (root mean square or mean and variance);
* ``after``:   semmoe_combine_norm -- the layer's combine (or a dense block's rows), the norm after it, a gate, the scaled
               residual, and the norm before the next block;
* ``product``: semmoe_w4_grouped_gemm -- bf16 rows, sorted by expert, times their expert's matrix of 4-bit codes, each
               group of columns of a row with a scale (and a zero point);
* ``ffn``:     semmoe_w4_grouped_ffn -- the SwiGLU experts on such weights.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's norm before the router: latency alone
        dict(name="norm_T1_H2048", op="norm", T=1, H=2048, x="bf16", kind="rms", bias=False, offset=0.0, w="bf16"),
        # mean and variance, fp32, a row that ends inside a warp's last load
        dict(name="norm_T777_H1060_layer_f32", op="norm", T=777, H=1060, x="f32", kind="layer", bias=True, offset=0.0, w="f32"),
        # a prefill batch, weights held as their distance from 1
        dict(name="norm_T16384_H2048", op="norm", T=16384, H=2048, x="bf16", kind="rms", bias=False, offset=1.0, w="f32"),
        # the end of a layer in a decode batch: shared experts, a budget per request, norms after it and before the next
        dict(name="after_T64_H2048_shared", op="after", T=64, H=2048, k=6, x="bf16", shared=True, budgets=True, post="rms",
             next="rms", gate="", block_scale=1.0, res_scale=1.0, offset=0.0, w="bf16"),
        # a dense block before the layer: a gate per token and channel, no norm after, mean and variance before the next
        dict(name="after_dense_T4096_H2048", op="after", T=4096, H=2048, k=0, x="bf16", shared=False, budgets=False, post="",
             next="layer", gate="tokens", block_scale=1.0, res_scale=0.7, offset=0.0, w="f32"),
        # the end of a layer in the largest prefill batch: a gate per channel, both norms
        dict(name="after_T16384_H2048", op="after", T=16384, H=2048, k=8, x="bf16", shared=False, budgets=False, post="rms",
             next="rms", gate="channels", block_scale=0.5, res_scale=1.0, offset=0.0, w="bf16"),
        # one row times one matrix: the smallest product
        dict(name="product_1row_2048x2048", op="product", T=1, k=1, E=1, N=2048, K=2048, group=128, zeros=False, scale="bf16"),
        # a decode batch's second expert product, zero points
        dict(name="product_T64_E64_1408to2048", op="product", T=64, k=6, E=64, N=2048, K=1408, group=128, zeros=True,
             scale="bf16"),
        # hundreds of rows per expert, odd sizes, small groups, fp32 scales
        dict(name="product_T3001_E23_odd", op="product", T=3001, k=3, E=23, N=1000, K=1056, group=32, zeros=True, scale="f32"),
        # one decoded token through 8 of 128 experts
        dict(name="ffn_T1_E128", op="ffn", T=1, k=8, E=128, H=2048, I=768, group=128, zeros=False, scale="bf16"),
        # a decode batch that touches nearly every expert: bound by the weights' bytes
        dict(name="ffn_T64_E64", op="ffn", T=64, k=6, E=64, H=2048, I=1408, group=64, zeros=True, scale="bf16"),
        # the largest prefill: 131072 rows over 128 experts of 768
        dict(name="ffn_T16384_E128", op="ffn", T=16384, k=8, E=128, H=2048, I=768, group=128, zeros=False, scale="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "after", "product", "ffn", "ffn"])
    if op in ("norm", "after"):
        x = rng.choice(["bf16", "bf16", "f32"])
        H = (8 if x == "bf16" else 4) * _log(rng, 8, 512)
        T = _log(rng, 1, min(16384, (1 << 24) // H))
        w = rng.choice(["f32", x])
        if op == "norm":
            return dict(op=op, T=T, H=H, x=x, kind=rng.choice(["rms", "rms", "layer"]), bias=rng.random() < 0.4,
                        offset=rng.choice([0.0, 1.0]), w=w)
        return dict(op=op, T=T, H=H, k=rng.choice([0, 1, 2, 4, 6, 8]), x=x, shared=rng.random() < 0.4,
                    budgets=rng.random() < 0.3, post=rng.choice(["", "rms", "layer"]), next=rng.choice(["", "rms", "rms", "layer"]),
                    gate=rng.choice(["", "channels", "tokens"]), block_scale=rng.choice([1.0, 0.5]),
                    res_scale=rng.choice([1.0, 0.7]), offset=rng.choice([0.0, 1.0]), w=w)
    group = rng.choice([32, 64, 128])
    T, E = _log(rng, 1, 8192), _log(rng, 1, 128)
    k = rng.randint(1, min(8, E))
    base = dict(op=op, T=T, k=k, E=E, group=group, zeros=rng.random() < 0.5, scale=rng.choice(["bf16", "f32"]))
    if op == "product":
        return dict(base, N=8 * _log(rng, 8, 256), K=group * _log(rng, 1, 2048 // group))
    return dict(base, H=group * _log(rng, 1, 2048 // group), I=group * _log(rng, 1, 1408 // group))


def _pairs(c):
    """Live pairs of a case (their expected number with budgets)."""
    return c["T"] * (c["k"] + 1) / 2 if c["budgets"] and c["k"] else c["T"] * max(c["k"], 1)


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        return {"bytes": 2 * n * _size(c["x"]) + c["H"] * _size(c["w"]) * (2 if c["bias"] else 1), "flops": 5 * n}
    if c["op"] == "after":
        n, s = c["T"] * c["H"], _size(c["x"])
        rows = _pairs(c) * c["H"]  # the block's rows
        maps = 8 * c["T"] * c["k"]
        extra = n * s * (1 + (1 if c["shared"] else 0) + 1 + (1 if c["next"] else 0))  # residual, shared, out, next
        gate = {"": 0, "channels": c["H"] * _size(c["w"]), "tokens": n * s}[c["gate"]]
        weights = c["H"] * _size(c["w"]) * ((1 if c["post"] else 0) + (1 if c["next"] else 0))
        return {"bytes": rows * s + maps + extra + gate + weights, "flops": 2 * rows + 12 * n}
    P = c["T"] * c["k"]
    used = min(c["E"], P)  # experts that have rows, at most
    per = 0.5 + (_size(c["scale"]) + (1 if c["zeros"] else 0)) / c["group"]  # bytes of a weight
    if c["op"] == "product":
        return {"bytes": 2 * P * (c["K"] + c["N"]) + used * c["N"] * c["K"] * per, "flops": 2 * P * c["N"] * c["K"]}
    return {"bytes": 4 * P * c["H"] + used * 3 * c["H"] * c["I"] * per, "flops": 6 * P * c["H"] * c["I"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _norm_weights(c, gen, kind, bias=True):
    if not kind:
        return None, None
    w = (1.0 - c["offset"] + 0.2 * _randn(gen, c["H"])).to(_dtype(c["w"]))
    return w, (0.1 * _randn(gen, c["H"])).to(_dtype(c["w"])) if kind == "layer" and bias else None


def _routing(gen, T, k, E, budgets=False):
    """A batch's picks, popular experts more often, and the maps that sort the live pairs by expert."""
    popular = 0.6 * _randn(gen, E)
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-6, 1 - 1e-6)))
    idx = (popular + noise).topk(k, dim=1).indices
    live = torch.ones(T, k, dtype=torch.bool, device="cuda")
    if budgets:
        live = torch.arange(k, device="cuda") < torch.randint(1, k + 1, (T, 1), generator=gen, device="cuda")
    flat = torch.where(live, idx, E).reshape(-1)
    order = torch.argsort(flat, stable=True)[:int(live.sum())]
    count = torch.bincount(flat, minlength=E)[:E]
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]).to(torch.int32)
    back = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    back[order] = torch.arange(len(order), device="cuda", dtype=torch.int32)
    return dict(offsets=offsets, experts=torch.arange(E, device="cuda", dtype=torch.int32), pair_to_sorted=back,
                P=len(order), live=live)


def _weights(c, gen, E, rows, K):
    """Codes [E, rows, K / 2], scales and zero points [E, rows, K / group] of N(0, 1 / K) weights."""
    g = c["group"]
    codes, scales, zeros = [], [], []
    per = max(1, (1 << 26) // (rows * K))
    for e0 in range(0, E, per):
        w = _randn(gen, min(per, E - e0), rows, K // g, g) / math.sqrt(K)
        if c["zeros"]:  # the range of a group, with 0 inside it
            lo, hi = w.amin(-1, keepdim=True).clamp_max(0), w.amax(-1, keepdim=True).clamp_min(0)
            s = ((hi - lo) / 15).to(_dtype(c["scale"]))
            z = torch.round(-lo / s.float()).clamp(0, 15)
            zeros.append(z.squeeze(-1).to(torch.uint8))
        else:
            s, z = (w.abs().amax(-1, keepdim=True) / 7).to(_dtype(c["scale"])), 8
        q = (torch.round(w / s.float()) + z).clamp(0, 15).to(torch.uint8).flatten(-2)
        codes.append(q[..., 0::2] | (q[..., 1::2] << 4))
        scales.append(s.squeeze(-1))
    return torch.cat(codes), torch.cat(scales), torch.cat(zeros) if zeros else None


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] in ("norm", "after"):
        T, H, dt = c["T"], c["H"], _dtype(c["x"])
        size = torch.exp(_randn(gen, T, 1))  # rows of different size
    if c["op"] == "norm":
        x = (_randn(gen, T, H) * size + (0.5 * size if c["kind"] == "layer" else 0.0)).to(dt)
        w, b = _norm_weights(c, gen, c["kind"])
        if c["bias"] and b is None:
            b = (0.1 * _randn(gen, H)).to(_dtype(c["w"]))
        return dict(case=c, x=x, w=w, b=b if c["bias"] else None)
    if c["op"] == "after":
        s = dict(case=c, residual=(2 * _randn(gen, T, H) * size).to(dt), maps=None, gates=None)
        if c["k"]:
            r = _routing(gen, T, c["k"], 4 * c["k"], c["budgets"])
            gates = torch.rand(T, c["k"], generator=gen, device="cuda") + 0.1
            gates = torch.where(r["live"], gates, 0)
            s.update(maps=r["pair_to_sorted"], gates=gates / gates.sum(1, keepdim=True), P=r["P"])
        s["y"] = _randn(gen, s["P"] if c["k"] else T, H).to(dt)
        s["shared"] = _randn(gen, T, H).to(dt) if c["shared"] else None
        s["gate"] = None
        if c["gate"]:
            s["gate"] = 0.5 + 0.3 * _randn(gen, T if c["gate"] == "tokens" else 1, H)
            s["gate"] = s["gate"].to(dt if c["gate"] == "tokens" else _dtype(c["w"]))
        s["post_w"], s["post_b"] = _norm_weights(c, gen, c["post"])
        s["next_w"], s["next_b"] = _norm_weights(c, gen, c["next"])
        return s
    T, k, E = c["T"], c["k"], c["E"]
    r = _routing(gen, T, k, E)
    tokens = _randn(gen, T, c["K"] if c["op"] == "product" else c["H"]).to(torch.bfloat16)
    x = torch.empty(r["P"], tokens.shape[1], dtype=torch.bfloat16, device="cuda")
    x[r["pair_to_sorted"].long()] = tokens.repeat_interleave(k, 0)
    if c["op"] == "product":
        return dict(case=c, x=x, w=_weights(c, gen, E, c["N"], c["K"]), **r)
    return dict(case=c, x=x, w13=_weights(c, gen, E, 2 * c["I"], c["H"]), w2=_weights(c, gen, E, c["H"], c["I"]), **r)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _norm(x, kind, w, b, offset):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    if w is not None:
        y = y * (w.float() + offset)
    return y if b is None else y + b.float()


def _after_plain(s):
    c = s["case"]
    T, H, k, dt = c["T"], c["H"], c["k"], _dtype(c["x"])
    if k:
        q = s["maps"].reshape(T, k)
        y = torch.zeros(T, H, device="cuda") if s["shared"] is None else s["shared"].float()
        for j in range(k):
            row = s["y"][q[:, j].clamp_min(0).long()].float()
            y = y + torch.where(q[:, j:j + 1] >= 0, s["gates"][:, j:j + 1] * row, 0)
    else:
        y = s["y"].float() if s["shared"] is None else s["shared"].float() + s["y"].float()
    if c["post"]:
        y = _norm(y, c["post"], s["post_w"], s["post_b"], c["offset"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    out = c["res_scale"] * s["residual"].float() + c["block_scale"] * y
    res = dict(out=out.to(dt))
    if c["next"]:
        res["next"] = _norm(out, c["next"], s["next_w"], s["next_b"], c["offset"]).to(dt)
    return res


def _matrices(w, group):
    """fp32 matrices [E, rows, K] of codes, scales and zero points."""
    codes, scales, zeros = w
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, group))
    q -= 8.0 if zeros is None else zeros.unsqueeze(-1).float()
    q *= scales.unsqueeze(-1).float()
    return q.flatten(-2)


def _by_expert(s, rows):
    """Rows [P, K] padded to [E, longest group, K], and where each row sits in it."""
    off = s["offsets"].long()
    count = off[1:] - off[:-1]
    longest = int(count.max())
    e_of = torch.repeat_interleave(torch.arange(len(count), device=off.device), count)
    slot = e_of * longest + torch.arange(len(e_of), device=off.device) - off[:-1][e_of]
    out = rows.new_zeros(len(count) * longest, rows.shape[1])
    out[slot] = rows
    return out.reshape(len(count), longest, -1), slot


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return dict(out=_norm(s["x"].float(), c["kind"], s["w"], s["b"], c["offset"]).to(_dtype(c["x"])))
    if c["op"] == "after":
        return _after_plain(s)
    a, slot = _by_expert(s, s["x"].float())
    if c["op"] == "product":
        out = torch.bmm(a, _matrices(s["w"], c["group"]).transpose(1, 2))
        return dict(out=out.flatten(0, 1)[slot].to(torch.bfloat16))
    I = c["I"]
    gu = torch.bmm(a, _matrices(s["w13"], c["group"]).transpose(1, 2))
    g, u = gu[..., :I], gu[..., I:]
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.bmm(h, _matrices(s["w2"], c["group"]).transpose(1, 2))
    return dict(y=y.flatten(0, 1)[slot].to(torch.bfloat16))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _run_own(s):
    from token_expert_routing_gb300 import _abi as abi
    c = s["case"]
    kinds = {"": abi.SEMMOE_NORM_NONE, "rms": abi.SEMMOE_NORM_RMS, "layer": abi.SEMMOE_NORM_LAYER}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        out = _empty((T, H), _dtype(c["x"]))
        abi.semmoe_norm(s["x"], T, H, kinds[c["kind"]], s["w"], s["b"], c["offset"], EPS, out)
        return dict(out=out)
    if c["op"] == "after":
        T, H = c["T"], c["H"]
        out = _empty((T, H), _dtype(c["x"]))
        nxt = _empty((T, H), _dtype(c["x"])) if c["next"] else None
        abi.semmoe_combine_norm(s["y"], s["maps"], s["gates"], s["shared"], T, H, c["k"], len(s["y"]), kinds[c["post"]],
                                s["post_w"], s["post_b"], kinds[c["next"]], s["next_w"], s["next_b"], c["offset"], EPS,
                                s["gate"], 0 if s["gate"] is None else len(s["gate"]), c["block_scale"], s["residual"],
                                c["res_scale"], out, nxt)
        return dict(out=out, next=nxt) if c["next"] else dict(out=out)
    P, E = s["P"], c["E"]
    if c["op"] == "product":
        out = _empty((P, c["N"]), torch.bfloat16)
        abi.semmoe_w4_grouped_gemm(s["x"], s["offsets"], s["experts"], *s["w"], P, E, c["N"], c["K"], c["group"], out)
        return dict(out=out)
    H, I = c["H"], c["I"]
    y = _empty((P, H), torch.bfloat16)
    abi.semmoe_w4_grouped_ffn(s["x"], s["offsets"], s["experts"], *s["w13"], *s["w2"], P, E, H, I, c["group"], y)
    return dict(y=y)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_norm(x, kind, w, b, offset):
    """Row by row statistics: the mean is taken off first, the squares are averaged about it."""
    n = x.shape[1]
    if kind == "layer":
        x = x - (x.sum(1) / n).unsqueeze(1)
    var = torch.einsum("th,th->t", x, x) / n
    y = x / torch.sqrt(var + EPS).unsqueeze(1)
    scale = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double() + offset
    shift = torch.zeros_like(scale) if b is None else b.double()
    return torch.addcmul(shift, y, scale)


def _exact_after(s):
    c = s["case"]
    T, H, k = c["T"], c["H"], c["k"]
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    if k:
        pair = torch.nonzero(s["maps"] >= 0).flatten()
        for p in pair.split(1 << 14):
            rows = s["y"][s["maps"][p].long()].double() * s["gates"].reshape(-1)[p].double().unsqueeze(1)
            y.index_add_(0, torch.div(p, k, rounding_mode="floor"), rows)
    else:
        y += s["y"].double()
    if s["shared"] is not None:
        y += s["shared"].double()
    if c["post"]:
        y = _exact_norm(y, c["post"], s["post_w"], s["post_b"], c["offset"])
    if s["gate"] is not None:
        y *= s["gate"].double()
    out = y * c["block_scale"] + s["residual"].double() * c["res_scale"]
    if not c["next"]:
        return dict(out=out)
    return dict(out=out, next=_exact_norm(out, c["next"], s["next_w"], s["next_b"], c["offset"]))


def _exact_matrix(w, e, group):
    """Matrix e of codes, scales and zero points in 64 bits."""
    codes, scales, zeros = w
    rows, half = codes[e].shape
    q = torch.empty(rows, 2 * half, dtype=torch.float64, device=codes.device)
    q[:, 0::2] = torch.remainder(codes[e], 16).double()
    q[:, 1::2] = torch.div(codes[e], 16, rounding_mode="floor").double()
    z = torch.full(scales[e].shape, 8.0, dtype=torch.float64, device=codes.device) if zeros is None else zeros[e].double()
    return (q - z.repeat_interleave(group, 1)) * scales[e].double().repeat_interleave(group, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        return dict(out=_exact_norm(s["x"].double(), c["kind"], s["w"], s["b"], c["offset"]))
    if c["op"] == "after":
        return _exact_after(s)
    off, P, E = s["offsets"].tolist(), s["P"], c["E"]
    out = torch.empty(P, c["N"] if c["op"] == "product" else c["H"], dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        a = s["x"][lo:hi].double()
        if c["op"] == "product":
            out[lo:hi] = a @ _exact_matrix(s["w"], e, c["group"]).T
            continue
        gu = a @ _exact_matrix(s["w13"], e, c["group"]).T
        g, u = gu[:, :c["I"]], gu[:, c["I"]:]
        out[lo:hi] = (g * torch.sigmoid(g) * u) @ _exact_matrix(s["w2"], e, c["group"]).T
    return dict(out=out) if c["op"] == "product" else dict(y=out)
