"""Measured cases of the expert-choice router and the 4-bit microscaled operators.

Four operators of an MoE layer's forward, each through its public call:

* ``route``:    semmoe_route_select -- router product, sigmoid or softmax scores, a bias that only
                chooses, groups, top-k, weights;
* ``quantize``: semmoe_mx4_quantize + semmoe_mx4_dequantize -- 32-value blocks with a power-of-two
                scale and 4-bit (e2m1) values, and the values they stand for;
* ``product``:  semmoe_mx4_grouped_gemm -- 4-bit rows, sorted by expert, times their expert's 4-bit matrix;
* ``ffn``:      semmoe_mx4_quantize_rows + semmoe_mx4_grouped_ffn -- token rows quantised into expert order,
                then the SwiGLU experts with a 4-bit hidden activation.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math

import torch

own = False

BLOCK = 32        # values per scale
TILE = 128        # rows per tile of the scales' layout
CHUNK = 128       # packed values per row of a tile: four scales
COUNT_CHUNK = 128  # tokens per column of the router's count table


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token routed over 256 experts in 8 groups, 4 kept: latency alone
        dict(name="route_T1_E256", op="route", T=1, H=2048, E=256, k=8, score="sigmoid", bias=True, off=0, G=8, keep=4,
             top=2, renorm=True, scale=2.5, budgets=False, w="bf16"),
        # a decode batch with a budget per request, softmax scores not renormalised, group maxima, an fp32 router
        dict(name="route_T512_E64_budgets", op="route", T=512, H=2048, E=64, k=6, score="softmax", bias=False, off=0,
             G=8, keep=3, top=1, renorm=False, scale=1.0, budgets=True, w="f32"),
        # a prefill batch, balance bias, two experts switched off, no groups
        dict(name="route_T16384_E128", op="route", T=16384, H=2048, E=128, k=8, score="sigmoid", bias=True, off=2, G=1,
             keep=1, top=1, renorm=True, scale=1.0, budgets=False, w="bf16"),
        # activations of narrow experts, fp32, a ragged last tile and a K that is no multiple of a tile's
        dict(name="quantize_1003x352_f32", op="quantize", groups=1, rows=1003, K=352, x="f32"),
        # one layer's gate and up weights: 64 experts x 2 x 1408 rows of 2048, bf16
        dict(name="quantize_w13_64x2x1408x2048", op="quantize", groups=128, rows=1408, K=2048, x="bf16"),
        # a decode batch's second expert product, fp32 out (to be reduced further)
        dict(name="product_T64_1408to2048_f32", op="product", T=64, k=6, E=64, N=2048, K=1408, out="f32"),
        # a prefill batch's second expert product
        dict(name="product_T16384_768to2048", op="product", T=16384, k=8, E=128, N=2048, K=768, out="bf16"),
        # one decoded token through 8 of 128 experts
        dict(name="ffn_T1_E128", op="ffn", T=1, k=8, E=128, H=2048, I=768),
        # a decode batch that touches nearly every expert: bound by the weights' bytes
        dict(name="ffn_T64_E64", op="ffn", T=64, k=6, E=64, H=2048, I=1408),
        # odd sizes: hidden 33 blocks, narrow experts, ragged groups
        dict(name="ffn_T777_odd", op="ffn", T=777, k=3, E=23, H=1056, I=352),
        # prefill, 64 experts of 1408
        dict(name="ffn_T4096_E64", op="ffn", T=4096, k=6, E=64, H=2048, I=1408),
        # the largest prefill: 131072 rows over 128 experts of 768
        dict(name="ffn_T16384_E128", op="ffn", T=16384, k=8, E=128, H=2048, I=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "quantize", "product", "ffn", "ffn"])
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8])
        per = max(2, _log(rng, 8, 256) // G)
        E = G * per
        keep = rng.randint(max(1, G // 2), G)
        k = rng.randint(1, min(12, keep * per))
        return dict(op=op, T=_log(rng, 1, 16384), H=8 * _log(rng, 16, 256), E=E, k=k,
                    score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6,
                    off=0, G=G, keep=keep, top=rng.choice([1, 2]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), budgets=rng.random() < 0.3, w=rng.choice(["bf16", "f32"]))
    if op == "quantize":
        return dict(op=op, groups=_log(rng, 1, 64), rows=_log(rng, 1, 1500), K=BLOCK * _log(rng, 1, 64),
                    x=rng.choice(["bf16", "f32"]))
    T, E = _log(rng, 1, 8192), _log(rng, 4, 128)
    k = rng.randint(1, min(8, E))
    if op == "product":
        return dict(op=op, T=T, k=k, E=E, N=8 * _log(rng, 8, 256), K=BLOCK * _log(rng, 1, 64),
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, T=T, k=k, E=E, H=BLOCK * _log(rng, 4, 64), I=BLOCK * _log(rng, 4, 44))


def work(case):
    c = case
    if c["op"] == "route":
        T, H, E = c["T"], c["H"], c["E"]
        table = E * (-(-(-(-T // COUNT_CHUNK)) // 4) * 4) * 4
        return {"bytes": T * H * 2 + E * H * (2 if c["w"] == "bf16" else 4) + T * c["k"] * 8 + table
                + (4 * E if c["bias"] else 0) + (4 * T if c["budgets"] else 0), "flops": 2 * T * H * E}
    if c["op"] == "quantize":
        n = c["groups"] * c["rows"] * c["K"]
        return {"bytes": n * (2 if c["x"] == "bf16" else 4) + n * 17 / 32 + n * 2, "flops": 4 * n}
    P = c["T"] * c["k"]
    used = min(c["E"], P)  # experts that have rows, at most
    if c["op"] == "product":
        N, K = c["N"], c["K"]
        return {"bytes": (P * K + used * N * K) * 17 / 32 + P * N * (2 if c["out"] == "bf16" else 4),
                "flops": 2 * P * N * K}
    H, I = c["H"], c["I"]
    return {"bytes": c["T"] * H * 2 + used * 3 * H * I * 17 / 32 + P * H * 2, "flops": 6 * P * H * I}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _encode(x):
    """Codes (uint8, 0..15) and biased scale exponents (uint8) of the rows of x, blocks of 32 along K."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(b, -e)
    m = v.abs()
    # round to nearest, ties to the even code: a midpoint below an odd code stays, one below an even code goes up
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + 8 * (torch.signbit(v)).to(torch.uint8)
    return code.flatten(-2), (e + 127).to(torch.uint8).squeeze(-1)


def _pack(code):
    c = code.unflatten(-1, (-1, 2))
    return (c[..., 0] | (c[..., 1] << 4)).contiguous()


def _scale_tiles(s, groups, rows):
    """Scales [groups * rows, K / 32] in tiles of 128 rows x 128 packed values (512 bytes, row r of a tile at
    byte 16 (r % 32) + 4 (r / 32) of each), every group starting a tile."""
    kb = s.shape[-1]
    s = s.reshape(groups, rows, kb)
    s = torch.nn.functional.pad(s, (0, -kb % 4, 0, -rows % TILE))
    s = s.reshape(groups, -1, 4, 32, (kb + 3) // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return s.reshape(-1).contiguous()


def _row_slots(rows_of, place):
    """Where scale block 0 of rows sits in _scale_tiles' tiles: (tile, byte) for rows `place` of groups of rows_of rows."""
    tiles = (rows_of + TILE - 1) // TILE
    base = torch.cumsum(tiles, 0) - tiles
    return base, place // TILE, 16 * (place % 32) + 4 * ((place % TILE) // 32)


def _weights(gen, groups, rows, K):
    """Codes [groups, rows, K / 2] and scale tiles of a weight matrix per group, N(0, 1 / K) before quantisation."""
    codes, scales = [], []
    per = max(1, (1 << 27) // (rows * K))
    for g0 in range(0, groups, per):
        n = min(per, groups - g0)
        w = torch.randn(n * rows, K, generator=gen, device="cuda") / math.sqrt(K)
        c, s = _encode(w.to(torch.bfloat16))
        codes.append(_pack(c))
        scales.append(_scale_tiles(s, n, rows))
    return torch.cat(codes).reshape(groups, rows, K // 2), torch.cat(scales)


def _routing(gen, T, k, E):
    """A batch's picks, popular experts more often, and the maps that sort the pairs by expert."""
    popular = 0.6 * torch.randn(E, generator=gen, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-6, 1 - 1e-6)))
    idx = (popular + noise).topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(idx, stable=True)
    count = torch.bincount(idx, minlength=E)
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]).to(torch.int32)
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device="cuda")
    return dict(offsets=offsets, experts=torch.arange(E, device="cuda", dtype=torch.int32),
                sorted_to_pair=order.to(torch.int32), pair_to_sorted=back.to(torch.int32))


def _margins(c, logits64, bias):
    """Rows whose picks no sum in another order changes: every gap that decides is well above rounding."""
    E, k, G = c["E"], c["k"], c["G"]
    s = torch.sigmoid(logits64) if c["score"] == "sigmoid" else torch.softmax(logits64, -1)
    ch = s if bias is None else s + bias.double()
    tol = 3e-5 * (1.0 if c["score"] == "sigmoid" else s.amax(-1))
    ok = torch.ones(len(s), dtype=torch.bool, device=s.device)
    live = ch
    if c["keep"] < G:
        g = ch.unflatten(-1, (G, -1))
        g = g.sort(dim=-1, descending=True).values[..., :c["top"]].clamp_min(-8.0).sum(-1)
        gs, at = g.sort(dim=-1, descending=True, stable=True)
        ok &= gs[:, c["keep"] - 1] - gs[:, c["keep"]] > tol
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, at[:, :c["keep"]], True)
        live = torch.where(keep.repeat_interleave(E // G, 1), ch, torch.full_like(ch, -math.inf))
    top = live.sort(dim=-1, descending=True).values[:, :k + 1]
    if top.shape[1] > 1:
        gap = top[:, :-1] - top[:, 1:]
        ok &= ((gap > 0.25 * tol.unsqueeze(1) if torch.is_tensor(tol) else gap > 0.25 * tol) | torch.isinf(top[:, 1:])).all(1)
    return ok


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "route":
        T, H, E = c["T"], c["H"], c["E"]
        w = (torch.randn(E, H, generator=gen, device="cuda") / math.sqrt(H)).to(_dtype(c["w"]))
        bias = 0.05 * torch.randn(E, generator=gen, device="cuda") if c["bias"] else None
        if c["off"]:
            bias[torch.randperm(E, generator=gen, device="cuda")[:c["off"]]] = -math.inf
        x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
        for _ in range(8):  # tokens whose picks hang on the last bits are drawn again
            bad = ~_margins(c, x.double() @ w.double().T, bias)
            x = torch.where(bad.unsqueeze(1), torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16), x)
        kpt = torch.randint(1, c["k"] + 1, (T,), generator=gen, device="cuda", dtype=torch.int32) if c["budgets"] else None
        return dict(case=c, x=x, w=w, bias=bias, kpt=kpt)
    if c["op"] == "quantize":
        M, K = c["groups"] * c["rows"], c["K"]
        x = torch.randn(M, K, generator=gen, device="cuda")
        x *= torch.exp(torch.randn(M, 1, generator=gen, device="cuda"))  # rows of different size
        x[:, ::37] *= 8.0                                                # and columns that stand out
        return dict(case=c, x=x.to(_dtype(c["x"])))
    T, k, E = c["T"], c["k"], c["E"]
    r = _routing(gen, T, k, E)
    if c["op"] == "product":
        K, P = c["K"], T * k
        code, s = _encode(torch.randn(P, K, generator=gen, device="cuda").to(torch.bfloat16))
        # the rows' scales in expert order: a tile of 128 rows never spans two experts
        count = (r["offsets"][1:] - r["offsets"][:-1]).long()
        e_of = torch.repeat_interleave(torch.arange(E, device="cuda"), count)
        base, tile, byte = _row_slots(count, torch.arange(P, device="cuda") - r["offsets"][:-1].long()[e_of])
        kc = -(-K // CHUNK)
        tiles = torch.zeros((P // TILE + E) * kc * 512, dtype=torch.uint8, device="cuda")
        kb = torch.arange(K // BLOCK, device="cuda")
        at = ((base[e_of] + tile) * kc).unsqueeze(1) * 512 + (kb // 4) * 512 + byte.unsqueeze(1) + kb % 4
        tiles[at] = s
        wc, ws = _weights(gen, E, c["N"], K)
        return dict(case=c, a=_pack(code), a_scales=tiles, b=wc, b_scales=ws, **r)
    x = torch.randn(T, c["H"], generator=gen, device="cuda").to(torch.bfloat16)
    w13, s13 = _weights(gen, 2 * E, c["I"], c["H"])
    w2, s2 = _weights(gen, E, c["H"], c["I"])
    return dict(case=c, x=x, w13=w13.reshape(E, 2 * c["I"], -1), s13=s13, w2=w2, s2=s2, **r)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _values(code, e):
    """fp32 values of codes [..., K] with biased exponents e [..., K / 32]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = table[(code & 7).long()]
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, BLOCK))
    return torch.ldexp(v, (e.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def _untile(tiles, groups, rows, K):
    kc, nt = -(-K // CHUNK), -(-rows // TILE)
    s = tiles[:groups * nt * kc * 512].reshape(groups, nt, kc, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    return s.reshape(groups, nt * TILE, kc * 4)[:, :rows, :K // BLOCK]


def _matrices(codes, tiles, groups, rows, K):
    return _values(_unpack(codes).reshape(groups, rows, K), _untile(tiles, groups, rows, K))


def _round_trip(x):
    return _values(*_encode(x))


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


def _route_plain(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    logits = s["x"].float() @ s["w"].float().T
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, -1)
    choice = logits if s["bias"] is None else score + s["bias"]
    if c["keep"] < G:
        by = score if s["bias"] is None else choice
        g = by.unflatten(-1, (G, -1)).sort(dim=-1, descending=True).values[..., :c["top"]]
        g = torch.where(torch.isinf(g[..., :1]), g[..., :1], torch.where(torch.isinf(g), 0, g).sum(-1, keepdim=True)).squeeze(-1)
        best = g.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, best, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, torch.full_like(choice, -math.inf))
    top = choice.sort(dim=-1, descending=True, stable=True)
    idx, picked = top.indices[:, :k], ~torch.isinf(top.values[:, :k])
    if s["kpt"] is not None:
        picked = picked & (torch.arange(k, device=idx.device) < s["kpt"].unsqueeze(1))
    w = torch.where(picked, score.gather(1, idx), 0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    idx = torch.where(picked, idx, -1).to(torch.int32)
    chunks = -(-T // COUNT_CHUNK)
    width = -(-chunks // 4) * 4
    at = idx.long() * width + (torch.arange(T, device=idx.device) // COUNT_CHUNK).unsqueeze(1)
    counts = torch.bincount(at[picked], minlength=E * width).reshape(E, width).to(torch.int32)
    return dict(idx=idx, w=w * c["scale"], counts=counts)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _route_plain(s)
    if c["op"] == "quantize":
        return dict(values=_round_trip(s["x"]).to(torch.bfloat16))
    E = c["E"]
    if c["op"] == "product":
        N, K, P = c["N"], c["K"], c["T"] * c["k"]
        off = s["offsets"].long()
        count = off[1:] - off[:-1]
        e_of = torch.repeat_interleave(torch.arange(E, device=off.device), count)
        base, tile, byte = _row_slots(count, torch.arange(P, device=off.device) - off[:-1][e_of])
        kc = -(-K // CHUNK)
        kb = torch.arange(K // BLOCK, device=off.device)
        at = ((base[e_of] + tile) * kc).unsqueeze(1) * 512 + (kb // 4) * 512 + byte.unsqueeze(1) + kb % 4
        a, slot = _by_expert(s, _values(_unpack(s["a"]), s["a_scales"][at]))
        out = torch.bmm(a, _matrices(s["b"], s["b_scales"], E, N, K).transpose(1, 2))
        return dict(out=out.flatten(0, 1)[slot].to(_dtype(c["out"])))
    H, I = c["H"], c["I"]
    rows = _round_trip(s["x"])[(s["sorted_to_pair"] // c["k"]).long()]
    a, slot = _by_expert(s, rows)
    w13 = _matrices(s["w13"], s["s13"], 2 * E, I, H).reshape(E, 2 * I, H)
    gu = torch.bmm(a, w13.transpose(1, 2))
    g, u = gu[..., :I], gu[..., I:]
    h = _round_trip(g / (1.0 + torch.exp(-g)) * u)
    y = torch.bmm(h, _matrices(s["w2"], s["s2"], E, H, I).transpose(1, 2))
    return dict(y=y.flatten(0, 1)[slot].to(torch.bfloat16))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _empty(n, dtype):
    return torch.empty(n, dtype=dtype, device="cuda")


def _run_own(s):
    from token_expert_routing_gb300 import _abi as abi
    c = s["case"]
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        idx, w = _empty((T, k), torch.int32), _empty((T, k), torch.float32)
        counts = _empty((E, abi.semmoe_pair_counts_stride(T)), torch.int32)
        score = abi.SEMMOE_SCORE_SIGMOID if c["score"] == "sigmoid" else abi.SEMMOE_SCORE_SOFTMAX
        abi.semmoe_route_select(s["x"], s["w"], None, None, score, s["bias"], c["G"], c["keep"], c["top"], c["renorm"],
                                c["scale"], s["kpt"], 0 if c["budgets"] else k, T, c["H"], E, k, idx, w,
                                pair_counts=counts)
        return dict(idx=idx, w=w, counts=counts)
    if c["op"] == "quantize":
        G, n, K = c["groups"], c["rows"], c["K"]
        codes = _empty((G * n, K // 2), torch.uint8)
        scales = _empty(abi.semmoe_mx4_scales_size(G * n, K, G), torch.uint8)
        values = _empty((G * n, K), torch.bfloat16)
        abi.semmoe_mx4_quantize(s["x"], G, n, K, codes, scales)
        abi.semmoe_mx4_dequantize(codes, scales, G, n, K, values)
        return dict(values=values)
    P, E = c["T"] * c["k"], c["E"]
    if c["op"] == "product":
        out = _empty((P, c["N"]), _dtype(c["out"]))
        abi.semmoe_mx4_grouped_gemm(s["a"], s["a_scales"], s["offsets"], s["experts"], s["b"], s["b_scales"], P, E,
                                    c["N"], c["K"], out)
        return dict(out=out)
    H, I = c["H"], c["I"]
    xq = _empty((P, H // 2), torch.uint8)
    xs = _empty(abi.semmoe_mx4_scales_size(P, H, E), torch.uint8)
    y = _empty((P, H), torch.bfloat16)
    ws = _empty(abi.semmoe_mx4_grouped_ffn_workspace_size(P, E, I), torch.uint8)
    abi.semmoe_mx4_quantize_rows(s["x"], c["T"], H, s["pair_to_sorted"], c["k"], P, s["offsets"], E, xq, xs)
    abi.semmoe_mx4_grouped_ffn(xq, xs, s["offsets"], s["experts"], s["w13"], s["s13"], s["w2"], s["s2"], P, E, H, I, y, ws)
    return dict(y=y)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_quantised(x):
    """The values that x's 4-bit blocks stand for, in 64 bits: a power of two per block, then the grid's own step."""
    b = x.double().reshape(len(x), -1, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    exponent = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    exponent = torch.where(torch.exp2(exponent) > amax, exponent - 1, exponent)          # log2 rounded up
    exponent = torch.where(torch.exp2(exponent + 1) <= amax, exponent + 1, exponent)     # or down
    scale = torch.exp2((exponent - 2).clamp(-127, 127))
    v = b / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
    q = (torch.round(v / step) * step).clamp(-6, 6)
    return (torch.where(amax > 0, q * scale, torch.zeros_like(q))).reshape(x.shape)


def _exact_matrix(codes, scales):
    """[rows, K] in 64 bits from packed codes and scales [rows, K / 32]."""
    c = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes & 15).long(), (codes >> 4).long()
    exponent, half = (c >> 1) & 3, (c & 1).double()
    size = torch.where(exponent == 0, 0.5 * half, torch.exp2(exponent.double() - 1) * (1 + 0.5 * half))
    size = torch.where((c & 8) != 0, -size, size)
    return size * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def _exact_scales(tiles, first_tile, rows, K):
    """[rows, K / 32] of one group whose scales start at tile first_tile."""
    kc = -(-K // CHUNK)
    r = torch.arange(rows, device=tiles.device).unsqueeze(1)
    b = torch.arange(K // BLOCK, device=tiles.device).unsqueeze(0)
    at = ((first_tile + r // 128) * kc + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    return tiles[at]


def _exact_route(s):
    c = s["case"]
    E, k, G, T = c["E"], c["k"], c["G"], c["T"]
    n = E // G
    logits = s["x"].double() @ s["w"].double().T
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        p = torch.exp(logits - logits.max(1, keepdim=True).values)
        score = p / p.sum(1, keepdim=True)
    choice = score.clone() if s["bias"] is None else score + s["bias"].double()
    live = torch.isfinite(choice)
    if c["keep"] < G:
        total = torch.stack([choice[:, g * n:(g + 1) * n].topk(c["top"], 1).values.sum(1) for g in range(G)], 1)
        rank = (total.unsqueeze(1) > total.unsqueeze(2)).sum(2)
        live &= (rank < c["keep"]).repeat_interleave(n, 1)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=score.device)
    w = torch.zeros(T, k, dtype=torch.float64, device=score.device)
    row = torch.arange(T, device=score.device)
    for j in range(k):
        left = torch.where(live, choice, -math.inf)
        best, e = left.max(1)
        take = torch.isfinite(best)
        if s["kpt"] is not None:
            take &= s["kpt"] > j
        idx[:, j] = torch.where(take, e, -1).to(torch.int32)
        w[:, j] = torch.where(take, score[row, e], 0)
        live[row, e] = False
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(idx=idx, w=w * c["scale"], counts=None)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        return _exact_route(s)
    if c["op"] == "quantize":
        return dict(values=torch.cat([_exact_quantised(x) for x in s["x"].split(1 << 15)]))
    off = s["offsets"].tolist()
    P, E = off[-1], c["E"]
    if c["op"] == "product":
        N, K = c["N"], c["K"]
        out = torch.empty(P, N, dtype=torch.float64, device="cuda")
        tile = 0
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            a = _exact_matrix(s["a"][lo:hi], _exact_scales(s["a_scales"], tile, hi - lo, K))
            b = _exact_matrix(s["b"][e], _exact_scales(s["b_scales"], e * -(-N // TILE), N, K))
            out[lo:hi] = a @ b.T
            tile += -(-(hi - lo) // TILE)
        return dict(out=out)
    H, I = c["H"], c["I"]
    x = _exact_quantised(s["x"])
    y = torch.empty(P, H, dtype=torch.float64, device="cuda")
    ti, th = -(-I // TILE), -(-H // TILE)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        a = x[torch.div(s["sorted_to_pair"][lo:hi].long(), c["k"], rounding_mode="floor")]
        g = a @ _exact_matrix(s["w13"][e, :I], _exact_scales(s["s13"], 2 * e * ti, I, H)).T
        u = a @ _exact_matrix(s["w13"][e, I:], _exact_scales(s["s13"], (2 * e + 1) * ti, I, H)).T
        h = _exact_quantised(g / (1 + torch.exp(-g)) * u)
        y[lo:hi] = h @ _exact_matrix(s["w2"][e], _exact_scales(s["s2"], e * th, H, I)).T
    return dict(y=y)
