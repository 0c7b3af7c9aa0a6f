"""Workloads of the routing to experts, the movement of their rows, and the block-scaled (microscaling) experts.

What a mixture-of-experts layer calls around its grouped products, one operator a pass:

* ``route``         the router's scores (softmax or sigmoid) to each token's experts and weights, with a bias for
                    balance, groups of experts and renormalised weights; ``route_grad`` its gradient.
* ``rows``          the (token, expert) pairs sorted by expert: offsets, the row of each pair, the pair of each row.
* ``gather``        rows of tokens copied into expert order; ``combine`` the weighted sum back; ``combine_grad``
                    the gradients of the rows and of the weights.
* ``quantize``      rows to block-scaled numbers (a shared power of two per 32) and back to 16 bits: the values that
                    4-bit or 8-bit inference sees.
* ``product``       y[r] = act(x[r] W[e(r)]^T + bias[e(r)]) over block-scaled codes, rows grouped by expert.

``run`` computes them in plain torch operations, or through the library when ``own`` is true.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EMAX = {"e2m1": 2, "e4m3": 8}
_MOST = {"e2m1": 6.0, "e4m3": 448.0}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One decoded token: launch latency.
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 128, "top": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_sum": 1, "renorm": True, "scale": 1.0, "dtype": "f32",
         "masked": 0.0},
        # A long prompt, many small experts in groups, sigmoid scores with a bias for balance.
        {"name": "route_prompt", "op": "route", "tokens": 16384, "experts": 256, "top": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_sum": 2, "renorm": True, "scale": 2.5, "dtype": "f32",
         "masked": 0.0},
        # Training with softmax scores that are not renormalised: every logit has a gradient.
        {"name": "route_grad", "op": "route_grad", "tokens": 16384, "experts": 128, "top": 8, "score": "softmax",
         "renorm": False, "scale": 1.0, "dtype": "f32", "masked": 0.02},
        # A decoding batch's pairs.
        {"name": "rows_batch", "op": "rows", "tokens": 128, "experts": 64, "top": 4, "dropped": 0.0, "skew": 0.7},
        # A long prompt's pairs, some tokens of which are padding.
        {"name": "rows_prompt", "op": "rows", "tokens": 16384, "experts": 256, "top": 8, "dropped": 0.05, "skew": 0.7},
        # The end of a layer, serving a prompt.
        {"name": "combine_prompt", "op": "combine", "tokens": 8192, "d": 4096, "top": 8, "dtype": "bf16",
         "out": "bf16", "dropped": 0.0, "pad": 0},
        # The same in training, odd sizes, some pairs dropped.
        {"name": "combine_grad", "op": "combine_grad", "tokens": 4099, "d": 2056, "top": 6, "dtype": "bf16",
         "dropped": 0.05, "pad": 0},
        # 64 rows of a decoding batch, gathered from its tokens.
        {"name": "quantize_batch", "op": "quantize", "tokens": 16, "top": 4, "k": 4096, "elem": "e2m1",
         "dtype": "bf16", "pad": 0},
        # The rows of a long prompt.
        {"name": "quantize_prompt", "op": "quantize", "tokens": 32768, "top": 1, "k": 4096, "elem": "e2m1",
         "dtype": "bf16", "pad": 0},
        # 4-bit experts, decoding: 16 tokens to 4 of 64 experts each, bound by the weights.
        {"name": "product_batch", "op": "product", "elem": "e2m1", "groups": 64, "rows": 64, "n": 2048, "k": 4096,
         "out": "bf16", "epi": "none", "skew": 0.7, "pad": 0},
        # 8-bit block-scaled experts at ragged sizes into fp32.
        {"name": "product_ragged", "op": "product", "elem": "e4m3", "groups": 24, "rows": 777, "n": 1000, "k": 1056,
         "out": "f32", "epi": "bias", "skew": 1.5, "pad": 1},
        # 4-bit experts, filling prompts: the largest product.
        {"name": "product_prompt", "op": "product", "elem": "e2m1", "groups": 32, "rows": 32768, "n": 4096, "k": 4096,
         "out": "bf16", "epi": "bias_silu", "skew": 0.5, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """A size over [lo, hi], log-uniform, in multiples of `step`: mostly of 64 as well."""
    v = _log_int(rng, lo, hi)
    return max(lo, v // step * step if rng.random() < 0.3 else v // 64 * 64)


def draw(rng):
    while True:
        op = rng.choice(["route", "route", "route_grad", "rows", "gather", "combine", "combine_grad", "quantize",
                         "quantize", "product", "product", "product"])
        case = {"op": op}
        if op in ("route", "route_grad", "rows"):
            case["tokens"] = _log_int(rng, 1, 16384)
            case["experts"] = rng.choice([8, 16, 60, 64, 128, 160, 256, 257])
            case["top"] = rng.randint(1, 8)
        if op in ("route", "route_grad"):
            case["score"] = rng.choice(["softmax", "sigmoid"])
            case["renorm"] = rng.random() < 0.5
            case["scale"] = rng.choice([1.0, 2.5])
            case["dtype"] = rng.choice(["f32", "f32", "f16", "bf16"])
            case["masked"] = rng.choice([0.0, 0.02, 0.3])
        if op == "route":
            case["bias"] = rng.random() < 0.5
            limited = case["experts"] % 8 == 0 and rng.random() < 0.5
            case["groups"] = 8 if limited else 1
            case["top_groups"] = rng.randint(2, 6) if limited else 1
            case["group_sum"] = rng.randint(1, 2) if limited else 1
        if op == "rows":
            case["dropped"] = rng.choice([0.0, 0.05, 0.5])
            case["skew"] = rng.choice([0.0, 0.7, 1.5])
        if op in ("gather", "combine", "combine_grad"):
            case["tokens"] = _log_int(rng, 1, 8192)
            case["d"] = _size(rng, 64, 8192, 1)
            case["top"] = rng.randint(1, 8)
            case["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
            case["dropped"] = rng.choice([0.0, 0.05, 0.5])
            case["pad"] = rng.choice([0, 0, 1])
        if op == "combine":
            case["out"] = rng.choice([case["dtype"], "f32"])
        if op == "quantize":
            case["tokens"] = _log_int(rng, 1, 32768)
            case["top"] = rng.choice([1, 1, 4, 8])
            case["k"] = _size(rng, 64, 8192, 32)
            case["elem"] = rng.choice(["e2m1", "e2m1", "e4m3"])
            case["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
            case["pad"] = rng.choice([0, 0, 1])
        if op == "product":
            case["elem"] = rng.choice(["e2m1", "e2m1", "e4m3"])
            case["groups"] = _log_int(rng, 1, 128)
            case["rows"] = _log_int(rng, 1, 32768)
            case["n"] = _size(rng, 256, 8192, 1)
            case["k"] = _size(rng, 256, 8192, 32)
            case["out"] = rng.choice(["bf16", "bf16", "f16", "f32"])
            case["epi"] = rng.choice(["none", "bias", "bias_silu", "bias_gelu"])
            case["skew"] = rng.choice([0.0, 0.5, 1.0, 1.5])
            case["pad"] = rng.choice([0, 0, 1])
        w = work(case)
        if w["flops"] <= 1.0e12 and w["bytes"] <= 8.0e8 and case.get("groups", 1) * case.get("n", 1) * case.get("k", 1) <= 6e8:
            return case


# ------------------------------------------------------------------ inputs --

def _counts(case, gen=None):
    """Rows per group: the same multiset for every seed (a power law of exponent `skew`), in a seeded order."""
    G, rows = case["groups"], case["rows"]
    p = [1.0 / (i + 1) ** case["skew"] for i in range(G)]
    share = [rows * v / sum(p) for v in p]
    counts = [int(v) for v in share]
    rest = sorted(range(G), key=lambda i: (counts[i] - share[i], i))
    for i in rest[:rows - sum(counts)]:
        counts[i] += 1
    if gen is None:
        return counts
    return [counts[i] for i in torch.randperm(G, generator=gen).tolist()]


def _pitch(n, pad, to):
    return (n + to - 1) // to * to + (to if pad else 0)


def _block_codes(x, elem):
    """The scale codes (rows x K/32) and the scaled blocks (rows x K/32 x 32, fp32) of the rows of x."""
    blocks = x.float().reshape(x.shape[0], -1, 32)
    peak = blocks.abs().amax(2)
    floor_log2 = torch.frexp(peak)[1] - 1
    e = torch.where(peak > 0, floor_log2 - _EMAX[elem], torch.full_like(floor_log2, -127)).clamp(-127, 127)
    # a power of two may leave fp32's range where the two halves of it do not
    half = torch.div(e, 2, rounding_mode="floor")
    scaled = torch.ldexp(torch.ldexp(blocks, -half[..., None]), (half - e)[..., None])
    return (e + 127).to(torch.uint8), scaled.clamp(-_MOST[elem], _MOST[elem])


def _e2m1_index(v):
    """Index of |v| among the eight magnitudes, nearest, ties to the even one."""
    a = v.abs()
    return ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())


def _codes(x, elem):
    """Element codes (as the library stores them: E2M1 two to a byte, even k low) and scale codes of the rows of x."""
    scale, scaled = _block_codes(x, elem)
    flat = scaled.reshape(x.shape[0], -1)
    if elem == "e4m3":
        return flat.to(torch.float8_e4m3fn).view(torch.uint8), scale
    c = _e2m1_index(flat) + 8 * torch.signbit(flat).int()
    return (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8), scale


def prepare(case, seed):
    dev = torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": dict(case), "dev": dev}
    op = case["op"]

    def normal(rows, cols, dtype, std=1.0, pad=0, to=8):
        t = torch.empty(rows, _pitch(cols, pad, to), dtype=dtype, device=dev)
        t.normal_(0.0, std, generator=gen)
        return t[:, :cols]

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    if op in ("route", "route_grad"):
        T, E, top = case["tokens"], case["experts"], case["top"]
        st["logits"] = normal(T, E, _DT[case["dtype"]], 1.5, to=1)
        if case["masked"]:  # experts that a token may not take, and padding tokens that may take none
            st["logits"].masked_fill_(uniform(T, E) < case["masked"], -math.inf)
            st["logits"].masked_fill_(uniform(T, 1) < case["masked"] / 2, -math.inf)
        if op == "route":
            st["bias"] = uniform(E) * 0.2 - 0.1 if case["bias"] else None
            st["expert"] = torch.empty(T, top, dtype=torch.int32, device=dev)
            st["weight"] = torch.empty(T, top, device=dev)
        else:
            st["expert"] = _choose(st["logits"].double(), top, None, 1, 1, 1)
            st["dweight"] = normal(T, top, torch.float32, to=1)
            st["dlogits"] = torch.empty(T, E, dtype=_DT[case["dtype"]], device=dev)
    elif op == "rows":
        T, E, top = case["tokens"], case["experts"], case["top"]
        p = torch.arange(1, E + 1, device=dev).float().pow(-case["skew"])
        p = p[torch.randperm(E, generator=host).to(dev)]
        # `top` different experts of each token, the likelier ones more often
        race = torch.log(uniform(T, E).clamp_min(1e-30)).neg() / p
        st["expert"] = race.argsort(1)[:, :top].to(torch.int32)
        st["expert"] = torch.where(uniform(T, top) < case["dropped"], torch.full_like(st["expert"], -1), st["expert"])
        st["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        st["row"] = torch.empty(T, top, dtype=torch.int32, device=dev)
        st["source"] = torch.empty(T * top, dtype=torch.int32, device=dev)
        st["workspace"] = torch.empty(4 << 20, dtype=torch.uint8, device=dev)
    elif op in ("gather", "combine", "combine_grad"):
        T, top, d, dt = case["tokens"], case["top"], case["d"], _DT[case["dtype"]]
        keep = uniform(T * top) >= case["dropped"]
        # the kept pairs' rows, in the order that sorting them by expert gives: any permutation
        order = torch.randperm(T * top, generator=host).to(dev)
        order = order[keep[order]]
        n = order.numel()
        st["rows"] = n
        st["source"] = torch.full((T * top,), -1, dtype=torch.int32, device=dev)
        st["source"][:n] = order.to(torch.int32)
        st["row"] = torch.full((T * top,), -1, dtype=torch.int32, device=dev)
        st["row"][order] = torch.arange(n, dtype=torch.int32, device=dev)
        st["row"] = st["row"].view(T, top)
        st["weight"] = uniform(T, top)
        if op != "gather":
            st["y"] = normal(T * top, d, dt, 1.0, case["pad"])
        if op != "combine":
            st["x"] = normal(T, d, dt, 1.0, case["pad"])
            st["out"] = torch.zeros(T * top, d, dtype=dt, device=dev)
            st["dweight"] = torch.zeros(T, top, device=dev)
        else:
            st["out"] = torch.empty(T, d, dtype=_DT[case["out"]], device=dev)
    elif op == "quantize":
        T, top, k = case["tokens"], case["top"], case["k"]
        st["x"] = normal(T, k, _DT[case["dtype"]], 1.0, case["pad"])
        # a few channels far larger than the rest, as activations of trained models have
        st["x"][:, torch.randint(0, k, (max(1, k // 512),), generator=host).to(dev)] *= 20
        st["source"] = torch.randperm(T * top, generator=host).to(torch.int32).to(dev) if top > 1 else None
        per = 2 if case["elem"] == "e2m1" else 1
        st["codes"] = torch.empty(T * top, _pitch(k // per, 0, 16), dtype=torch.uint8, device=dev)
        st["scale"] = torch.empty(T * top, _pitch(k // 32, 0, 16), dtype=torch.uint8, device=dev)
        st["out"] = torch.empty(T * top, k, dtype=torch.bfloat16, device=dev)
    else:
        G, rows, n, k, elem = case["groups"], case["rows"], case["n"], case["k"], case["elem"]
        counts = _counts(case, host)
        ends = torch.tensor([0] + counts).cumsum(0)
        st["ends"] = ends.tolist()
        st["offsets"] = ends.to(torch.int32).to(dev)
        width = k // 2 if elem == "e2m1" else k

        def coded(lead, std):
            # pitches of whole 16 bytes, as the quantiser above is asked for them
            q = torch.zeros(lead, _pitch(width, case["pad"], 16), dtype=torch.uint8, device=dev)
            s = torch.zeros(lead, _pitch(k // 32, case["pad"], 16), dtype=torch.uint8, device=dev)
            for at in range(0, lead, 1 << 14):
                m = min(1 << 14, lead - at)
                c, sc = _codes(torch.empty(m, k, device=dev).normal_(0.0, std, generator=gen), elem)
                q[at:at + m, :width] = c
                s[at:at + m, :k // 32] = sc
            return q, s

        st["xq"], st["xs"] = coded(rows, 1.0)
        st["wq"], st["ws"] = coded(G * n, 1.0 / math.sqrt(k))
        st["bias"] = torch.empty(G, n, device=dev).normal_(0.0, math.sqrt(0.1), generator=gen) \
            if case["epi"] != "none" else None
        st["out"] = torch.empty(rows, n, dtype=_DT[case["out"]], device=dev)
    return st


# -------------------------------------------------------------- plain forms --

def _choose(score, top, bias, groups, top_groups, group_sum):
    """Indexes of the `top` highest selection scores of each row (-1: none left), highest first, ties to the lower
    index; in 64 bits, since neighbours may lie closer than fp32 scores are exact."""
    sel = torch.where(score > -math.inf, score, torch.full_like(score, -math.inf))
    if bias is not None:
        sel = sel + bias.double()
    T, E = sel.shape
    if groups > 1:
        best = sel.view(T, groups, E // groups).sort(dim=2, descending=True).values[:, :, :group_sum]
        worth = torch.where(best[:, :, 0] > -math.inf,
                            torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2),
                            torch.full_like(best[:, :, 0], -math.inf))
        kept = worth.argsort(dim=1, descending=True, stable=True)[:, :top_groups]
        allowed = torch.zeros(T, groups, dtype=torch.bool, device=sel.device).scatter_(1, kept, True)
        sel = torch.where(allowed.repeat_interleave(E // groups, 1), sel, torch.full_like(sel, -math.inf))
    value, index = sel.sort(dim=1, descending=True, stable=True)
    value, index = value[:, :top], index[:, :top]
    return torch.where(value > -math.inf, index, torch.full_like(index, -1)).to(torch.int32)


def _scores(x, kind):
    """Scores in the type of x; -inf logits have none (0)."""
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_route(st):
    case, x = st["case"], st["logits"]
    if st["bias"] is not None or case["group_sum"] > 1:
        sel = torch.where(x.double() > -math.inf, _scores(x.double(), case["score"]),
                          torch.full((), -math.inf, dtype=torch.float64, device=st["dev"]))
    else:
        sel = x.double()  # the scores have the logits' order
    expert = _choose(sel, case["top"], st["bias"], case["groups"], case["top_groups"], case["group_sum"])
    s = _scores(x.float(), case["score"]).gather(1, expert.long().clamp_min(0)) * (expert >= 0)
    if case["renorm"]:
        total = s.sum(1, keepdim=True)
        s = s / torch.where(total > 0, total, torch.ones_like(total))
    return {"expert": expert, "weight": case["scale"] * s}


def _plain_route_grad(st):
    case, x = st["case"], st["logits"].float()
    s = _scores(x, case["score"])
    at, live = st["expert"].long().clamp_min(0), st["expert"] >= 0
    g = case["scale"] * st["dweight"] * live
    chosen = s.gather(1, at) * live
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        w = chosen / torch.where(total > 0, total, torch.ones_like(total))
        slope = w * (1 - chosen) if case["score"] == "sigmoid" else w
        d = slope * (g - (g * w).sum(1, keepdim=True))
    elif case["score"] == "sigmoid":
        d = g * chosen * (1 - chosen)
    else:
        d = g * chosen
    dx = torch.zeros_like(x).scatter_add_(1, at, d)
    if case["score"] == "softmax" and not case["renorm"]:
        dx = dx - s * d.sum(1, keepdim=True)
    return dx.to(_DT[case["dtype"]])


def _plain_rows(st):
    E = st["case"]["experts"]
    flat = st["expert"].flatten().long()
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    order = key.argsort(dim=0, stable=True)
    ends = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    at = torch.arange(flat.numel(), device=st["dev"])
    live = at < ends[-1]
    row = torch.empty_like(flat).scatter_(0, order, torch.where(live, at, torch.full_like(at, -1)))
    source = torch.where(live, order, torch.full_like(order, -1))
    return {"offsets": offsets.to(torch.int32), "row": row.view(st["expert"].shape).to(torch.int32),
            "source": source.to(torch.int32)}


def _plain_move(st):
    case, op, n = st["case"], st["case"]["op"], st["rows"]
    if op == "combine":
        live = (st["row"] >= 0)[..., None]
        y = st["y"][st["row"].long().clamp_min(0)].float()
        return (torch.where(live, y, torch.zeros_like(y)) * st["weight"][..., None]).sum(1).to(_DT[case["out"]])
    src = st["source"][:n].long()
    moved = st["x"][src // case["top"]].float() * st["weight"].flatten()[src, None]
    rest = torch.zeros(st["out"].shape[0] - n, case["d"], device=st["dev"])
    dy = torch.cat([moved, rest]).to(_DT[case["dtype"]])
    if op == "gather":
        return dy
    live = st["row"] >= 0
    y = st["y"][st["row"].long().clamp_min(0)].float()
    dw = torch.where(live[..., None], y, torch.zeros_like(y)).mul(st["x"].float()[:, None, :]).sum(2)
    return {"dy": dy, "dweight": dw}


def _plain_quantize(st):
    case, x = st["case"], st["x"]
    if st["source"] is not None:
        x = x[st["source"].long() // case["top"]]
    scale, scaled = _block_codes(x, case["elem"])
    if case["elem"] == "e4m3":
        value = scaled.to(torch.float8_e4m3fn).float()
    else:
        value = torch.tensor(_E2M1, device=st["dev"])[_e2m1_index(scaled).long()].copysign(scaled)
    e = scale.int() - 127
    return {"values": torch.ldexp(value, e[..., None]).reshape(x.shape).to(torch.bfloat16), "scale": scale}


def _values(codes, scale, k, elem):
    """The rows that codes and scales stand for, in fp32 (exact)."""
    if elem == "e4m3":
        v = codes[:, :k].contiguous().view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
        c = codes[:, :k // 2].int()
        v = torch.stack([table[c % 16], table[c // 16]], 2)
    e = scale[:, :k // 32].int() - 127
    return torch.ldexp(v.reshape(codes.shape[0], k // 32, 32), e[..., None]).reshape(codes.shape[0], k)


def _act(z, epi):
    if epi == "bias_silu":
        return z / (1 + torch.exp(-z))
    if epi == "bias_gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return z


def _plain_product(st):
    case = st["case"]
    n, k, elem = case["n"], case["k"], case["elem"]
    x = _values(st["xq"], st["xs"], k, elem)
    parts = []
    for e, (r0, r1) in enumerate(zip(st["ends"], st["ends"][1:])):  # ragged sizes: one product for each expert
        if r0 == r1:
            continue
        z = x[r0:r1] @ _values(st["wq"][e * n:(e + 1) * n], st["ws"][e * n:(e + 1) * n], k, elem).t()
        if st["bias"] is not None:
            z = z + st["bias"][e]
        parts.append(_act(z, case["epi"]).to(_DT[case["out"]]))
    return torch.cat(parts)


def _plain(st):
    op = st["case"]["op"]
    if op == "route":
        return _plain_route(st)
    if op == "route_grad":
        return _plain_route_grad(st)
    if op == "rows":
        return _plain_rows(st)
    if op == "quantize":
        return _plain_quantize(st)
    if op == "product":
        return _plain_product(st)
    return _plain_move(st)


# ------------------------------------------------------- the library's calls --

def _library(st):
    import dense_gemm_epilogues_tcgen05_gb300 as g
    code = {"f32": g.F32, "f16": g.F16, "bf16": g.BF16}
    elems = {"e2m1": g.MX_E2M1, "e4m3": g.MX_E4M3}
    scores = {"softmax": g.SCORE_SOFTMAX, "sigmoid": g.SCORE_SIGMOID}
    epi = {"none": g.EPI_NONE, "bias": g.EPI_BIAS, "bias_silu": g.EPI_BIAS_SILU, "bias_gelu": g.EPI_BIAS_GELU}
    case = st["case"]
    op = case["op"]
    if op == "route":
        T, E = case["tokens"], case["experts"]
        g.gemm_route(T, E, case["top"], code[case["dtype"]], st["logits"], E, st["expert"], st["weight"], st["bias"],
                     scores[case["score"]], case["groups"], case["top_groups"], case["group_sum"], case["renorm"],
                     case["scale"])
        return {"expert": st["expert"], "weight": st["weight"]}
    if op == "route_grad":
        T, E = case["tokens"], case["experts"]
        g.gemm_route_grad(T, E, case["top"], code[case["dtype"]], st["logits"], E, st["expert"], st["dweight"],
                          st["dlogits"], E, scores[case["score"]], case["renorm"], case["scale"])
        return st["dlogits"]
    if op == "rows":
        g.gemm_route_rows(case["tokens"], case["top"], case["experts"], st["expert"], st["offsets"], st["row"],
                          st["source"], st["workspace"], st["workspace"].numel())
        return {"offsets": st["offsets"], "row": st["row"], "source": st["source"]}
    if op in ("gather", "combine", "combine_grad"):
        T, top, d, n, dt = case["tokens"], case["top"], case["d"], st["rows"], code[case["dtype"]]
        if op == "combine":
            y = st["y"]
            g.gemm_rows_combine(T, top, d, T * top, dt, y, y.stride(0), st["row"], st["weight"], 0.0,
                                code[case["out"]], st["out"], d)
            return st["out"]
        x = st["x"]
        if op == "gather":
            g.gemm_rows_gather(T * top, d, T, top, dt, x, x.stride(0), st["source"], st["weight"], st["out"], d)
            return st["out"]
        y = st["y"]
        g.gemm_rows_combine_grad(T, top, d, T * top, dt, x, x.stride(0), dt, y, y.stride(0), st["row"], st["weight"],
                                 st["out"], d, st["dweight"])
        return {"dy": st["out"], "dweight": st["dweight"]}
    k, elem, per = case["k"], elems[case["elem"]], 2 if case["elem"] == "e2m1" else 1
    if op == "quantize":
        x, q, s, rows = st["x"], st["codes"], st["scale"], case["tokens"] * case["top"]
        g.gemm_mx_quantize(rows, k, elem, code[case["dtype"]], x, x.stride(0), q, q.shape[1] * per, s, s.shape[1],
                           st["source"], case["top"], case["tokens"])
        g.gemm_mx_dequantize(rows, k, elem, q, q.shape[1] * per, s, s.shape[1], g.BF16, st["out"], k)
        return {"values": st["out"], "scale": s[:, :k // 32]}
    n, xq, wq, xs, ws = case["n"], st["xq"], st["wq"], st["xs"], st["ws"]
    g.gemm_mx_grouped(case["groups"], case["rows"], n, k, elem, st["offsets"], xq, xq.shape[1] * per, xs, xs.shape[1],
                      wq, n * wq.shape[1] * per, wq.shape[1] * per, ws, n * ws.shape[1], ws.shape[1], st["out"], n,
                      code[case["out"]], 1.0, 0.0, st["bias"], epi[case["epi"]])
    return st["out"]


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------------- work --

def work(case):
    """Each input read once, each output written once; weights of experts without rows are not needed."""
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, top, es = case["tokens"], case["experts"], case["top"], _SIZE[case["dtype"]]
        if op == "route":
            return {"bytes": T * E * es + 8 * T * top + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
        # of renormalised scores, only the chosen logits are needed
        read = T * E * es if case["score"] == "softmax" and not case["renorm"] else T * top * es
        return {"bytes": read + 8 * T * top + T * E * es, "flops": 4 * T * E}
    if op == "rows":
        pairs = case["tokens"] * case["top"]
        return {"bytes": 12 * pairs + 4 * (case["experts"] + 1), "flops": pairs}
    if op in ("gather", "combine", "combine_grad"):
        T, top, d, es = case["tokens"], case["top"], case["d"], _SIZE[case["dtype"]]
        pairs = T * top
        live = max(1, int(pairs * (1 - case["dropped"])))
        if op == "gather":
            return {"bytes": (min(T, live) + live) * d * es + 4 * pairs + 4 * live, "flops": live * d}
        if op == "combine":
            return {"bytes": live * d * es + T * d * _SIZE[case["out"]] + 8 * pairs, "flops": 2 * live * d}
        return {"bytes": (T + 2 * live) * d * es + 12 * pairs, "flops": 3 * live * d}
    if op == "quantize":
        rows, k = case["tokens"] * case["top"], case["k"]
        return {"bytes": case["tokens"] * k * _SIZE[case["dtype"]] + rows * (2 * k + k // 32), "flops": 4 * rows * k}
    rows, n, k = case["rows"], case["n"], case["k"]
    busy = sum(1 for c in _counts(case) if c)
    held = (k // 2 if case["elem"] == "e2m1" else k) + k // 32
    return {"bytes": (rows + busy * n) * held + rows * n * _SIZE[case["out"]]
            + (4 * busy * n if case["epi"] != "none" else 0), "flops": 2 * rows * n * k}


# -------------------------------------------------------------- definitions --

def exact(case, seed):
    """The definitions in 64 bits."""
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("route", "route_grad"):
        x = st["logits"].to(f64)
        free = torch.isneginf(x)
        s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        s = s.masked_fill(free, 0.0)
        if op == "route":
            rank = x if st["bias"] is None and case["group_sum"] == 1 else s.masked_fill(free, -math.inf)
            expert = _choose(rank, case["top"], st["bias"], case["groups"], case["top_groups"], case["group_sum"])
        else:
            expert = st["expert"]
        hot = torch.zeros(*expert.shape, case["experts"] + 1, dtype=f64, device=st["dev"])
        hot.scatter_(2, expert.long().remainder(case["experts"] + 1)[..., None], 1.0)
        hot = hot[..., :case["experts"]]  # slot by expert; a slot without one is a row of zeros
        picked = torch.einsum("tse,te->ts", hot, s)
        total = picked.sum(1, keepdim=True).clamp_min(1e-300) if case["renorm"] else 1.0
        w = case["scale"] * picked / total
        if op == "route":
            return {"expert": None, "weight": w}
        g = st["dweight"].to(f64)
        # through the weights to the scores, then through the scores to the logits
        ds = case["scale"] * g / total
        if case["renorm"]:
            ds = ds - (g * w).sum(1, keepdim=True) / total
        ds = torch.einsum("tse,ts->te", hot, ds)
        if case["score"] == "sigmoid":
            return ds * s * (1 - s)
        return s * (ds - (ds * s).sum(1, keepdim=True))
    if op == "rows":
        return None
    if op in ("gather", "combine", "combine_grad"):
        T, top, d = case["tokens"], case["top"], case["d"]
        flat = st["row"].flatten().long()
        w = st["weight"].flatten().to(f64)
        if op == "combine":
            y = torch.zeros(T, d, dtype=f64, device=st["dev"])
            for slot in range(top):
                r, ws = flat[slot::top], w[slot::top]
                ok = r >= 0
                y[ok] += ws[ok, None] * st["y"][r[ok]].to(f64)
            return y
        moved = torch.zeros(T * top, d, dtype=f64, device=st["dev"])
        dw = torch.zeros(T * top, dtype=f64, device=st["dev"])
        for slot in range(top):
            r = flat[slot::top]
            ok = r >= 0
            x = st["x"][ok].to(f64)
            moved[r[ok]] = w[slot::top][ok, None] * x
            if op == "combine_grad":
                t = torch.nonzero(ok)[:, 0]
                dw[t * top + slot] = torch.einsum("td,td->t", x, st["y"][r[ok]].to(f64))
        return moved if op == "gather" else {"dy": moved, "dweight": dw.view(T, top)}
    if op == "quantize":
        x = st["x"].to(f64)
        if st["source"] is not None:
            x = x.index_select(0, torch.div(st["source"].long(), case["top"], rounding_mode="floor"))
        if x.numel() > 1 << 28:
            return None
        b = x.view(x.shape[0], -1, 32)
        peak = b.abs().max(2, keepdim=True).values

        def binade(t):  # log2 of a power of two may come out just below it; no other fp32 value is that near to one
            return torch.floor(torch.log2(t) + 1e-12)

        unit = torch.exp2(binade(peak.clamp_min(2.0 ** -120)) - _EMAX[case["elem"]])
        v = (b / unit).clamp(-_MOST[case["elem"]], _MOST[case["elem"]])
        # steps of the element type: 2^(exponent - fraction bits), the smallest exponent shared with the subnormals
        frac, low = (1, 0) if case["elem"] == "e2m1" else (3, -6)
        step = torch.exp2(binade(v.abs().clamp_min(2.0 ** low)) - frac)
        return {"values": (torch.round(v / step) * step * unit).view(x.shape), "scale": None}
    n, k, elem = case["n"], case["k"], case["elem"]

    def decode(q, s):
        if elem == "e4m3":
            c = q[:, :k].long()
            e, m = c.div(8, rounding_mode="floor") % 16, c % 8
            v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).to(f64)), m * 2.0 ** -9)
            v = torch.where(c >= 128, -v, v)
        else:
            c = torch.stack([q[:, :k // 2] & 15, q[:, :k // 2] >> 4], 2).view(q.shape[0], k).long()
            e, m = c.div(2, rounding_mode="floor") % 4, c % 2
            v = torch.where(e > 0, (2 + m) * torch.exp2((e - 2).to(f64)), m * 0.5)
            v = torch.where(c >= 8, -v, v)
        return v * torch.exp2(s[:, :k // 32].to(f64) - 127).repeat_interleave(32, 1)

    y = torch.empty(case["rows"], n, dtype=f64, device=st["dev"])
    for e, (r0, r1) in enumerate(zip(st["ends"], st["ends"][1:])):
        if r1 == r0:
            continue
        w = decode(st["wq"][e * n:(e + 1) * n], st["ws"][e * n:(e + 1) * n])
        z = torch.einsum("rk,nk->rn", decode(st["xq"][r0:r1], st["xs"][r0:r1]), w)
        if st["bias"] is not None:
            z = z + st["bias"][e].to(f64)
        if case["epi"] == "bias_silu":
            z = z * torch.sigmoid(z)
        elif case["epi"] == "bias_gelu":
            z = z * (0.5 * torch.special.erfc(-z * math.sqrt(0.5)))
        y[r0:r1] = z
    return y
