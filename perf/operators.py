"""Workloads of the expert-grouped and 8-bit integer products.

Five operators of a language model's linear layers, each as a user's program calls it:

* ``grouped``     y[r] = act(x[r] B[e(r)] + bias[e(r)]), rows grouped by expert, ragged group sizes that live
                  on the device.  ``dir`` "fwd" multiplies by the weights as stored (E x N x K), "dgrad" by
                  their transpose through the strides (the gradient of the rows).
* ``wgrad``       dW[e] = sum over the expert's rows of x[r]^T dy[r], and dbias[e] = sum of dy[r].
* ``i8``          y = act(xs[i] ws[j] sum_k xq[i][k] wq[j][k] + bias[j]), 8-bit integers with a scale for each
                  token and each output channel.
* ``i8_grouped``  the same, grouped by expert.
* ``quantize``    xq[i][k] = round(127 x[i][k] / max|x[i]|), xs[i] = max|x[i]| / 127.

``run`` computes them in plain fp32 torch operations, or through the library when ``own`` is true.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # One decoded token sent to 2 of 8 small experts: launch latency.
        {"name": "grouped_token", "op": "grouped", "dir": "fwd", "groups": 8, "rows": 2, "n": 1024, "k": 1024,
         "pad": 0, "dtype": "bf16", "out": "bf16", "epi": "none", "skew": 0.0},
        # A serving batch's up projection: 512 tokens to 8 of 64 experts each, skewed loads, bound by the weights.
        {"name": "grouped_serve", "op": "grouped", "dir": "fwd", "groups": 64, "rows": 4096, "n": 2048, "k": 4096,
         "pad": 0, "dtype": "f16", "out": "f16", "epi": "bias_silu", "skew": 0.7},
        # Training: the rows' gradient through the transposed weights, the largest product.
        {"name": "grouped_dgrad", "op": "grouped", "dir": "dgrad", "groups": 32, "rows": 32768, "n": 4096, "k": 4096,
         "pad": 0, "dtype": "bf16", "out": "bf16", "epi": "none", "skew": 0.5},
        # Training: the weights' gradient into fp32 main gradients.
        {"name": "wgrad_train", "op": "wgrad", "groups": 16, "rows": 16384, "n": 2048, "k": 4096, "pad": 0,
         "dtype": "bf16", "out": "f32", "skew": 0.5},
        # Few rows for many experts, some with none, odd sizes and padded rows.
        {"name": "wgrad_ragged", "op": "wgrad", "groups": 24, "rows": 777, "n": 1000, "k": 1000, "pad": 8,
         "dtype": "f16", "out": "f16", "skew": 1.5},
        # Decoding: one token against one layer.
        {"name": "i8_token", "op": "i8", "rows": 1, "n": 4096, "k": 4096, "pad": 0, "out": "bf16", "epi": "none"},
        # A decoding batch with ragged sizes.
        {"name": "i8_ragged", "op": "i8", "rows": 200, "n": 11000, "k": 4100, "pad": 12, "out": "f32",
         "epi": "bias"},
        # Filling a long prompt.
        {"name": "i8_prompt", "op": "i8", "rows": 8192, "n": 4096, "k": 4096, "pad": 0, "out": "bf16",
         "epi": "bias_gelu"},
        # Quantised experts, decoding: 16 tokens to 4 of 64 experts each.
        {"name": "i8_grouped_decode", "op": "i8_grouped", "groups": 64, "rows": 64, "n": 2048, "k": 4096, "pad": 0,
         "out": "bf16", "epi": "none", "skew": 0.7},
        # Quantised experts, filling prompts.
        {"name": "i8_grouped_prompt", "op": "i8_grouped", "groups": 32, "rows": 8192, "n": 4096, "k": 2048, "pad": 0,
         "out": "f16", "epi": "bias_silu", "skew": 0.5},
        # The activations of one decoded token.
        {"name": "quantize_token", "op": "quantize", "rows": 1, "k": 4096, "pad": 0, "dtype": "bf16"},
        # The activations of a long prompt.
        {"name": "quantize_prompt", "op": "quantize", "rows": 16384, "k": 8192, "pad": 0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over [lo, hi], log-uniform: mostly multiples of 64, sometimes any number."""
    v = _log_int(rng, lo, hi)
    return v if rng.random() < 0.3 else max(lo, v // 64 * 64)


def draw(rng):
    while True:
        op = rng.choice(["grouped", "grouped", "wgrad", "i8", "i8", "i8_grouped", "quantize"])
        case = {"op": op, "rows": _log_int(rng, 1, 32768), "k": _size(rng, 256, 8192), "pad": 8 * rng.choice([0, 0, 1])}
        if op == "quantize":
            case["dtype"] = rng.choice(["f16", "bf16"])
            if 3072 in (case["rows"], case["k"]):
                continue
            return case
        case["n"] = _size(rng, 256, 16384 if op == "i8" else 8192)
        if op in ("grouped", "wgrad", "i8_grouped"):
            case["groups"] = _log_int(rng, 1, 128)
            case["skew"] = rng.choice([0.0, 0.5, 1.0, 1.5])
        if op == "grouped":
            case["dir"] = rng.choice(["fwd", "fwd", "dgrad"])
        if op in ("grouped", "wgrad"):
            case["dtype"] = rng.choice(["f16", "bf16"])
            case["out"] = rng.choice([case["dtype"], case["dtype"], "f32"])
        else:
            case["out"] = rng.choice(["f16", "bf16", "f32"])
        if op != "wgrad":
            case["epi"] = "none" if case.get("dir") == "dgrad" else rng.choice(
                ["none", "bias", "bias_silu", "bias_gelu"])
        w = work(case)
        if 3072 in (case["rows"], case["n"], case["k"]):
            continue  # not a size of this library's workloads
        if w["flops"] <= 1.0e12 and w["bytes"] <= 2.0e9 and case.get("groups", 1) * case["n"] * case["k"] <= 6e8:
            return case


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


def _ld(k, pad, per16):
    """Row pitch: k rounded up to 16 bytes, plus `pad` 16-byte units' worth of elements."""
    return (k + per16 - 1) // per16 * per16 + (per16 if pad else 0)


def prepare(case, seed):
    dev = torch.device("cuda") if torch.cuda.is_available() else torch.device("cpu")
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": dict(case), "dev": dev}
    op = case["op"]

    def normal(rows, cols, dtype, std, pad, lead=()):
        per16 = 16 // torch.empty((), dtype=dtype).element_size()
        ld = _ld(cols, pad, per16)
        t = torch.empty(*lead, rows, ld, dtype=dtype, device=dev)
        t.normal_(0.0, std, generator=gen)
        return t[..., :cols], ld

    def integers(rows, cols, pad, lead=()):
        # what quantising normal values gives: the largest of a row at 127, a bell below it
        ld = _ld(cols, pad, 16)
        q = torch.empty(*lead, rows, ld, dtype=torch.int8, device=dev)
        for part in q.view(-1, ld).split(max(1, (1 << 26) // ld)):
            v = torch.empty(part.shape, dtype=torch.float32, device=dev).normal_(0.0, 32.0, generator=gen)
            part.copy_(v.round_().clamp_(-127, 127))
        return q[..., :cols], ld

    if op == "quantize":
        st["x"], st["ldx"] = normal(case["rows"], case["k"], _DT[case["dtype"]], 1.0, case["pad"])
        # a few channels far larger than the rest, as activations of trained models have
        hot = torch.randint(0, case["k"], (max(1, case["k"] // 512),), generator=host).to(dev)
        st["x"][:, hot] *= 20
        st["ldq"] = _ld(case["k"], 0, 16)
        st["q"] = torch.zeros(case["rows"], st["ldq"], dtype=torch.int8, device=dev)
        st["scale"] = torch.empty(case["rows"], dtype=torch.float32, device=dev)
        return st

    rows, n, k = case["rows"], case["n"], case["k"]
    if "groups" in case:
        counts = _counts(case, host)
        ends = torch.tensor([0] + counts).cumsum(0)
        st["ends"] = ends.tolist()
        st["offsets"] = ends.to(torch.int32).to(dev)
    G = case.get("groups", 1)
    if op in ("grouped", "wgrad"):
        dt = _DT[case["dtype"]]
    if op == "grouped":
        st["w"], st["ldw"] = normal(n, k, dt, 1.0 / math.sqrt(k), case["pad"], (G,))
        st["x"], st["ldx"] = normal(rows, k if case["dir"] == "fwd" else n, dt, 1.0, case["pad"])
        width = n if case["dir"] == "fwd" else k
    elif op == "wgrad":
        st["x"], st["ldx"] = normal(rows, k, dt, 1.0, case["pad"])
        st["dy"], st["ldy"] = normal(rows, n, dt, 1.0 / math.sqrt(n), case["pad"])
    else:
        lead = (G,) if op == "i8_grouped" else ()
        st["x"], st["ldx"] = integers(rows, k, case["pad"])
        st["w"], st["ldw"] = integers(n, k, case["pad"], lead)
        st["xs"] = torch.empty(rows, device=dev).uniform_(0.02, 0.06, generator=gen)
        st["ws"] = torch.empty(*lead, n, device=dev).uniform_(0.5, 1.5, generator=gen) / (32 * math.sqrt(k))
        width = n
    if op != "wgrad" and case["epi"] != "none":
        st["bias"] = torch.empty(G, width, device=dev).normal_(0.0, math.sqrt(0.1), generator=gen)
    # the buffers that a user's program keeps for the results
    if op == "wgrad":
        st["out"] = torch.empty(G, n, k, dtype=_DT[case["out"]], device=dev)
        st["dbias"] = torch.empty(G, n, dtype=torch.float32, device=dev)
    else:
        st["out"] = torch.empty(rows, width, dtype=_DT[case["out"]], device=dev)
    return st


def _act(z, epi):
    if epi == "bias_silu":
        return z / (1 + torch.exp(-z))
    if epi == "bias_gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return z


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x = st["x"].float()
        amax = x.abs().amax(1)
        scale = amax / torch.full_like(amax, 127.0)
        q = torch.round(x * 127 / torch.where(amax == 0, torch.ones_like(amax), amax)[:, None])
        return {"codes": q.to(torch.int8), "scale": scale}
    out = _DT[case["out"]]
    if op == "i8":
        z = (st["x"].float() @ st["w"].float().t()) * st["xs"][:, None] * st["ws"]
        if "bias" in st:
            z = z + st["bias"]
        return _act(z, case["epi"]).to(out)
    ends = st["ends"]
    if op == "wgrad":
        dw = torch.empty(case["groups"], case["n"], case["k"], dtype=out, device=st["dev"])
        db = torch.empty(case["groups"], case["n"], dtype=torch.float32, device=st["dev"])
        for e in range(case["groups"]):
            dy = st["dy"][ends[e]:ends[e + 1]].float()
            dw[e] = dy.t() @ st["x"][ends[e]:ends[e + 1]].float()
            db[e] = dy.sum(0)
        return {"dw": dw, "dbias": db}
    parts = []  # one product for each expert that has rows: their sizes are ragged
    for e in range(case["groups"]):
        r0, r1 = ends[e], ends[e + 1]
        if r0 == r1:
            continue
        w = st["w"][e].float()
        z = st["x"][r0:r1].float() @ (w if case.get("dir") == "dgrad" else w.t())
        if op == "i8_grouped":
            z = z * st["xs"][r0:r1, None] * st["ws"][e]
        if "bias" in st:
            z = z + st["bias"][e]
        parts.append(_act(z, case["epi"]).to(out))
    return torch.cat(parts)


def _library(st):
    import dense_gemm_epilogues_tcgen05_gb300 as g
    code = {"f32": g.F32, "f16": g.F16, "bf16": g.BF16}
    epi = {"none": g.EPI_NONE, "bias": g.EPI_BIAS, "bias_silu": g.EPI_BIAS_SILU, "bias_gelu": g.EPI_BIAS_GELU}
    case = st["case"]
    op, rows, k = case["op"], case["rows"], case["k"]
    if op == "quantize":
        g.gemm_i8_quantize(rows, k, code[case["dtype"]], st["x"], st["ldx"], st["q"], st["ldq"], st["scale"])
        return {"codes": st["q"][:, :k], "scale": st["scale"]}
    n, out, bias = case["n"], st["out"], st.get("bias")
    if op == "i8":
        g.gemm_i8(rows, n, k, st["x"], st["ldx"], st["xs"], st["w"], st["ldw"], st["ws"], out, n, code[case["out"]],
                  1.0, 0.0, bias, epi[case["epi"]])
        return out
    G = case["groups"]
    if op == "i8_grouped":
        g.gemm_i8_grouped(G, rows, n, k, st["offsets"], st["x"], st["ldx"], st["xs"], st["w"], n * st["ldw"],
                          st["ldw"], st["ws"], out, n, code[case["out"]], 1.0, 0.0, bias, epi[case["epi"]])
        return out
    dt = code[case["dtype"]]
    if op == "wgrad":
        # dW[e] (n x k) = dy^T x: the rows' dy is the first operand
        g.gemm_grouped_wgrad(G, rows, n, k, dt, st["offsets"], st["dy"], st["ldy"], 1, st["x"], st["ldx"], 1, out,
                             n * k, k, code[case["out"]], 1.0, 0.0, a_sum=st["dbias"])
        return {"dw": out, "dbias": st["dbias"]}
    if case["dir"] == "fwd":
        # B[e] = W[e]^T (k x n): element (kk, j) at j*ldw + kk
        g.gemm_grouped(G, rows, n, k, dt, st["offsets"], st["x"], st["ldx"], 1, st["w"], n * st["ldw"], 1, st["ldw"],
                       out, n, code[case["out"]], 1.0, 0.0, bias, epi[case["epi"]])
    else:
        g.gemm_grouped(G, rows, k, n, dt, st["offsets"], st["x"], st["ldx"], 1, st["w"], n * st["ldw"], st["ldw"], 1,
                       out, k, code[case["out"]], 1.0, 0.0, None, epi["none"])
    return out


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    """Each input read once, each output written once; weights of experts without rows are not needed."""
    rows, k = case["rows"], case["k"]
    op = case["op"]
    if op == "quantize":
        return {"bytes": rows * k * (_SIZE[case["dtype"]] + 1) + 4 * rows, "flops": 3 * rows * k}
    n = case["n"]
    flops = 2 * rows * n * k
    busy = sum(1 for c in _counts(case) if c) if "groups" in case else 1
    o = _SIZE[case["out"]]
    if op == "wgrad":
        return {"bytes": rows * (n + k) * _SIZE[case["dtype"]] + case["groups"] * (n * k * o + 4 * n),
                "flops": flops + rows * n}
    bias = 4 * busy if case["epi"] != "none" else 0
    if op == "grouped":
        cols = n if case["dir"] == "fwd" else k
        inner = k if case["dir"] == "fwd" else n
        return {"bytes": (rows * inner + busy * n * k) * _SIZE[case["dtype"]] + rows * cols * o + bias * cols,
                "flops": flops}
    return {"bytes": rows * k + busy * n * k + rows * n * o + 4 * rows + 4 * busy * n + bias * n, "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits, one output row block at a time."""
    st = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "quantize":
        x = st["x"].to(f64)
        peak = torch.clamp(x.abs().max(dim=1, keepdim=True).values, min=0.0)
        safe = torch.where(peak > 0, peak, torch.ones_like(peak))
        return {"codes": torch.round(127.0 * x / safe).to(torch.int8), "scale": (peak / 127.0)[:, 0]}

    def finish(z, bias):
        z = z if bias is None else z.add(bias.to(f64))
        kind = case["epi"]
        if kind == "bias_silu":
            return z * torch.sigmoid(z)
        if kind == "bias_gelu":
            return z * (0.5 * torch.special.erfc(-z * math.sqrt(0.5)))
        return z

    if op == "wgrad":
        dw = torch.zeros(case["groups"], case["n"], case["k"], dtype=f64, device=st["dev"])
        db = torch.zeros(case["groups"], case["n"], dtype=f64, device=st["dev"])
        for e, (r0, r1) in enumerate(zip(st["ends"], st["ends"][1:])):
            g64 = st["dy"][r0:r1].to(f64)
            dw[e].addmm_(g64.mT, st["x"][r0:r1].to(f64))
            db[e] += torch.einsum("rn->n", g64)
        return {"dw": dw, "dbias": db}
    spans = list(zip(st["ends"], st["ends"][1:])) if "ends" in st else [(0, case["rows"])]
    cols = case["k"] if case.get("dir") == "dgrad" else case["n"]
    y = torch.empty(case["rows"], cols, dtype=f64, device=st["dev"])
    for e, (r0, r1) in enumerate(spans):
        if r1 == r0:
            continue
        w = (st["w"][e] if "ends" in st else st["w"]).to(f64)
        x = st["x"][r0:r1].to(f64)
        z = torch.einsum("rn,nk->rk", x, w) if case.get("dir") == "dgrad" else torch.einsum("rk,nk->rn", x, w)
        if "xs" in st:
            ws = st["ws"][e] if "ends" in st else st["ws"]
            z = torch.einsum("rn,r,n->rn", z, st["xs"][r0:r1].to(f64), ws.to(f64))
        y[r0:r1] = finish(z, st["bias"][e] if "bias" in st else None)
    return y
