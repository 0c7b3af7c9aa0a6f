"""A mixture-of-experts layer on the routing and the grouped products: serving in 16 bits, with 8-bit weights and
activations, with 4-bit block-scaled ones, and one training step with its gradients.

    python examples/moe_layer.py [--tokens 2048 --experts 32 --top 4 --d 2048 --f 1024]

Each token goes to its `top` experts (gemm_route).  Sorted by expert (gemm_route_rows), the token copies are rows of
one array, and the experts' row ranges (`offsets`) stay on the device: no copy back, no loop over experts.

    y[token] = sum over its experts e of  w[token, e] * ( act(x W1[e]^T + b1[e]) W2[e]^T )
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_epilogues_tcgen05_gb300 as g  # noqa: E402


class MoeLayer:
    """Weights W1 (E x F x D), b1 (E x F), W2 (E x D x F), router (E x D); D and F multiples of 16."""

    def __init__(self, d, f, experts, top, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std, dtype=torch.bfloat16):
            return torch.empty(*shape, device=device, dtype=dtype).normal_(0.0, std, generator=gen)

        self.d, self.f, self.experts, self.top = d, f, experts, top
        self.router = normal(experts, d, std=d ** -0.5, dtype=torch.float32)
        self.w1 = normal(experts, f, d, std=d ** -0.5)
        self.b1 = normal(experts, f, std=0.1, dtype=torch.float32)
        self.w2 = normal(experts, d, f, std=f ** -0.5)

    def choose(self, x):
        """The router's logits, each token's experts and their weights (tokens x top)."""
        T, dev = x.shape[0], x.device
        logits = x.float().contiguous() @ self.router.t()
        if self.top > g.ROUTE_MAX_TOP:  # more than gemm_route chooses
            chosen, expert = logits.topk(self.top)
            weight = torch.softmax(chosen, 1)
            return logits, expert.int().masked_fill(weight.isnan(), -1), weight
        expert = torch.empty(T, self.top, dtype=torch.int32, device=dev)
        weight = torch.empty(T, self.top, device=dev)
        g.gemm_route(T, self.experts, self.top, g.F32, logits, self.experts, expert, weight)
        return logits, expert, weight

    def sort(self, expert):
        """Offsets of the experts' rows, the row of each pair and the pair of each row."""
        T, E, dev = expert.shape[0], self.experts, expert.device
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        row, source = torch.empty_like(expert), torch.empty(expert.numel(), dtype=torch.int32, device=dev)
        need = g.gemm_route_rows_workspace_size(T, self.top, E)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        g.gemm_route_rows(T, self.top, E, expert, offsets, row, source, workspace, need)
        return offsets, row, source

    def route(self, x):
        """Offsets of the experts' rows, the token of each row and its weight, rows sorted by expert (behind the last:
        token 0, weight 0)."""
        _, expert, weight = self.choose(x)
        offsets, _, source = self.sort(expert)
        pair = source.long().clamp(min=0)
        return offsets, pair // self.top, weight.flatten()[pair] * (source >= 0)

    def gather(self, x, source):
        """The tokens' rows in the experts' order."""
        rows = torch.empty(source.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        x, pitch = pitched(x)
        g.gemm_rows_gather(rows.shape[0], x.shape[1], x.shape[0], self.top, g.BF16, x, pitch, source, None, rows,
                           rows.shape[1])
        return rows

    def combine(self, y, row, weight=None):
        """The (weighted) sum of each token's rows, fp32."""
        out = torch.empty(row.shape[0], y.shape[1], device=y.device)
        g.gemm_rows_combine(row.shape[0], self.top, y.shape[1], y.shape[0], g.BF16, y, y.shape[1], row, weight, 0.0, g.F32,
                            out, out.shape[1])
        return out

    @staticmethod
    def marked(out, logits):
        """out, NaN for tokens whose softmax is NaN (a logit that is NaN or infinity, or all -infinity): the routing
        leaves out experts without a score, and would hide it."""
        return out.masked_fill(~torch.isfinite(logits.amax(1, keepdim=True)), float("nan"))

    def _up(self, rows, offsets, epilogue):
        out = torch.empty(rows.shape[0], self.f, dtype=torch.bfloat16, device=rows.device)
        g.gemm_grouped(self.experts, rows.shape[0], self.f, self.d, g.BF16, offsets, rows, self.d, 1, self.w1,
                       self.f * self.d, 1, self.d, out, self.f, g.BF16, 1.0, 0.0, self.b1, epilogue)
        return out

    def _down(self, h, offsets, weight=None):
        out = torch.empty(h.shape[0], self.d, dtype=torch.bfloat16, device=h.device)
        g.gemm_grouped(self.experts, h.shape[0], self.d, self.f, g.BF16, offsets, h, self.f, 1, self.w2,
                       self.d * self.f, 1, self.f, out, self.d, g.BF16, 1.0, 0.0, None, g.EPI_NONE, row_scale=weight)
        return out

    def forward(self, x):
        """Serving: rows gathered, two grouped products with bias and SiLU in the first, the weighted sum."""
        logits, expert, weight = self.choose(x)
        offsets, row, source = self.sort(expert)
        y = self._down(self._up(self.gather(x, source), offsets, g.EPI_BIAS_SILU), offsets)
        return self.marked(self.combine(y, row, weight), logits)

    def quantize(self):
        """8-bit weights, a scale for each output channel."""
        self.q1, self.s1 = quantize_rows(self.w1.view(-1, self.d))
        self.q2, self.s2 = quantize_rows(self.w2.view(-1, self.f))

    def forward_i8(self, x):
        """Serving with 8-bit weights and activations: the rows are quantised before each product."""
        logits, expert, weight = self.choose(x)
        offsets, row, source = self.sort(expert)
        rows, token = source.numel(), source.long().clamp(min=0) // self.top
        qx, sx = quantize_rows(x)
        h = torch.empty(rows, self.f, dtype=torch.bfloat16, device=x.device)
        g.gemm_i8_grouped(self.experts, rows, self.f, self.d, offsets, qx[token], self.d, sx[token], self.q1,
                          self.f * self.d, self.d, self.s1, h, self.f, g.BF16, 1.0, 0.0, self.b1, g.EPI_BIAS_SILU)
        qh, sh = quantize_rows(h)
        y = torch.empty(rows, self.d, dtype=torch.bfloat16, device=x.device)
        g.gemm_i8_grouped(self.experts, rows, self.d, self.f, offsets, qh, self.f, sh, self.q2,
                          self.d * self.f, self.f, self.s2, y, self.d, g.BF16, 1.0, 0.0, None, g.EPI_NONE)
        return self.marked(self.combine(y, row, weight), logits)

    def quantize_mx(self):
        """4-bit weights, a power of two for each 32 inputs."""
        self.m1, self.ms1 = quantize_mx_rows(self.w1.view(-1, self.d))
        self.m2, self.ms2 = quantize_mx_rows(self.w2.view(-1, self.f))

    def forward_mx(self, x):
        """Serving with 4-bit block-scaled weights and activations (D and F multiples of 32): tokens are quantised as
        they are gathered."""
        logits, expert, weight = self.choose(x)
        offsets, row, source = self.sort(expert)
        rows = source.numel()
        h = torch.empty(rows, self.f, dtype=torch.bfloat16, device=x.device)
        self._mx_product(quantize_mx_rows(x, source, self.top), (self.m1, self.ms1), offsets, self.d, self.b1,
                         g.EPI_BIAS_SILU, h)
        y = torch.empty(rows, self.d, dtype=torch.bfloat16, device=x.device)
        self._mx_product(quantize_mx_rows(h), (self.m2, self.ms2), offsets, self.f, None, g.EPI_NONE, y)
        return self.marked(self.combine(y, row, weight), logits)

    def _mx_product(self, x, w, offsets, k, bias, epilogue, out):
        (qx, sx), (qw, sw), n = x, w, out.shape[1]
        g.gemm_mx_grouped(self.experts, out.shape[0], n, k, g.MX_E2M1, offsets, qx, 2 * qx.shape[1], sx, sx.shape[1], qw,
                          2 * n * qw.shape[1], 2 * qw.shape[1], sw, n * sw.shape[1], sw.shape[1], out, n, g.BF16, 1.0, 0.0,
                          bias, epilogue)

    def train_step(self, x, dy, router=False):
        """Output and the gradients of x, W1, b1 and W2 for the output's gradient dy; with `router` (top up to
        g.ROUTE_MAX_TOP) also that of the router, through the weights (the choice of experts held fixed)."""
        logits, expert, weight = self.choose(x)
        offsets, row, source = self.sort(expert)
        rows, E, T = source.numel(), self.experts, x.shape[0]
        xr = self.gather(x, source)
        z = self._up(xr, offsets, g.EPI_BIAS)  # kept for the backward pass
        sig = torch.sigmoid(z.float())
        h = (z.float() * sig).to(torch.bfloat16)
        y = self._down(h, offsets)
        out = self.marked(self.combine(y, row, weight), logits)

        dr, dw = torch.empty_like(y), torch.empty_like(weight) if router else None
        dy, pitch = pitched(dy if dy.dtype == torch.bfloat16 else dy.float())
        g.gemm_rows_combine_grad(T, self.top, self.d, rows, g.BF16 if dy.dtype == torch.bfloat16 else g.F32, dy, pitch,
                                 g.BF16, y, self.d, row, weight, dr, self.d, dw)
        dw2 = torch.empty(E, self.d, self.f, device=x.device)
        g.gemm_grouped_wgrad(E, rows, self.d, self.f, g.BF16, offsets, dr, self.d, 1, h, self.f, 1, dw2,
                             self.d * self.f, self.f, g.F32, 1.0, 0.0)
        dh = torch.empty(rows, self.f, dtype=torch.bfloat16, device=x.device)  # dr W2: the strides swapped
        g.gemm_grouped(E, rows, self.f, self.d, g.BF16, offsets, dr, self.d, 1, self.w2, self.d * self.f, self.f, 1,
                       dh, self.f, g.BF16, 1.0, 0.0, None, g.EPI_NONE)
        dz = (dh.float() * (sig * (1 + z.float() * (1 - sig)))).to(torch.bfloat16)
        dw1 = torch.empty(E, self.f, self.d, device=x.device)
        db1 = torch.empty(E, self.f, device=x.device)
        g.gemm_grouped_wgrad(E, rows, self.f, self.d, g.BF16, offsets, dz, self.f, 1, xr, self.d, 1, dw1,
                             self.f * self.d, self.d, g.F32, 1.0, 0.0, a_sum=db1)
        dxr = torch.empty(rows, self.d, dtype=torch.bfloat16, device=x.device)
        g.gemm_grouped(E, rows, self.d, self.f, g.BF16, offsets, dz, self.f, 1, self.w1, self.f * self.d, self.d, 1,
                       dxr, self.d, g.BF16, 1.0, 0.0, None, g.EPI_NONE)
        grads = {"x": self.combine(dxr, row), "w1": dw1, "b1": db1, "w2": dw2}  # a gather's gradient is the sum
        if router:
            dlogits = torch.empty_like(logits)
            g.gemm_route_grad(T, E, self.top, g.F32, logits, E, expert, dw, dlogits, E)
            grads["x"] += dlogits @ self.router
            grads["router"] = dlogits.t() @ x.float()
        return out, grads

    def reference(self, x, requires_grad=False, router=False):
        """The same layer expert by expert in plain fp32 operations, the routing among them; with gradients, its leaves
        as well (with `router`, the router's weights among them)."""
        logits = x.float().contiguous() @ self.router.t()
        expert = logits.argsort(dim=1, descending=True, stable=True)[:, :self.top]
        expert = torch.where(logits.isnan().all(1, keepdim=True), self.experts, expert)  # (no expert)
        weight = torch.softmax(logits.gather(1, expert.clamp(max=self.experts - 1)), 1).flatten()
        counts = torch.bincount(expert.flatten(), minlength=self.experts + 1).tolist()
        pair = expert.flatten().argsort(stable=True)[:sum(counts[:self.experts])]
        token, weight = pair // self.top, weight[pair]
        leaf = [t.float().requires_grad_(requires_grad) for t in (x, self.w1, self.b1, self.w2)]
        if router:
            leaf.append(self.router.clone().requires_grad_(requires_grad))
            chosen = torch.softmax((leaf[0] @ leaf[4].t()).gather(1, expert.clamp(max=self.experts - 1)), 1)
            weight = chosen.flatten()[pair]
        x, w1, b1, w2 = leaf[:4]
        parts, end = [], 0
        for e in range(self.experts):
            r = slice(end, end + counts[e])
            end += counts[e]
            h = torch.nn.functional.silu(x[token[r]] @ w1[e].t() + b1[e])
            parts.append(weight[r, None] * (h @ w2[e].t()))
        out = self.marked(torch.zeros_like(x).index_add(0, token, torch.cat(parts)), logits)
        return (out, leaf) if requires_grad else out


def pitched(x):
    """x with its rows contiguous (a copy where they are not, or overlap), and their pitch."""
    x = x if x.stride(1) == 1 and x.stride(0) >= x.shape[1] else x.contiguous()
    return x, max(x.stride(0), x.shape[1])


def quantize_rows(x):
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scale = torch.empty(x.shape[0], device=x.device)
    x, pitch = pitched(x)
    g.gemm_i8_quantize(x.shape[0], x.shape[1], g.BF16, x, pitch, q, x.shape[1], scale)
    return q, scale


def quantize_mx_rows(x, source=None, top=1):
    """4-bit codes and scales of x's rows (or of those that `source` names), pitches of whole 16 bytes."""
    rows, k = x.shape[0] if source is None else source.numel(), x.shape[1]
    codes = torch.empty(rows, (k // 2 + 15) // 16 * 16, dtype=torch.uint8, device=x.device)
    scale = torch.empty(rows, (k // 32 + 15) // 16 * 16, dtype=torch.uint8, device=x.device)
    x, pitch = pitched(x)
    g.gemm_mx_quantize(rows, k, g.MX_E2M1, g.BF16, x, pitch, codes, 2 * codes.shape[1], scale, scale.shape[1], source,
                       top, x.shape[0])
    return codes, scale


def relative(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("experts", 32), ("top", 4), ("d", 2048), ("f", 1024)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    layer = MoeLayer(a.d, a.f, a.experts, a.top)
    layer.quantize()
    blocks = a.d % 32 == 0 and a.f % 32 == 0  # what the 4-bit products take
    if blocks:
        layer.quantize_mx()
    x = torch.randn(a.tokens, a.d, device="cuda").bfloat16()
    dy = torch.randn(a.tokens, a.d, device="cuda").bfloat16()
    router = a.top <= g.ROUTE_MAX_TOP
    want, leaf = layer.reference(x, requires_grad=True, router=router)
    want.backward(dy.float())
    print(f"serving, bf16        off by {relative(layer.forward(x), want):.1e}")
    print(f"serving, 8-bit       off by {relative(layer.forward_i8(x), want):.1e}")
    if blocks:
        print(f"serving, 4-bit       off by {relative(layer.forward_mx(x), want):.1e}")
    out, grads = layer.train_step(x, dy, router)
    print(f"training, output     off by {relative(out, want):.1e}")
    for (name, grad), t in zip(grads.items(), leaf):
        print(f"training, d{name:<9} off by {relative(grad, t.grad):.1e}")
    for name, step in (("serving, bf16", lambda: layer.forward(x)), ("serving, 8-bit", lambda: layer.forward_i8(x)),
                       *([("serving, 4-bit", lambda: layer.forward_mx(x))] if blocks else []),
                       ("training step", lambda: layer.train_step(x, dy, router))):
        for _ in range(3):
            step()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(10):
            step()
        t1.record()
        torch.cuda.synchronize()
        print(f"{name:<20} {t0.elapsed_time(t1) / 10 * 1e3:.0f} us")
    if g.gemm_device_status() != g.OK:
        raise SystemExit("a kernel gave up waiting")


if __name__ == "__main__":
    main()
