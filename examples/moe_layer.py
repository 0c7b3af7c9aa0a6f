"""A mixture-of-experts layer on the grouped and 8-bit products: serving in 16 bits, serving with 8-bit
weights and activations, and one training step with its gradients.

    python examples/moe_layer.py [--tokens 2048 --experts 32 --top 4 --d 2048 --f 1024]

Each token goes to its `top` experts.  Sorted by expert, the token copies are rows of one array, and the
experts' row ranges (`offsets`) stay on the device: no copy back, no loop over experts.

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

    def route(self, x):
        """Offsets of the experts' rows, the token of each row and its weight, rows sorted by expert."""
        weight, expert = torch.topk(torch.softmax(x.float() @ self.router.t(), -1), self.top, sorted=False)
        weight = weight / weight.sum(-1, keepdim=True)
        flat = expert.flatten()
        order = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=self.experts)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = counts.cumsum(0)
        return offsets, order // self.top, weight.flatten()[order]

    def _up(self, rows, offsets, epilogue):
        out = torch.empty(rows.shape[0], self.f, dtype=torch.bfloat16, device=rows.device)
        g.gemm_grouped(self.experts, rows.shape[0], self.f, self.d, g.BF16, offsets, rows, self.d, 1, self.w1,
                       self.f * self.d, 1, self.d, out, self.f, g.BF16, 1.0, 0.0, self.b1, epilogue)
        return out

    def _down(self, h, offsets, weight):
        out = torch.empty(h.shape[0], self.d, dtype=torch.bfloat16, device=h.device)
        g.gemm_grouped(self.experts, h.shape[0], self.d, self.f, g.BF16, offsets, h, self.f, 1, self.w2,
                       self.d * self.f, 1, self.f, out, self.d, g.BF16, 1.0, 0.0, None, g.EPI_NONE, row_scale=weight)
        return out

    def forward(self, x):
        """Serving: two grouped products, bias and SiLU in the first, the router's weights in the second."""
        offsets, token, weight = self.route(x)
        y = self._down(self._up(x[token], offsets, g.EPI_BIAS_SILU), offsets, weight)
        return torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, y.float())

    def quantize(self):
        """8-bit weights, a scale for each output channel."""
        self.q1, self.s1 = quantize_rows(self.w1.view(-1, self.d))
        self.q2, self.s2 = quantize_rows(self.w2.view(-1, self.f))

    def forward_i8(self, x):
        """Serving with 8-bit weights and activations: the rows are quantised before each product."""
        offsets, token, weight = self.route(x)
        rows = token.shape[0]
        qx, sx = quantize_rows(x)
        h = torch.empty(rows, self.f, dtype=torch.bfloat16, device=x.device)
        g.gemm_i8_grouped(self.experts, rows, self.f, self.d, offsets, qx[token], self.d, sx[token], self.q1,
                          self.f * self.d, self.d, self.s1, h, self.f, g.BF16, 1.0, 0.0, self.b1, g.EPI_BIAS_SILU)
        qh, sh = quantize_rows(h)
        y = torch.empty(rows, self.d, dtype=torch.bfloat16, device=x.device)
        g.gemm_i8_grouped(self.experts, rows, self.d, self.f, offsets, qh, self.f, sh * weight, self.q2,
                          self.d * self.f, self.f, self.s2, y, self.d, g.BF16, 1.0, 0.0, None, g.EPI_NONE)
        return torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, y.float())

    def train_step(self, x, dy):
        """Output and the gradients of x, W1, b1 and W2 for the output's gradient dy (the routing held fixed)."""
        offsets, token, weight = self.route(x)
        rows, E = token.shape[0], self.experts
        xr = x[token]
        z = self._up(xr, offsets, g.EPI_BIAS)  # kept for the backward pass
        sig = torch.sigmoid(z.float())
        h = (z.float() * sig).to(torch.bfloat16)
        y = self._down(h, offsets, weight)
        out = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, y.float())

        dr = (dy[token].float() * weight[:, None]).to(torch.bfloat16)
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
        dx = torch.zeros_like(x, dtype=torch.float32).index_add_(0, token, dxr.float())
        return out, {"x": dx, "w1": dw1, "b1": db1, "w2": dw2}

    def reference(self, x, requires_grad=False):
        """The same layer expert by expert in plain fp32 operations; with gradients, its leaves as well."""
        offsets, token, weight = self.route(x)
        leaf = [t.float().requires_grad_(requires_grad) for t in (x, self.w1, self.b1, self.w2)]
        x, w1, b1, w2 = leaf
        ends, parts = offsets.tolist(), []
        for e in range(self.experts):
            r = slice(ends[e], ends[e + 1])
            h = torch.nn.functional.silu(x[token[r]] @ w1[e].t() + b1[e])
            parts.append(weight[r, None] * (h @ w2[e].t()))
        out = torch.zeros_like(x).index_add(0, token, torch.cat(parts))
        return (out, leaf) if requires_grad else out


def quantize_rows(x):
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scale = torch.empty(x.shape[0], device=x.device)
    g.gemm_i8_quantize(x.shape[0], x.shape[1], g.BF16, x, x.shape[1], q, x.shape[1], scale)
    return q, scale


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
    x = torch.randn(a.tokens, a.d, device="cuda").bfloat16()
    dy = torch.randn(a.tokens, a.d, device="cuda").bfloat16()
    want, leaf = layer.reference(x, requires_grad=True)
    want.backward(dy.float())
    print(f"serving, bf16        off by {relative(layer.forward(x), want):.1e}")
    print(f"serving, 8-bit       off by {relative(layer.forward_i8(x), want):.1e}")
    out, grads = layer.train_step(x, dy)
    print(f"training, output     off by {relative(out, want):.1e}")
    for (name, grad), t in zip(grads.items(), leaf):
        print(f"training, d{name:<9} off by {relative(grad, t.grad):.1e}")
    for name, step in (("serving, bf16", lambda: layer.forward(x)), ("serving, 8-bit", lambda: layer.forward_i8(x)),
                       ("training step", lambda: layer.train_step(x, dy))):
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
