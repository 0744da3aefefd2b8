#!/usr/bin/env python3
"""A quantised mixture-of-experts feed-forward layer out of this library's
operators, with int8 (W8A8) or MXFP4 experts.

    python examples/moe_layer.py [--format w8a8|mxfp4] [--tokens 1,16,256,2048]
                                 [--experts 64] [--top 8] [--hidden 4096] [--ffn 2048]

The steps for T tokens, k experts each:

    h = x + residual;  n = rmsnorm(h) * weight      one kernel, int8 rows out
    routing: logits = n . router, top k, sort by expert
    gate, up = n[token] . W1[expert]                grouped product, rows gathered
    a = silu(gate) * up                             one kernel, int8 rows out
    y = a . W2[expert]                              grouped product
    out[token] = sum over its k rows of weight * y  torch

With MXFP4 experts the normalised rows and the activations go through
quantize_mxfp4 instead.  Nothing but the routing's sort runs between the
kernels, no step waits for the host, and the sizes the kernels need to know
(how many rows each expert got) stay on the GPU.

The router reads the normalised rows as the int8 codes give them, so where two
experts' logits lie close together it may choose the other one.

Run as a program it checks the layer against a plain float64 evaluation of the
same weights with the same routing, prints the error and how many choices a
float64 router would have made differently, and times it.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import precision_dense_gemm_02_amd as lp  # noqa: E402


def quantize_weights_int8(w):
    """int8 weights and one fp32 scale per output column; w: G x N x K."""
    scale = w.float().abs().amax(2) / 127
    return (w.float() / scale[..., None]).round().to(torch.int8), scale


class MoELayer:
    """Weights of one layer on the GPU; `w1` is G x 2F x H (gate over up), `w2`
    G x H x F, `router` G x H, `norm` H, in fp16 or bf16."""

    def __init__(self, w1, w2, router, norm, top, fmt="w8a8", eps=1e-6):
        self.fmt, self.top, self.eps = fmt, top, eps
        self.norm, self.router = norm, router
        self.G, self.H = router.shape
        if fmt == "w8a8":
            self.w1, self.s1 = quantize_weights_int8(w1)
            self.w2, self.s2 = quantize_weights_int8(w2)
        elif fmt == "mxfp4":
            self.w1, self.s1 = self._mx(w1)
            self.w2, self.s2 = self._mx(w2)
        else:
            raise ValueError(f"format must be w8a8 or mxfp4, not {fmt}")

    @staticmethod
    def _mx(w):
        G, N, K = w.shape
        codes, scales = lp.quantize_mxfp4(w.reshape(G * N, K))
        return codes.reshape(G, N, -1), scales.reshape(G, N, -1)

    def route(self, n):
        """Which experts each row of n goes to: (offsets, row_index, the rows
        of C that hold each token's k results, their weights)."""
        p, chosen = torch.softmax(n @ self.router.t().to(n.dtype), dim=1).topk(self.top, dim=1)
        flat = chosen.reshape(-1)
        order = flat.argsort(stable=True)
        offsets = torch.searchsorted(flat[order], torch.arange(self.G + 1, device=n.device)).to(torch.int32)
        place = torch.empty_like(order)
        place[order] = torch.arange(order.numel(), device=n.device)
        return offsets, (order // self.top).to(torch.int32), place.reshape(-1, self.top), p / p.sum(1, keepdim=True)

    def __call__(self, x, residual):
        """(the layer's output, the residual stream h), both like x: T x H."""
        t = x.dtype
        q, scale, h = lp.add_rmsnorm_quantize(x, self.norm, self.eps, residual=residual)
        n = (q * scale[:, None]).to(t)          # the router's input, and MXFP4's
        offsets, index, place, weight = self.route(n)
        if self.fmt == "w8a8":
            g = lp.gemm_i8_dequant_grouped(q, self.w1, offsets, scale, self.s1, row_index=index, out_dtype=t)
            a, a_scale = lp.silu_mul_quantize(g)
            y = lp.gemm_i8_dequant_grouped(a, self.w2, offsets, a_scale, self.s2)
        else:
            c, s = lp.quantize_mxfp4(n)
            g = lp.gemm_mxfp4_grouped(c, s, self.w1, self.s1, offsets, row_index=index, out_dtype=t)
            a, a_scale = lp.silu_mul_quantize(g)
            c, s = lp.quantize_mxfp4((a * a_scale[:, None]).to(t))
            y = lp.gemm_mxfp4_grouped(c, s, self.w2, self.s2, offsets)
        out = (y[place] * weight[..., None]).sum(1)
        return out.to(t), h

    def chosen(self, n):
        """The experts that the router takes for each row of n: T x top."""
        return torch.softmax(n @ self.router.t().to(n.dtype), dim=1).topk(self.top, dim=1).indices

    def normalised(self, x, residual):
        """(h, the normalised rows in float64, those the layer's router reads,
        which are rounded to int8 codes)."""
        h = (x.double() + residual.double()).to(x.dtype)
        d = h.double()
        n = d / torch.sqrt((d * d).mean(1, keepdim=True) + self.eps) * self.norm.double()
        q, scale, _ = lp.add_rmsnorm_quantize(x, self.norm, self.eps, residual=residual)
        return h, n, (q * scale[:, None]).to(x.dtype)

    def routing_changes(self, x, residual):
        """The share of the T x top choices that float64 would not have made:
        rounding the rows moves experts whose logits lie close together."""
        _, n, rounded = self.normalised(x, residual)
        exact = torch.zeros(len(n), self.G, dtype=torch.bool, device=n.device).scatter_(1, self.chosen(n), True)
        return 1 - exact.gather(1, self.chosen(rounded)).double().mean().item()

    def plain(self, x, residual):
        """The layer in float64 on the stored (quantised) weights, without
        rounding any activation; routed as the layer routes, so what rounding
        changes in the routing (`routing_changes`) is not in the difference."""
        h, n, rounded = self.normalised(x, residual)
        chosen = self.chosen(rounded)
        p = torch.gather(torch.softmax(n @ self.router.double().t(), dim=1), 1, chosen)
        p = p / p.sum(1, keepdim=True)
        out = torch.zeros_like(n)
        for e in range(self.G):
            token, slot = (chosen == e).nonzero(as_tuple=True)
            if not len(token):
                continue
            if self.fmt == "w8a8":
                w1 = self.w1[e].double() * self.s1[e].double()[:, None]
                w2 = self.w2[e].double() * self.s2[e].double()[:, None]
            else:
                w1 = lp.dequantize_mxfp4(self.w1[e], self.s1[e]).double()
                w2 = lp.dequantize_mxfp4(self.w2[e], self.s2[e]).double()
            gate, up = (n[token] @ w1.t()).chunk(2, 1)
            y = (gate * torch.sigmoid(gate) * up) @ w2.t()
            out.index_add_(0, token, y * p[token, slot][:, None])
        return out, h


def random_layer(G, H, F, top, fmt, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    return MoELayer(normal(G, 2 * F, H, scale=H ** -0.5), normal(G, H, F, scale=F ** -0.5), normal(G, H, scale=H ** -0.5),
                    (1 + normal(H, scale=0.1)).to(dtype), top, fmt)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--format", default="w8a8", choices=("w8a8", "mxfp4"))
    ap.add_argument("--tokens", default="1,16,256,2048")
    for name, value in (("experts", 64), ("top", 8), ("hidden", 4096), ("ffn", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    args = ap.parse_args()
    layer = random_layer(args.experts, args.hidden, args.ffn, args.top, args.format)
    for T in (int(t) for t in args.tokens.split(",")):
        x = torch.randn(T, args.hidden, device="cuda").to(torch.bfloat16)
        r = torch.randn(T, args.hidden, device="cuda").to(torch.bfloat16)
        out, _ = layer(x, r)
        ref, _ = layer.plain(x, r)
        err = ((out.double() - ref).norm() / ref.norm()).item()
        moved = layer.routing_changes(x, r)
        for _ in range(5):
            layer(x, r)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(20):
            layer(x, r)
        torch.cuda.synchronize()
        print(f"{args.format} {T} tokens: {(time.perf_counter() - t0) / 20 * 1e6:.0f} us, "
              f"error against float64 {err:.2e} with the same routing, "
              f"{100 * moved:.1f}% of the choices differ from float64's", flush=True)


if __name__ == "__main__":
    main()
