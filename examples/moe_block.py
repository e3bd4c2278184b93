"""A mixture-of-experts block with its experts in 8-bit integers or in NVFP4, on the library's entry points.

    python examples/moe_block.py            # a token, a ragged batch and a prompt, against the plain form

One block is: the norm before it (fused with the previous block's output norm, gate and residual scale), the
router's logits (a plain matrix product), nvfp4_moe_route with its plan, the experts' two products with their
rows read through the plan, and nvfp4_moe_combine.  `train_step` runs the same block's router, sum and norms
forward and backward, with the experts' products as fixed linear maps.  `finetune_step` trains low-rank adapters beside the
experts' frozen 8-bit products, and the router with its balance loss, and clips their gradients.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_bit_block_quantize_amd as nv  # noqa: E402


class MoEBlock:
    """Random weights of one block: d channels, `experts` experts of `hidden` units, `top_k` a token."""

    def __init__(self, d=1024, hidden=512, experts=16, top_k=4, groups=4, group_top_k=2, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std: torch.randn(*s, generator=g, device=device) * std
        self.d, self.hidden, self.experts, self.top_k = d, hidden, experts, top_k
        self.groups, self.group_top_k, self.alpha, self.scale = groups, group_top_k, 0.5, 2.5
        self.w_post, self.w_pre, self.gate = 1 + r(d, std=0.1), 1 + r(d, std=0.1), 0.5 + r(d, std=0.1)
        self.router = r(experts, d, std=d ** -0.5).to(torch.bfloat16)
        self.bias = r(experts, std=0.01)
        self.up = r(experts * 2 * hidden, d, std=d ** -0.5).to(torch.bfloat16)      # gate and up rows of each expert
        self.down = r(experts * d, hidden, std=hidden ** -0.5).to(torch.bfloat16)
        # laid out once: 8-bit rows for the integer products, 16 x 16 tiles for the NVFP4 ones
        q, s = (nv.nvfp4_int8_quantize(w) for w in (self.up, self.down))
        self.up8 = nv.Int8Tensor(q.data, q.scales, 2 * hidden, d, experts)
        self.down8 = nv.Int8Tensor(s.data, s.scales, d, hidden, experts)
        self.up4 = nv.nvfp4_quantize_grouped(self.up.view(experts, 2 * hidden, d), flags=nv.NVFP4_BLOCK2D)
        self.down4 = nv.nvfp4_quantize_grouped(self.down.view(experts, d, hidden), flags=nv.NVFP4_BLOCK2D)
        self.route_flags = nv.NVFP4_ROUTE_SIGMOID | nv.NVFP4_ROUTE_RENORM | nv.NVFP4_ROUTE_GROUP_SUM2

    def route(self, n):
        logits = (n @ self.router.t()).float()
        return (logits,) + nv.nvfp4_moe_route(logits, self.top_k, flags=self.route_flags, bias=self.bias,
                                              num_groups=self.groups, group_top_k=self.group_top_k, scale=self.scale)

    def experts_int8(self, n, plan):
        """The experts' rows in the plan's order: each token is quantized once and read through the plan."""
        h = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(n), self.up8, plan=plan, gather=True)
        a, b = h.split(self.hidden, dim=1)
        h = torch.nn.functional.silu(a) * b
        return nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(h), self.down8, plan=plan)

    def experts_nvfp4(self, n, plan):
        """The same on the NVFP4 products, which take gathered rows and the experts' offsets on the host."""
        offsets = plan.offsets.tolist()
        rows = offsets[-1]
        h = nv.nvfp4_moe_gather(n, plan)[:rows]
        h = nv.nvfp4_gemm(nv.nvfp4_quantize(h), self.up4, group_offsets=offsets)
        a, b = h.split(self.hidden, dim=1)
        h = torch.nn.functional.silu(a) * b
        out = torch.empty((plan.rows.shape[0], self.d), dtype=n.dtype, device=n.device)
        nv.nvfp4_gemm(nv.nvfp4_quantize(h), self.down4, group_offsets=offsets, out=out[:rows])
        return out

    def forward(self, x, y, nvfp4=False):
        """x: the residual stream; y: the previous block's output.  Returns (x after y, this block's output)."""
        f = nv.nvfp4_block_norm(x, y, w_post=self.w_post, gate=self.gate, w_pre=self.w_pre, alpha=self.alpha)
        _, _, weights, plan = self.route(f.n)
        rows = (self.experts_nvfp4 if nvfp4 else self.experts_int8)(f.n, plan)
        return f.x, nv.nvfp4_moe_combine(rows, plan, weights)

    def train_step(self, x, y, rows_of, rows_grad, dout):
        """Gradients of sum(out * dout) for the norms, the gate and the router, through experts given as a map
        of their gathered rows and the plan (rows_of) and its gradient (rows_grad)."""
        f = nv.nvfp4_block_norm(x, y, w_post=self.w_post, gate=self.gate, w_pre=self.w_pre, alpha=self.alpha)
        logits, ids, weights, plan = self.route(f.n)
        rows = rows_of(nv.nvfp4_moe_gather(f.n, plan), plan)
        out = nv.nvfp4_moe_combine(rows, plan, weights)
        drows, dweights = nv.nvfp4_moe_combine_backward(dout, rows, plan, weights)
        dn = nv.nvfp4_moe_combine(rows_grad(drows, plan), plan)  # the gather's gradient: the sum over a token's slots
        dlogits = nv.nvfp4_moe_route_backward(logits, ids, dweights, flags=self.route_flags, scale=self.scale)
        drouter = dlogits.t() @ f.n.float()
        dn = (dn.float() + dlogits @ self.router.float()).to(f.n.dtype)
        grads = nv.nvfp4_block_norm_backward(None, dn, x, y, f.rstd_post, f.rstd_pre, w_post=self.w_post, gate=self.gate,
                                             w_pre=self.w_pre, alpha=self.alpha)
        return out, grads, drouter, (ids, dn)

    def add_adapters(self, rank=16, seed=1):
        """An adapter for each expert's two products (of a trained one: neither factor is zero), and the products' transposes
        for the gradients of their inputs, laid out once."""
        g = torch.Generator(device=self.up.device).manual_seed(seed)
        E, d, hidden = self.experts, self.d, self.hidden

        def adapters(n, k):
            a = (torch.randn(E * rank, k, generator=g, device=self.up.device) * k ** -0.5).to(torch.bfloat16)
            b = (torch.randn(E * n, rank, generator=g, device=self.up.device) * 0.3 * rank ** -0.5).to(torch.bfloat16)
            return nv.Adapters(a, b, torch.ones(E, device=self.up.device), rank, k, n, E)

        self.up_adapters, self.down_adapters = adapters(2 * hidden, d), adapters(d, hidden)
        turned = lambda w, n: w.view(E, n, -1).transpose(1, 2).reshape(-1, n).contiguous()
        q, s = nv.nvfp4_int8_quantize(turned(self.up, 2 * hidden)), nv.nvfp4_int8_quantize(turned(self.down, d))
        self.up8_t = nv.Int8Tensor(q.data, q.scales, d, 2 * hidden, E)
        self.down8_t = nv.Int8Tensor(s.data, s.scales, hidden, d, E)

    def finetune_step(self, x, y, dout, coef=0.01, max_norm=1.0):
        """Loss sum(out * dout) + balance loss: (out, MoEBalance, gradient norm, clipped gradients of the down and up
        adapters' factors and of the router, gradients of the norms)."""
        f = nv.nvfp4_block_norm(x, y, w_post=self.w_post, gate=self.gate, w_pre=self.w_pre, alpha=self.alpha)
        logits, ids, weights, plan = self.route(f.n)
        balance = nv.nvfp4_moe_balance(logits, ids, coef, flags=self.route_flags)
        rows = nv.nvfp4_moe_gather(f.n, plan)
        u = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(rows), self.up8, plan=plan)
        u, h_up = nv.nvfp4_adapter(rows, self.up_adapters, u, plan=plan, with_h=True, out=u)
        a, b = u.float().split(self.hidden, dim=1)
        s = torch.sigmoid(a)
        z = (a * s * b).to(u.dtype)
        v = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(z), self.down8, plan=plan)
        v, h_down = nv.nvfp4_adapter(z, self.down_adapters, v, plan=plan, with_h=True, out=v)
        out = nv.nvfp4_moe_combine(v, plan, weights)

        dv, dweights = nv.nvfp4_moe_combine_backward(dout, v, plan, weights)
        dz = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(dv), self.down8_t, plan=plan)
        down = nv.nvfp4_adapter_backward(dv, z, self.down_adapters, h_down, dx_base=dz, plan=plan, dx=dz)
        dz = down.dx.float()
        du = torch.cat([dz * b * s * (1 + a * (1 - s)), dz * a * s], dim=1).to(u.dtype)
        drows = nv.nvfp4_int8_gemm(nv.nvfp4_int8_quantize(du), self.up8_t, plan=plan)
        up = nv.nvfp4_adapter_backward(du, rows, self.up_adapters, h_up, dx_base=drows, plan=plan, dx=drows)
        dn = nv.nvfp4_moe_combine(up.dx, plan)
        dlogits = nv.nvfp4_moe_route_backward(logits, ids, dweights, flags=self.route_flags, scale=self.scale)
        dlogits = nv.nvfp4_moe_balance_backward(logits, ids, balance, coef, flags=self.route_flags, dlogits=dlogits, out=dlogits)
        drouter = dlogits.t() @ f.n.float()
        dn = (dn.float() + dlogits @ self.router.float()).to(f.n.dtype)
        norms = nv.nvfp4_block_norm_backward(None, dn, x, y, f.rstd_post, f.rstd_pre, w_post=self.w_post, gate=self.gate,
                                             w_pre=self.w_pre, alpha=self.alpha)
        grads = [down.da, down.db, up.da, up.db, drouter]
        norm = nv.nvfp4_grad_clip(grads, max_norm)
        return out, balance, norm, grads, norms

    def plain(self, x, y):
        """The block in fp32 tensor operations, without any rounding of weights or activations."""
        norm = lambda v, w: v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + 1e-6) * w
        x = x.float() + self.alpha * self.gate * norm(y.float(), self.w_post)
        n = norm(x, self.w_pre)
        # (the routing is taken from the library: a near tie may fall either way)
        _, ids, weights, _ = self.route(n.to(y.dtype))
        out = torch.zeros_like(x)
        up = self.up.float().view(self.experts, 2 * self.hidden, self.d)
        down = self.down.float().view(self.experts, self.d, self.hidden)
        for e in range(self.experts):
            t, j = (ids == e).nonzero(as_tuple=True)
            a, b = (n[t] @ up[e].t()).split(self.hidden, dim=1)
            out.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(a) * b) @ down[e].t()))
        return x, out


def main():
    block = MoEBlock()
    for tokens in (1, 37, 2048):
        g = torch.Generator(device="cuda").manual_seed(tokens)
        x, y = (torch.randn(tokens, block.d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        want_x, want = block.plain(x, y)
        for name, nvfp4 in (("int8", False), ("nvfp4", True)):
            got_x, got = block.forward(x, y, nvfp4)
            err = lambda a, b: ((a.float() - b).norm() / b.norm()).item()
            print(f"{tokens:5d} tokens, experts in {name:5s}: residual off by {err(got_x, want_x):.1e}, block by {err(got, want):.1e}")


if __name__ == "__main__":
    main()
