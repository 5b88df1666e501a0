"""A mixture-of-experts block on the library's operators: RMS norm with the
residual's addition, routing, experts with NVFP4 weights (16x16 scales) and a
dense branch with MXFP8 weights.

  decode    a few tokens: the routed matrix-vector products, activations in
            BF16 as they are;
  prefill   many tokens: the dispatch plan gathers them by expert for the
            grouped products, activations quantized to NVFP4; the norm's MXFP8
            output is the dense branch's operand;
  gradients of the router and the norm, as a training step takes them.

    python examples/moe_block.py [--tokens 4096] [--hidden 7168] [--ffn 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_block_scaled_quantize_amd as nv  # noqa: E402


class MoEBlock:
    def __init__(self, hidden, ffn, experts, top_k, groups=1, top_groups=1, seed=0, eps=1e-6):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return scale * torch.randn(*shape, generator=g, device="cuda")

        self.hidden, self.ffn, self.experts, self.top_k = hidden, ffn, experts, top_k
        self.groups, self.top_groups, self.eps = groups, top_groups, eps
        self.norm = (1.0 + normal(hidden, scale=0.1)).bfloat16()
        self.router = normal(experts, hidden, scale=hidden ** -0.5).bfloat16()
        self.bias = normal(experts, scale=0.01)  # of the balance of the experts' loads
        self.up = self._stack([normal(2 * ffn, hidden, scale=hidden ** -0.5) for _ in range(experts)])
        self.down = self._stack([normal(hidden, ffn, scale=ffn ** -0.5) for _ in range(experts)])
        self.dense = nv.nvfp4_mx_quantize(normal(hidden, hidden, scale=hidden ** -0.5))

    @staticmethod
    def _stack(weights):
        """Weights of all experts under each other, 16x16 scales, a tensor scale each."""
        q = [nv.nvfp4_quantize(w, layout=nv.NVFP4_BLK_2D) for w in weights]
        return nv.NVFP4Tensor(torch.cat([t.codes for t in q]), torch.cat([t.scales for t in q]),
                              torch.cat([t.tensor_scale for t in q]), sum(t.rows for t in q), q[0].cols,
                              nv.NVFP4_SCALE_2D)

    def route(self, y, plan):
        # (the router's product in binary32: near scores keep their order)
        logits = y.float() @ self.router.float().t()
        r = nv.nvfp4_route(logits, self.top_k, bias=self.bias, score=nv.NVFP4_ROUTE_SIGMOID, groups=self.groups,
                           top_groups=self.top_groups, plan=plan)
        return logits, r

    def decode(self, x, residual):
        """(the new residual stream, the block's output) of a few tokens."""
        n = nv.nvfp4_rmsnorm(x, self.norm, residual=residual, eps=self.eps)
        _, r = self.route(n.y, plan=False)
        a = nv.nvfp4_expert_gemv(n.y, r.ids, self.up, self.experts, epilogue=nv.NVFP4_EPI_SWIGLU)
        return n.h, nv.nvfp4_expert_gemv(a, r.ids, self.down, self.experts, weights=r.weights)

    def prefill(self, x, residual):
        """(the new residual stream, the experts' output, the dense branch's
        output) of many tokens."""
        n = nv.nvfp4_rmsnorm(x, self.norm, residual=residual, eps=self.eps, mx_elem=nv.NVFP4_MX_E4M3)
        _, r = self.route(n.y, plan=True)
        gathered = n.y[(r.order // self.top_k).long()]
        amax = torch.zeros(1, device=x.device)
        h = nv.nvfp4_grouped_gemm(nv.nvfp4_quantize(gathered), r.offsets, self.up, self.experts,
                                  epilogue=nv.NVFP4_EPI_SWIGLU, amax_out=amax)
        o = nv.nvfp4_grouped_gemm(nv.nvfp4_quantize(h, amax_in=amax), r.offsets, self.down, self.experts,
                                  out_dtype=torch.float32)
        o = o[r.position.long()].view(x.shape[0], self.top_k, self.hidden)
        moe = (o * r.weights.unsqueeze(2)).sum(dim=1).to(x.dtype)
        return n.h, moe, nv.nvfp4_mx_gemm(n.mx, self.dense, out_dtype=torch.bfloat16)

    def gradients(self, x, residual, dweights, dscores, dh):
        """Gradients of the residual stream (by way of the router's logits
        alone, plus dh), of the norm's weight and of the router's weight, from
        those of the chosen weights and of all scores."""
        n = nv.nvfp4_rmsnorm(x, self.norm, residual=residual, eps=self.eps, rstd=True)
        logits, r = self.route(n.y, plan=False)
        dlogits = nv.nvfp4_route_backward(dweights, logits, r.ids, score=nv.NVFP4_ROUTE_SIGMOID, dscores=dscores)
        drouter = dlogits.t().contiguous() @ n.y.float()
        dy = (dlogits @ self.router.float()).to(n.h.dtype)
        dx, dnorm = nv.nvfp4_rmsnorm_backward(dy, n.h, n.rstd, self.norm, dh=dh)
        return dx, dnorm, drouter


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--decode", type=int, default=4)
    p.add_argument("--hidden", type=int, default=7168)
    p.add_argument("--ffn", type=int, default=2048)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top-k", type=int, default=4)
    a = p.parse_args()
    block = MoEBlock(a.hidden, a.ffn, a.experts, a.top_k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16() for _ in range(2))

    def timed(f, n=20):
        for _ in range(3):
            f()
        s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s.record()
        for _ in range(n):
            f()
        e.record()
        torch.cuda.synchronize()
        return s.elapsed_time(e) / n * 1e3

    few = (x[:a.decode], res[:a.decode])
    h, moe, _ = block.prefill(x, res)
    dh, dmoe = block.decode(*few)
    off = ((dmoe.float() - moe[:a.decode].float()).norm() / dmoe.float().norm()).item()
    assert torch.equal(dh, h[:a.decode])
    print(f"decode of {a.decode} tokens:  {timed(lambda: block.decode(*few)):8.1f} us")
    print(f"prefill of {a.tokens} tokens: {timed(lambda: block.prefill(x, res)):8.1f} us")
    print(f"prefill (activations in NVFP4) against decode (in BF16): relative difference {off:.3f}")


if __name__ == "__main__":
    main()
