"""A feed-forward block whose first layer is kept in bf16, in the two uses of such a layer:

  serve  the gated layer in one launch -> FP8 quantisation -> the shared down projection -> each request's
         low-rank adapter added to its rows
  train  the gated layer as an autograd function over the library's forward and gradients

    python examples/gated_ffn.py [--tokens 512] [--hidden 1024] [--inter 512] [--adapters 8] [--rank 16] [--steps 5]

Both run on random weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_x128_amd as fg  # noqa: E402


class GatedFfn(torch.autograd.Function):
    """act(x Wg^T) * (x Wu^T).  `keep`: the two products are kept for the gradients, else formed again."""

    @staticmethod
    def forward(ctx, x, w, act, keep):
        pre = x.new_empty((x.shape[0], w.shape[0])) if keep else None
        h = fg.gated_ffn(x, w, act=act, pre=pre)
        ctx.save_for_backward(x, w, pre)
        ctx.act = act
        return h

    @staticmethod
    def backward(ctx, dh):
        x, w, pre = ctx.saved_tensors
        dx, dw = GatedFfnGradients.apply(dh.contiguous(), x, w, pre, ctx.act, *ctx.needs_input_grad[:2])
        return dx, dw, None, None


class GatedFfnGradients(torch.autograd.Function):
    """GatedFfn's gradients, which have none of their own: differentiating them is refused, whatever requires it."""

    @staticmethod
    def forward(ctx, dh, x, w, pre, act, need_dx, need_dw):
        return fg.gated_ffn_backward(dh, x, w, pre=pre, act=act, need_dX=need_dx, need_dW=need_dw)

    @staticmethod
    def backward(ctx, *unused):
        raise RuntimeError("GatedFfn has no second derivative")


class Block:
    """hidden -> 2 x inter (bf16) -> hidden (FP8, 128x128 blocks), with low-rank adapters of the down projection."""

    def __init__(self, hidden, inter, adapters, rank, act="silu", device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device=device)
        self.act = act
        self.w1 = (normal(2 * inter, hidden) / hidden ** 0.5).to(torch.bfloat16)
        w2 = normal(hidden, inter) / inter ** 0.5
        blocks = w2.view(hidden // 128, 128, inter // 128, 128)
        self.s2 = (blocks.abs().amax((1, 3)) / 448).contiguous()
        self.w2 = (blocks / self.s2[:, None, :, None]).to(torch.float8_e4m3fn).view(hidden, inter)
        self.a = (normal(adapters, rank, inter) / inter ** 0.5).to(torch.bfloat16)
        self.b = (normal(adapters, hidden, rank) / rank ** 0.5).to(torch.bfloat16)
        self.scales = torch.rand((adapters,), generator=g, device=device) + 0.5

    def serve(self, x, ids):
        """x [T, hidden] and the adapter of each row (negative: none) -> [T, hidden]."""
        h = fg.gated_ffn(x, self.w1, act=self.act)
        codes, scales = fg.quantize_1x128(h)
        y = fg.gemm_nt(codes, scales, self.w2, self.s2)
        order = ids.argsort(stable=True).int() if x.shape[0] > 64 else None
        return fg.lora_add(y, h, self.a, self.b, ids, self.scales, order=order, out=y)

    def train(self, x, target, steps, lr=0.1, keep=True):
        """Gradient steps on the gated layer alone, of the mean square between its results and `target`; the losses."""
        w = self.w1.clone().requires_grad_()
        losses = []
        for _ in range(steps):
            h = GatedFfn.apply(x, w, self.act, keep)
            loss = (h.float() - target).square().mean()
            (grad,) = torch.autograd.grad(loss, w)
            with torch.no_grad():
                w -= lr * grad
            losses.append(loss.item())
        return losses


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--inter", type=int, default=512)
    p.add_argument("--adapters", type=int, default=8)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    block = Block(a.hidden, a.inter, a.adapters, a.rank)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, a.adapters, (a.tokens,), device="cuda", dtype=torch.int32)
    y = block.serve(x, ids)
    plain = block.serve(x, torch.full_like(ids, -1))
    print("served %s, the adapters move it by %.3f of its norm" % (tuple(y.shape), ((y - plain).float().norm() / plain.float().norm()).item()))
    target = torch.randn((a.tokens, a.inter), device="cuda")
    print("losses", " ".join("%.4f" % v for v in block.train(x, target, a.steps)))


if __name__ == "__main__":
    main()
