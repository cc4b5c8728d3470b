"""One MoE layer on one GPU, from token rows to token rows, in the two forms serving uses:

  prefill  router -> dispatch into the contiguous layout (FP8) -> grouped GEMM, SwiGLU + requantisation,
           grouped GEMM -> weighted combine
  decode   router -> the first 4-bit expert layer with SwiGLU -> the second -> weighted combine

    python examples/moe_layer.py [--tokens 1024] [--hidden 1024] [--inter 512] [--experts 32] [--topk 4]

Both run on random weights; the 4-bit weights are the prefill's FP8 weights rounded to MXFP4, so the two
forms agree to that rounding.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_x128_amd as fg  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantize_weights(w):
    """float32 [E,N,K] -> (E4M3 codes, scales [E,ceil(N/128),K/128] of 128x128 blocks)."""
    E, N, K = w.shape
    blocks = w.view(E, N // 128, 128, K // 128, 128)
    s = blocks.abs().amax((2, 4)).clamp_min(1e-4) / 448
    q = (blocks / s[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(E, N, K), s.contiguous()


def quantize_mxfp4(w):
    """float32 [E,N,K] -> (codes uint8 [E,N,K/2], E8M0 scales uint8 [E,N,K/32])."""
    E, N, K = w.shape
    runs = w.view(E, N, K // 32, 32)
    e = torch.ceil(torch.log2(runs.abs().amax(3).clamp_min(2.0 ** -100) / 6.0)).clamp(-120, 120)
    size = runs.abs() / torch.exp2(e)[..., None]
    table = torch.tensor(E2M1, device=w.device)
    code = torch.bucketize(size, (table[1:] + table[:-1]) / 2).to(torch.uint8) | ((runs < 0).to(torch.uint8) << 3)
    code = code.view(E, N, K)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


class MoeLayer:
    def __init__(self, hidden, inter, experts, topk, n_group=1, topk_group=1, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device=device)
        self.topk, self.experts, self.inter = topk, experts, inter
        self.route = dict(score="sigmoid", n_group=n_group, topk_group=topk_group, group_top=min(2, experts // n_group),
                          renorm=True, scale=1.0)
        self.gate = normal(experts, hidden) / hidden ** 0.5
        self.bias = normal(experts) * 0.02
        w1, w2 = normal(experts, 2 * inter, hidden) / hidden ** 0.5, normal(experts, hidden, inter) / inter ** 0.5
        self.w1, self.s1 = quantize_weights(w1)
        self.w2, self.s2 = quantize_weights(w2)
        self.w1_4, self.s1_4 = quantize_mxfp4(w1)
        self.w2_4, self.s2_4 = quantize_mxfp4(w2)

    def router(self, x):
        logits = x.float() @ self.gate.t()
        return fg.route_topk(logits, self.topk, bias=self.bias, **self.route)

    def prefill(self, x):
        ids, w = self.router(x)
        a, sa, m_indices, rows = fg.moe_dispatch_contiguous(x, ids, self.experts)
        y = fg.grouped_contiguous(a, sa, self.w1, self.s1, m_indices)
        h, sh = fg.swiglu_quantize_1x128(y)
        return fg.moe_combine(fg.grouped_contiguous(h, sh, self.w2, self.s2, m_indices), w, rows)

    def decode(self, x):
        ids, w = self.router(x)
        h = fg.w4_gemv_experts(x, self.w1_4, self.s1_4, ids, swiglu=True)
        return fg.moe_combine(fg.w4_gemv_experts(h, self.w2_4, self.s2_4, ids), w)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--inter", type=int, default=512)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--topk", type=int, default=4)
    a = p.parse_args()
    layer = MoeLayer(a.hidden, a.inter, a.experts, a.topk)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    prefill = layer.prefill(x)
    few = min(4, a.tokens)
    decode = layer.decode(x[:few].contiguous())
    off = (decode.float() - prefill[:few].float()).norm() / prefill[:few].float().norm()
    print("prefill %s, decode %s, relative difference of the two weight formats %.3f"
          % (tuple(prefill.shape), tuple(decode.shape), off.item()))


if __name__ == "__main__":
    main()
