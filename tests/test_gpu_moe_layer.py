"""GPU: the whole MoE layer of examples/moe_layer.py, router to combine, in its prefill form (FP8 grouped
products) and its decode form (4-bit products), against a plain float64 layer on the same decoded weights.

The prefill form rounds activations to E4M3 twice (relative 2^-4 of an element at most, independent, so about
2^-5.5 of a row's norm each) and bf16 in between; the decode form rounds to bf16 alone (2^-9).  So 0.08 and 0.01
of a row's norm bound them with room."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402


def plain(x, ids, w, w1, w2):
    """float64 layer on the CPU."""
    out = torch.zeros(x.shape, dtype=torch.float64)
    x = x.double().cpu()
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            g, u = (w1[e] @ x[t]).chunk(2)
            out[t] += float(w[t, j]) * (w2[e] @ (g * torch.sigmoid(g) * u))
    return out


def decoded(codes, scales):
    return (codes.double() * scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)).cpu()


def decoded4(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long().cpu()
    table = torch.tensor(moe_layer.E2M1, dtype=torch.float64)
    v = torch.cat((table, -table))[q]
    return v * torch.exp2(scales.double().cpu() - 127).repeat_interleave(32, 2)


def relative(got, ref):
    return ((got.double().cpu() - ref).norm(dim=1) / ref.norm(dim=1)).max().item()


@pytest.mark.parametrize("tokens,experts,topk,n_group,topk_group", [(1, 8, 2, 1, 1), (37, 16, 4, 4, 2), (300, 8, 2, 1, 1)])
def test_layer(tokens, experts, topk, n_group, topk_group):
    layer = moe_layer.MoeLayer(256, 128, experts, topk, n_group, topk_group, seed=tokens)
    x = torch.randn((tokens, 256), device="cuda", generator=torch.Generator("cuda").manual_seed(tokens)).to(torch.bfloat16)
    ids, w = layer.router(x)
    ref8 = plain(x, ids, w, decoded(layer.w1, layer.s1), decoded(layer.w2, layer.s2))
    assert relative(layer.prefill(x), ref8) < 0.08
    ref4 = plain(x, ids, w, decoded4(layer.w1_4, layer.s1_4), decoded4(layer.w2_4, layer.s2_4))
    assert relative(layer.decode(x), ref4) < 0.01
