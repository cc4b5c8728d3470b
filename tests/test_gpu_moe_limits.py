"""GPU: the largest batches that routing, dispatch, combine and the 4-bit products accept."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402


def test_route_of_the_most_tokens():
    T = (1 << 28) - 17
    logits = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    ids, w = fg.route_topk(logits, 1, score="sigmoid", renorm=False)
    assert bool((ids == 0).all()) and bool((w == 0.5).all())
    dx = fg.route_topk_backward(logits, ids, w, score="sigmoid", renorm=False)
    assert bool((dx == 0.125).all())
    with pytest.raises(fg.Fp8GemmError):
        fg.route_topk(torch.zeros((T + 1, 1), dtype=torch.bfloat16, device="cuda"), 1)


def test_combine_of_the_most_tokens():
    T = (1 << 24) - 1
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    Y = (rows[:, None] % 251 + torch.arange(8, device="cuda") * 0).to(torch.bfloat16)
    back = rows.flip(0)[:, None].contiguous()
    assert torch.equal(fg.moe_combine(Y, None, back), Y.flip(0))
    dY, dw = fg.moe_combine_backward(Y, Y, None, back)
    assert torch.equal(dY, Y.flip(0)) and torch.equal(dw[:, 0], 8 * Y[:, 0].float() * Y.flip(0)[:, 0].float())


def test_dispatch_of_the_most_pairs():
    T, G, H = (1 << 24) - 1024, 1024, 128
    X = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    X *= (torch.arange(T, device="cuda") % 200 + 1).to(torch.bfloat16)[:, None]
    ids = (torch.arange(T, device="cuda") * 40503 % G).to(torch.int32)[:, None].contiguous()
    codes, scales, where, rows = fg.moe_dispatch_contiguous(X, ids, G)
    flat = ids[:, 0].long()
    count = torch.bincount(flat, minlength=G)
    first = ((count + 127) // 128 * 128).cumsum(0) - (count + 127) // 128 * 128
    order = flat.sort(stable=True)
    row = torch.empty_like(flat)
    row[order.indices] = torch.arange(T, device="cuda") - (count.cumsum(0) - count)[order.values] + first[order.values]
    assert torch.equal(rows[:, 0].long(), row)
    assert torch.equal(where[row].long(), flat) and int((where >= 0).sum()) == T
    assert torch.equal(scales[0][row], X[:, 0].float() / torch.full((T,), 448.0, device="cuda"))
    assert bool((codes.view(torch.uint8)[row] == 0x7E).all())          # 448
    assert fg.read_device_error() == 0


def test_w4_of_the_most_rows():
    M, N, K = 1 << 20, 16, 32
    W = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    S = torch.ones((N, 1), dtype=torch.bfloat16, device="cuda")
    X = torch.randint(-3, 4, (M, K), device="cuda").to(torch.bfloat16)
    V = torch.stack((W & 15, W >> 4), 2).view(N, K).float() - 8
    assert torch.equal(fg.w4_gemv(X, W, S), (X.float() @ V.t()).to(torch.bfloat16))
