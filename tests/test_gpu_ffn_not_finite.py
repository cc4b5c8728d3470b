"""GPU: NaN in the gate of the gated block's gradients, in every kernel, against the same call without it: what it must not
reach keeps its bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_gpu_gated import normal  # noqa: E402

bf16 = torch.bfloat16


def gradients(dH, X, W, act, pre):
    dpre = torch.empty((X.shape[0], W.shape[0]), dtype=bf16, device="cuda")
    dX, dW = fg.gated_ffn_backward(dH, X, W, pre=pre, act=act, dpre=dpre)
    return dpre, dX, dW


def the_same_but(got, want, mask):
    """NaN where `mask` says, else the bits of `want`."""
    assert got[mask].isnan().all() and torch.isfinite(want).all()
    assert torch.equal(got[~mask], want[~mask])


# few rows (a kernel of their own), and tiles of each size
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("tile,M,I,K", [(None, 5, 40, 72), (None, 16, 64, 128), ("64x64", 70, 72, 136), ("128x128", 300, 136, 200),
                                        ("128x256", 300, 136, 200), ("256x256", 300, 264, 136)])
def test_nan_gate_reaches_its_gradient(tile, M, I, K, act, monkeypatch):
    """dg = dH u act'(g) and du = dH act(g) are NaN where g is, with u and dH finite: products formed again from a W with a
    NaN, or with opposite infinities, in a gate row, and products that were kept."""
    if tile:
        monkeypatch.setenv("FP8GEMM_FORCE_CONFIG", "product:%s:1" % tile)
    X, W, dH = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I)
    X[:, :2] = 1.0
    column = torch.zeros((M, 2 * I), dtype=torch.bool, device="cuda")
    column[:, [11, I + 11]] = True
    rows = column[0][:, None].expand(2 * I, K)
    dpre, dX, dW = gradients(dH, X, W, act, None)
    for values in ((float("nan"), 1.0), (float("inf"), -float("inf"))):
        bad = W.clone()
        bad[11, 0], bad[11, 1] = values
        dp, dx, dw = gradients(dH, X, bad, act, None)
        the_same_but(dp, dpre, column)
        the_same_but(dw, dW, rows)
        assert dx.isnan().any(1).all()
    # a NaN in an up row: du = dH act(g) does not have it
    bad = W.clone()
    bad[I + 11, 0] = float("nan")
    dp, _, dw = gradients(dH, X, bad, act, None)
    gate = column.clone()
    gate[:, I + 11] = False
    the_same_but(dp, dpre, gate)
    the_same_but(dw, dW, gate[0][:, None].expand(2 * I, K))
    # kept, in one row
    pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    fg.gated_ffn(X, W, act=act, pre=pre)
    dpre, dX, dW = gradients(dH, X, W, act, pre)
    pre[2, 11] = float("nan")
    dp, dx, dw = gradients(dH, X, W, act, pre)
    one = torch.zeros_like(column)
    one[2, [11, I + 11]] = True
    the_same_but(dp, dpre, one)
    the_same_but(dx, dX, one.any(1)[:, None].expand(M, K))
    the_same_but(dw, dW, rows)
