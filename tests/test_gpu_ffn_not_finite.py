"""GPU: NaN in the gate of the gated block's gradients, and infinities in an adapter's second matrix, in every kernel.

Both are compared with the same call without such values: what they must not reach keeps its bits."""
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


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_infinite_gate(act):
    """act' of an infinite gate is its limit: dg = dH u above, zero below; du = dH act(g) is infinite above."""
    M, I, K = 5, 40, 72
    X, W, dH, pre = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I), normal(4, M, 2 * I)
    pre[2, 11], pre[3, 11] = float("inf"), -float("inf")
    dpre = gradients(dH, X, W, act, pre)[0]
    assert dpre[2, 11] == (dH[2, 11].float() * pre[2, I + 11].float()).to(bf16) and dpre[3, 11] == 0
    assert dpre[2, I + 11] == float("inf") * dH[2, 11].sign()


# by row, a few rows a workgroup, 64 rows; ranks of every kernel
@pytest.mark.parametrize("T,L,R,K,N", [(20, 4, 24, 264, 136), (40, 4, 16, 2568, 136), (40, 4, 16, 4168, 136), (70, 4, 104, 1200, 136),
                                       (40, 4, 32, 4168, 136), (40, 4, 56, 4168, 136), (1100, 4, 16, 200, 264), (1100, 4, 32, 200, 136),
                                       (700, 3, 56, 136, 136), (700, 3, 72, 136, 136), (700, 3, 128, 136, 136)])
def test_infinities_of_b(T, L, R, K, N):
    """An infinite value of B gives the infinity of the formula, with the sign of B, A x and the scale, whatever A x is:
    any value, one that bf16 holds exactly, one near the least; and NaN where A x is zero."""
    X, Y = normal(T, T, K), normal(T + 1, T, N)
    A, B = normal(T + 2, L, R, K, scale=K ** -0.5), normal(T + 3, L, N, R, scale=R ** -0.5)
    ids = (torch.arange(T, device="cuda") % 3).int()
    ids[[2, 4, 7, 10]] = 1
    scales = torch.tensor([0.5, 1.5, -2.0, 1.0][:L], device="cuda")
    A[1, :, 0] = 0.5
    X[[2, 4, 7]] = 0.0
    X[2, 0], X[7, 0] = 3.0, -2.0 ** -100                        # A x of 1.5, 0 and -2^-101
    for sign in (1.0, -1.0):
        scales[1] = 1.5 * sign
        want = fg.lora_add(Y, X, A, B, ids, scales)
        n = torch.arange(N, device="cuda")
        r = n % R
        at = torch.tensor([float("inf"), -float("inf"), 0.0], device="cuda")[n % 3]
        inf = at != 0
        bad = B.clone()
        bad[1, n[inf], r[inf]] = at[inf].to(bf16)
        got = fg.lora_add(Y, X, A, bad, ids, scales)
        mine = ids == 1
        assert torch.equal(got[~mine], want[~mine]) and torch.equal(got[:, ~inf], want[:, ~inf])
        v = (X[mine].double() @ A[1].double().t())[:, r[inf]]
        sure = (v == 0) | (v.abs() > 2.0 ** -12) | (v.abs() == 2.0 ** -101)      # fp32 sums keep the sign of these
        assert sure.float().mean() > 0.99 and (v == 0).any() and (v.abs() == 2.0 ** -101).any()
        ref = v * at[inf].double() * sign                      # zero times infinity is NaN
        res = got[mine][:, inf].double()
        assert torch.equal(res[sure].isnan(), ref[sure].isnan())
        there = sure & ~ref.isnan()
        assert torch.equal(res[there], ref[there])
