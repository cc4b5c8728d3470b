"""GPU: the gated block's gradients against the formula in 64 bits from end to end, dpre's rounding included.

Each value: dpre is rounded once (2^-8 of it at most), each sum is in fp32 and rounded once, so a result is off by
2^-8 |ref| and by 2^-8 sum |dpre| |w| beside what test_gpu_gated.py allows for dpre before its rounding and for the sums.
All values: a rounding is off by 2^-8 / sqrt(3) of a value at most in its root mean square (evenly spread over the step of
the binade's least value).  Those of dpre's values are independent of each other, so their squares add in a sum, and the sum's norm
is off by as much, relative to sqrt(sum dpre^2 w^2), as one rounding is; with the result's own that is 2^-8 sqrt(2 / 3) of the
norm where signs are random, as here.  A hundredth on top is for the sums and the sample."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_gpu_gated import SUM, act64, normal, products, within  # noqa: E402


@pytest.mark.parametrize("act,kept", [("silu", True), ("gelu_tanh", False)])
@pytest.mark.parametrize("M,I,K", [(2, 1024, 2048), (77, 512, 1536), (300, 1416, 456), (1023, 336, 456)])
def test_from_end_to_end(M, I, K, act, kept):
    X, W, dH = normal(M, M, K), normal(I, 2 * I, K, scale=K ** -0.5), normal(K, M, I)
    pre = None
    (g, u), (sg, su) = products(X, W)
    tg, tu = SUM * sg, SUM * su
    if kept:
        pre = torch.empty((M, 2 * I), dtype=torch.bfloat16, device="cuda")
        fg.gated_ffn(X, W, act=act, pre=pre)
        g, u = pre.double().chunk(2, dim=1)
        tg = tu = torch.zeros_like(g)
    d, x, w = dH.double(), X.double(), W.double()
    a, da = act64(g, act)
    dp = torch.cat((d * u * da, d * a), 1)
    off = torch.cat((d.abs() * (1.13 * tu + 1.2 * u.abs() * tg) + 2.0 ** -20 * (d * u).abs() * (1 + g.abs()),
                     d.abs() * (1.13 * tg) + 2.0 ** -20 * (d * g).abs()), 1)
    off += 2.0 ** -8 * (dp.abs() + off) + SUM * 1.01 * (dp.abs() + off)
    dX, dW = fg.gated_ffn_backward(dH, X, W, pre=pre, act=act)
    for got, ref, tol in ((dX, dp @ w, off @ w.abs()), (dW, dp.t() @ x, off.t() @ x.abs())):
        within(got, ref, (1 + 2.0 ** -8) * tol)
        error = float((got.double() - ref).norm() / ref.norm())
        assert error <= 1.01 * 2.0 ** -8 * np.sqrt(2 / 3), error
