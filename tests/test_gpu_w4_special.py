"""GPU: INT4 products with infinite, NaN and very large X, against the definition in 64 bits: V = (q - z) s,
a group's sum of x (q - z) formed first, in fp32, then scaled.

Tolerances.  A group's sum is sum x (16 + q) - (16 + z) sum x, two sums of at most 128 terms in fp32, each
term at most 31 |x|: off by less than 2 * 128 * 2^-24 = 2^-16 of sum 31 |x| s.  An output that this does not
leave finite is formed from q - z itself: 2^-14 sum |x v| and a bf16 rounding, as in the operator's own tests."""
import numpy as np
import pytest

from test_gpu_w4 import FORMATS, bf16, close, dev, weights

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402

INT4 = [f for f in FORMATS if f[0] == "int4"]
# few rows, 32-row tiles, X by chunks with the special value in the last one, several blocks of rows, a wave per tile
SIZES = [(5, 40, 256), (16, 9000, 384), (13, 33, 9344), (40, 20, 640), (2, 24600, 256), (3, 70, 4224)]


def with_infinity(v, x, at, value):
    """The row x . V^T where x[at] is `value`: NaN if it is NaN or met by a weight of 0, else an infinity's sign."""
    met = np.sign(v[:, at]) * np.sign(value)
    return np.where(np.isnan(met) | (met == 0), np.nan, np.copysign(np.inf, met))


@pytest.mark.parametrize("fmt,group,zeros", INT4)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_infinities_follow_the_definition(M, N, K, fmt, group, zeros):
    rng = np.random.default_rng(M + K)
    W, S, Z, v = weights(rng, (N,), K, fmt, group, zeros)
    X, x = bf16(rng.standard_normal((M, K)))
    base = fg.w4_gemv(X, W, S, Z)
    row, at = M - 1, K - 5
    others = [m for m in range(M) if m != row]
    for value in (np.inf, -np.inf, np.nan):
        X[row, at] = value
        y = fg.w4_gemv(X, W, S, Z)
        assert np.array_equal(y[row].float().cpu().numpy(), with_infinity(v, x, at, value).astype(np.float32), equal_nan=True)
        assert torch.equal(y[others], base[others])


@pytest.mark.parametrize("fmt,group,zeros", INT4)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_very_large_values(M, N, K, fmt, group, zeros):
    """Rows of one sign near 1e36 with codes next to the zero points: the sums of 16 + q times them pass fp32's
    range, those of x (q - z) do not.  Rows of ordinary size beside them are what they are alone."""
    rng = np.random.default_rng(M * 3 + K)
    z = rng.integers(1, 15, (N, K // group)) if zeros else np.full((N, K // group), 8)
    q = z.repeat(group, 1) + rng.integers(-1, 2, (N, K))
    S, s = bf16(np.full((N, K // group), 2.0 ** -9))
    W = dev((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8))
    Z = dev(z.astype(np.uint8)) if zeros else None
    v = (q - z.repeat(group, 1)) * s.repeat(group, 1)
    small, _ = bf16(rng.standard_normal((M, K)))
    base = fg.w4_gemv(small, W, S, Z)
    for size in (1e36, 2.0 ** 115, 2.0 ** 114):
        big = size * (1 + 0.2 * rng.random((M, K)))
        X, x = bf16(big)
        X[0] = small[0]
        x[0] = small[0].float().cpu().numpy()
        y = fg.w4_gemv(X, W, S, Z)
        if M > 1:
            assert torch.equal(y[0], base[0])
        slack = 31 * 2.0 ** -9 * np.abs(x[1:]).sum(1, keepdims=True) * 2.0 ** -2       # 2^-16 by close's 2^-14
        close(y[1:], x[1:] @ v.T, np.abs(x[1:]) @ np.abs(v).T + (0 if size == 1e36 else slack))


@pytest.mark.parametrize("fmt,group,zeros", INT4)
def test_experts_with_infinities(fmt, group, zeros):
    """By expert, with several tokens on one and several passes over it."""
    rng = np.random.default_rng(group)
    T, k, E, N, K = 20, 2, 3, 50, 512
    W, S, Z, v = weights(rng, (E, N), K, fmt, group, zeros)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    X, x = bf16(rng.standard_normal((T, K)))
    base = fg.w4_gemv_experts(X, W, S, dev(ids), Z)
    for t in (0, 11, 19):
        X[t, 40] = float("inf")
    y = fg.w4_gemv_experts(X, W, S, dev(ids), Z)
    for p in range(T * k):
        if p // k in (0, 11, 19):
            want = with_infinity(v[ids[p // k, p % k]], x[p // k], 40, np.inf)
            assert np.array_equal(y[p].float().cpu().numpy(), want.astype(np.float32), equal_nan=True)
        else:
            assert torch.equal(y[p], base[p])


@pytest.mark.parametrize("fmt,group,zeros", INT4)
def test_codes_at_the_zero_point(fmt, group, zeros):
    """Weights that are all 0: what is left is the rounding of the two sums."""
    rng = np.random.default_rng(9)
    N, K = 60, 1024
    z = rng.integers(0, 16, (N, K // group)) if zeros else np.full((N, K // group), 8)
    q = z.repeat(group, 1)
    W = dev((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8))
    S, s = bf16(np.full((N, K // group), 0.5))
    X, x = bf16(rng.standard_normal((3, K)))
    y = fg.w4_gemv(X, W, S, dev(z.astype(np.uint8)) if zeros else None).double().cpu().numpy()
    assert (np.abs(y) <= 2.0 ** -16 * 31 * 0.5 * np.abs(x).sum(1, keepdims=True)).all()
