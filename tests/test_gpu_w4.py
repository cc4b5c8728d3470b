"""GPU: products of few rows with 4-bit weights (dense and by expert) against a plain 64-bit
implementation.

Tolerance: products are exact in fp32 before they are summed (MXFP4) or form exact group sums up to
fp32 rounding (INT4, codes shifted by 16, so at most 5 times the terms' size); some hundred fp32
additions in a chain at most, so 2^-14 sum |x v| bounds the sum's error, and one rounding to bf16
adds 2^-8 |ref| at most.  SwiGLU: silu(g) u moves with its inputs by at most 1.1 |u| per g and |g|
per u.  Where every sum is a whole number below 2^24, results are bit-equal."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
FORMATS = [("mxfp4", 32, False), ("int4", 32, False), ("int4", 32, True), ("int4", 64, True), ("int4", 64, False),
           ("int4", 128, False), ("int4", 128, True)]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy().astype(np.float64)


def weights(rng, shape, K, fmt, group, zeros, whole=False):
    """Device tensors (W, scales, zeros) and the values they stand for."""
    q = rng.integers(0, 16, (*shape, K))
    W = dev((q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8))
    if fmt == "mxfp4":
        e = np.full((*shape, K // 32), 128) if whole else rng.integers(118, 126, (*shape, K // 32))
        return W, dev(e.astype(np.uint8)), None, E2M1[q] * np.exp2(e - 127.0).repeat(32, -1)
    s = np.full((*shape, K // group), 2.0) if whole else 0.01 + 0.02 * rng.random((*shape, K // group))
    S, s = bf16(s)
    z = rng.integers(0, 16, (*shape, K // group)) if zeros else np.full((*shape, K // group), 8)
    v = (q - z.repeat(group, -1)) * s.repeat(group, -1)
    return W, S, dev(z.astype(np.uint8)) if zeros else None, v


def close(got, ref, size):
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - ref)
    assert np.isfinite(err).all()
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * size).all(), float((err / (np.abs(ref) + size)).max())


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,N,groups", [(1, 1, 1), (1, 16, 2), (2, 17, 3), (1, 300, 5), (7, 33, 4), (15, 100, 9), (16, 64, 16),
                                        (17, 48, 6), (33, 31, 7), (70, 130, 3), (1, 4096, 28), (5, 1000, 33)])
def test_dense(M, N, groups, fmt, group, zeros):
    K = groups * group
    rng = np.random.default_rng(M * N + K)
    W, S, Z, v = weights(rng, (N,), K, fmt, group, zeros)
    X, x = bf16(rng.standard_normal((M, K)))
    close(fg.w4_gemv(X, W, S, Z), x @ v.T, np.abs(x) @ np.abs(v).T)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 512), (16, 100, 1152), (40, 20, 256)])
def test_dense_whole_numbers(M, N, K, fmt, group, zeros):
    """Every sum is a whole number below 2^24: the result is its bf16 rounding, bit for bit."""
    rng = np.random.default_rng(K)
    W, S, Z, v = weights(rng, (N,), K, fmt, group, zeros, whole=True)
    X, x = bf16(rng.integers(-3, 4, (M, K)))
    want = torch.from_numpy((x @ v.T).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(fg.w4_gemv(X, W, S, Z).cpu(), want)


def test_mxfp4_every_code_and_scale():
    """One nonzero x per row picks single weights: every code with small, ordinary and large scales."""
    K, N = 128, 64
    for lead in (7, 60, 127, 200, 240):
        q = (np.arange(N * K).reshape(N, K) * 7 + np.arange(N)[:, None]) % 16
        e = lead + np.arange(N * 4).reshape(N, 4) % 7
        W = dev((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8))
        x = np.zeros((16, K))
        at = np.arange(16) * 8 % K + np.arange(16) % 8
        x[np.arange(16), at] = np.exp2(127.0 - lead) if lead != 7 else np.exp2(100.0)
        X, x = bf16(x)
        v = E2M1[q] * np.exp2(e - 127.0).repeat(32, 1)
        want = torch.from_numpy((x @ v.T).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(fg.w4_gemv(X, W, dev(e.astype(np.uint8))).cpu(), want), lead


def test_special_values_stay_in_their_row():
    """An infinity or NaN in one row of X changes no other row, and the M > 16 rows past the end none."""
    rng = np.random.default_rng(3)
    for fmt, group, zeros in FORMATS:
        W, S, Z, v = weights(rng, (40,), 256, fmt, group, zeros)
        X, x = bf16(rng.standard_normal((5, 256)))
        base = fg.w4_gemv(X, W, S, Z)
        X[2, 9] = float("inf")
        X[4, 200] = float("nan")
        y = fg.w4_gemv(X, W, S, Z)
        for m in (0, 1, 3):
            assert torch.equal(y[m], base[m])
        assert torch.isnan(y[4]).all()
        assert not torch.isfinite(y[2]).any() or fmt == "mxfp4"


def expert_reference(x, v, ids, first, per_pair, swiglu):
    T, k = ids.shape
    E, N, _ = v.shape
    y = np.zeros((T * k, N))
    size = np.zeros((T * k, N))
    for p in range(T * k):
        e = int(ids[p // k, p % k]) - first
        if ids[p // k, p % k] >= 0 and 0 <= e < E:
            row = x[p] if per_pair else x[p // k]
            y[p], size[p] = v[e] @ row, np.abs(v[e]) @ np.abs(row)
    if not swiglu:
        return y, size
    g, u = np.split(y, 2, 1)
    sg, su = np.split(size, 2, 1)
    return g / (1 + np.exp(-g)) * u, 1.1 * np.abs(u) * sg + np.abs(g) * su + sg * su * 2.0 ** -14


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("T,k,E,N,groups,first", [(1, 1, 1, 2, 1, 0), (1, 8, 32, 66, 3, 0), (3, 2, 4, 32, 4, 1), (40, 1, 2, 34, 5, 0),
                                                  (16, 4, 9, 100, 2, 5), (2, 3, 64, 18, 9, 0)])
@pytest.mark.parametrize("swiglu,per_pair", [(False, False), (True, False), (False, True)])
def test_experts(T, k, E, N, groups, first, fmt, group, zeros, swiglu, per_pair):
    """By pair and by expert, more pairs on an expert than one tile holds, picks of other ranks."""
    K = groups * group
    rng = np.random.default_rng(T * N + K)
    W, S, Z, v = weights(rng, (E, N), K, fmt, group, zeros)
    ids = rng.integers(first, first + E, (T, k)).astype(np.int32)
    if T * k > 2:
        ids.reshape(-1)[rng.integers(0, T * k, 2)] = [-1, first + E]
    X, x = bf16(rng.standard_normal((T * k if per_pair else T, K)))
    out = torch.full((T * k, N // 2 if swiglu else N), float("nan"), dtype=torch.bfloat16, device="cuda")
    fg.w4_gemv_experts(X, W, S, dev(ids), Z, first_expert=first, swiglu=swiglu, out=out)
    ref, size = expert_reference(x, v, ids, first, per_pair and k > 1, swiglu)
    close(out, ref, size)
    there = ((ids >= first) & (ids < first + E)).reshape(-1)
    assert (out[dev(~there)] == 0).all()


def test_experts_past_one_window():
    """More pairs than one scan of the list holds (1024), few experts."""
    rng = np.random.default_rng(11)
    T, k, E, N, K = 1100, 2, 3, 20, 64
    W, S, Z, v = weights(rng, (E, N), K, "int4", 32, True)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    X, x = bf16(rng.standard_normal((T, K)))
    out = fg.w4_gemv_experts(X, W, S, dev(ids), Z)
    close(out, *expert_reference(x, v, ids, 0, False, False))


def test_the_decode_chain_in_a_graph():
    """Router, both expert layers and the combine of a decode step captured once: each replay, on new
    inputs and with eager work between, equals the eager calls."""
    rng = np.random.default_rng(12)
    T, k, E, H, I = 3, 4, 24, 256, 128
    W1, S1, _, _ = weights(rng, (E, 2 * I), H, "mxfp4", 32, False)
    W2, S2, Z2, _ = weights(rng, (E, H), I, "int4", 64, True)
    X = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), device="cuda")
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    w = torch.zeros((T, k), device="cuda")
    h = torch.zeros((T * k, I), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")

    def step():
        fg.route_topk(logits, k, score="sigmoid", ids=ids, weights=w)
        fg.w4_gemv_experts(X, W1, S1, ids, swiglu=True, out=h)
        fg.w4_gemv_experts(h, W2, S2, ids, Z2, out=y)
        fg.moe_combine(y, w, out=out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        X.normal_()
        logits.normal_()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (ids, w, h, y, out)]
        out.zero_()
        h.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (ids, w, h, y, out)):
            assert torch.equal(a, b)


def test_refusals():
    X = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((8, 64), dtype=torch.uint8, device="cuda")
    s8 = torch.full((8, 4), 127, dtype=torch.uint8, device="cuda")
    s16 = torch.ones((8, 1), dtype=torch.bfloat16, device="cuda")
    assert fg.w4_gemv(X, W, s8).shape == (2, 8) and fg.w4_gemv(X, W, s16).shape == (2, 8)
    assert fg.w4_gemv(X[:0], W, s8).shape == (0, 8)
    for bad in ((X.float(), W, s8), (X, W.to(torch.int8), s8), (X, W, s16.float())):
        with pytest.raises(TypeError):
            fg.w4_gemv(*bad)
    for bad in ((X[:, :64], W, s8), (X, W, s8[:4]), (X, W[:, :32], s8), (X, W, s16[:, :0])):
        with pytest.raises(ValueError):
            fg.w4_gemv(*bad)
    with pytest.raises(ValueError):
        fg.w4_gemv(X, W, s8, zeros=s8)
    with pytest.raises(fg.Fp8GemmError):
        fg.w4_gemv(X, W, torch.ones((8, 8), dtype=torch.bfloat16, device="cuda"))     # groups of 16
    ids = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fg.w4_gemv_experts(X[:1], W[None], s8[None], ids)
    with pytest.raises(TypeError):
        fg.w4_gemv_experts(X, W[None], s8[None], ids.long())
    with pytest.raises(ValueError):
        fg.w4_gemv_experts(X, W[None, :7], s8[None, :7], ids, swiglu=True)
