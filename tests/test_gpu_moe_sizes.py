"""GPU: the large sides of routing, token permutation and the 4-bit products: batches that take the
dispatch's four launches (also captured), its scratch past the stream's workspace, and tensors whose
offsets pass 32 bits.  Oracles and tolerances are those of the operators' own tests."""
import numpy as np
import pytest

import oracle
from test_gpu_permute import SENT, dev, pick, ranks, tokens
from test_gpu_w4 import FORMATS, bf16, close, expert_reference, weights

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402


@pytest.fixture(autouse=True)
def error_word():
    """Rows past a capacity set the device error word: it is left clear for the next test."""
    yield
    fg.read_device_error()


@pytest.mark.parametrize("T,k,G,H,M_max", [(1025, 8, 256, 256, 60), (1024, 8, 64, 128, 200), (8193, 1, 1, 128, 8200),
                                           (23000, 3, 70, 128, 2000), (1400, 6, 1024, 2176, 30), (9000, 1, 5, 16512, 4000)])
def test_dispatch_around_the_choice(T, k, G, H, M_max):
    """Both layouts at the largest batch of one launch and past it, more chunks than one scan step takes,
    rows wider than a workgroup's pass."""
    bits, X = tokens(T, H, T + G)
    ids = pick(T, k, G, seed=T)
    e, rank, count = ranks(ids, G, 0)
    co, so = oracle.quantize_1x128(bits)
    start = np.concatenate([[0], np.cumsum(-(-count // 128) * 128)])
    total = int(start[-1])
    for masked in (True, False):
        n = G * M_max if masked else total
        codes = torch.full((n, H), SENT, dtype=torch.uint8, device="cuda")
        scales = torch.full((G if masked else 1, H // 128, n // G if masked else n), float("nan"), device="cuda")
        if masked:
            _, _, where, rows = fg.moe_dispatch_masked(X, dev(ids), G, M_max, codes=codes.view(G, M_max, H), scales=scales)
            row = np.where((e >= 0) & (rank < M_max), e * M_max + rank, -1)
            assert np.array_equal(where.cpu().numpy(), np.minimum(count, M_max))
        else:
            _, _, where, rows = fg.moe_dispatch_contiguous(X, dev(ids), G, codes=codes, scales=scales[0])
            row = np.where(e >= 0, start[np.maximum(e, 0)] + rank, -1)
            want = np.full(total, -1, np.int32)
            for g in range(G):
                want[start[g]:start[g] + count[g]] = g
            assert np.array_equal(where.cpu().numpy(), want)
        assert np.array_equal(rows.cpu().numpy().reshape(-1), row)
        on = row >= 0
        want = np.full((n, H), SENT, np.uint8)
        want[row[on]] = co[np.arange(T).repeat(k)[on]]
        assert np.array_equal(codes.cpu().numpy(), want)
        want = np.full((n, H // 128), np.nan, np.float32)
        want[row[on]] = so[np.arange(T).repeat(k)[on]]
        assert np.array_equal(scales.transpose(1, 2).cpu().numpy().reshape(n, -1), want, equal_nan=True)


def test_dispatch_past_the_workspace():
    """A masked layout whose scratch does not fit the stream's workspace, and whose codes pass 4 GiB."""
    T, k, G, H, M_max = 3000, 3, 1024, 128, 36000
    bits, X = tokens(T, H, 5)
    ids = pick(T, k, G, seed=7)
    ids[:50, 0] = G - 1
    e, rank, count = ranks(ids, G, 0)
    codes = torch.full((G, M_max, H), SENT, dtype=torch.uint8, device="cuda")
    scales = torch.full((G, 1, M_max), float("nan"), device="cuda")
    _, _, mm, rows = fg.moe_dispatch_masked(X, dev(ids), G, M_max, codes=codes, scales=scales)
    row = np.where(e >= 0, e * M_max + rank, -1)
    assert row.max() * H > 1 << 32
    assert np.array_equal(mm.cpu().numpy(), count) and np.array_equal(rows.cpu().numpy().reshape(-1), row)
    co, so = oracle.quantize_1x128(bits)
    on = row >= 0
    at = dev(row[on].astype(np.int64))
    assert np.array_equal(codes.view(-1, H)[at].cpu().numpy(), co[np.arange(T).repeat(k)[on]])
    assert np.array_equal(scales.view(-1)[at].cpu().numpy(), so[np.arange(T).repeat(k)[on]][:, 0])
    codes.view(-1, H)[at] = SENT                       # nothing else was written
    scales.view(-1)[at] = float("nan")
    assert bool((codes == SENT).all()) and bool(torch.isnan(scales).all())


def test_large_dispatch_in_a_graph():
    """The four launches captured on a prepared stream: replays with other ids and eager work between them
    equal the eager calls."""
    T, k, G, H = 1200, 8, 40, 256
    _, X = tokens(T, H, 3)
    ids = dev(pick(T, k, G, 1))
    total = -(-(T * k + 127 * G) // 128) * 128
    out = [torch.zeros((total, H), dtype=torch.uint8, device="cuda"), torch.zeros((H // 128, total), device="cuda"),
           torch.zeros(total, dtype=torch.int32, device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda")]
    s = torch.cuda.Stream()
    fg.prepare_stream(s)
    torch.cuda.synchronize()

    def go():
        fg.moe_dispatch_contiguous(X, ids, G, codes=out[0], scales=out[1], m_indices=out[2], row_map=out[3])
    with torch.cuda.stream(s):
        go()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            go()
    for i in range(4):
        ids.copy_(dev(pick(T, k, G, 20 + i)))
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            go()
        s.synchronize()
        want = [t.clone() for t in out]
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_past_32_bits(score):
    """More than 2^31 logits: the last tokens' picks, weights and gradients are those of the same rows
    alone, and every token in between picks its own largest."""
    T, E, k = (1 << 23) + 5, 256, 4
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_()
    top = torch.arange(T, device="cuda") * 7 % E
    logits.scatter_(1, top[:, None], 9.0)              # above every draw of a normal variable here
    ids, w = fg.route_topk(logits, k, score=score)
    assert torch.equal(ids[:, 0].long(), top)
    dw = torch.ones((T, k), device="cuda")
    dw[:, 0] = 2.0
    dx = fg.route_topk_backward(logits, ids, dw, score=score)
    for part in (slice(0, 64), slice((1 << 23) - 40, T)):
        x = logits[part].clone()
        i2, w2 = fg.route_topk(x, k, score=score)
        assert torch.equal(ids[part], i2) and torch.equal(w[part], w2)
        assert torch.equal(dx[part], fg.route_topk_backward(x, i2, dw[part].clone(), score=score))


def test_combine_past_32_bits():
    """Rows of Y past 4 GiB, forward and backward."""
    T, k, H, R = 40, 4, 1024, 2200000
    rng = np.random.default_rng(8)
    Y = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    rows = rng.integers(0, R, T * k)
    rows[:80] = R - 1 - np.arange(80) * 7
    rows = np.unique(rows)[-T * k:]
    rows = np.concatenate([rows, np.full(T * k - len(rows), -1)]).astype(np.int32)
    rng.shuffle(rows)
    rows = rows.reshape(T, k)
    assert rows.max() == R - 1
    on = rows >= 0
    y = torch.from_numpy(rng.standard_normal((T * k, H)).astype(np.float32)).to(torch.bfloat16).view(T, k, H)
    Y[dev(rows[on].astype(np.int64))] = y[torch.from_numpy(on)].cuda()
    y = np.where(on[:, :, None], y.double().numpy(), 0.0)
    w = rng.standard_normal((T, k)).astype(np.float32)
    out = fg.moe_combine(Y, dev(w), dev(rows))
    terms = y * w[:, :, None].astype(np.float64)
    assert (np.abs(out.double().cpu().numpy() - terms.sum(1)) <=
            2.0 ** -8 * np.abs(terms.sum(1)) + 2.0 ** -22 * np.abs(terms).sum(1)).all()
    D = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    dY, dw = fg.moe_combine_backward(D.cuda(), Y, dev(w), dev(rows))
    d = D.double().numpy()
    prod = d[:, None, :] * y
    assert (np.abs(dw.double().cpu().numpy() - prod.sum(2)) <= 2.0 ** -19 * np.abs(prod).sum(2)).all()
    ref = (w[:, :, None].astype(np.float64) * d[:, None, :])[on]
    at = dev(rows[on].astype(np.int64))
    got = dY[at].double().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-37).all()
    dY[at] = 0
    assert bool((dY == 0).all())


@pytest.mark.parametrize("T,k", [(1, 4), (24, 2)])
def test_w4_experts_past_32_bits(T, k):
    """Weights of 4.8 GB: whole-number sums of the last experts' matrices, bit for bit."""
    E, N, K, group = 1152, 2048, 4096, 128
    W = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    S = torch.full((E, N, K // group), 2.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(E - 100, E, (T, k), dtype=torch.int32, device="cuda")
    ids[0] = torch.tensor([E - 1, 0, E // 2, E - 2][:k], dtype=torch.int32)
    X = torch.randint(-3, 4, (T, K), device="cuda").to(torch.bfloat16)
    y = fg.w4_gemv_experts(X, W, S, ids)
    assert W.numel() > 1 << 32
    for p in range(T * k):
        b = W[int(ids[p // k, p % k])].double()
        hi = torch.floor(b / 16)
        v = torch.stack((b - 16 * hi, hi), 2).view(N, K) - 8
        want = (2.0 * (v * X[p // k].double()).sum(1)).float().to(torch.bfloat16)
        assert torch.equal(y[p], want), p


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,N,K", [(16, 50, 4224), (13, 33, 9344), (9, 70, 8192), (4, 40, 24704), (1, 17, 70016), (21, 16, 16384),
                                   (12, 18, 6240)])
def test_w4_long_rows(M, N, K, fmt, group, zeros):
    """X in LDS by chunks: whole ones, a short last one, steps past the last pair."""
    K = K // group * group
    rng = np.random.default_rng(M * N + K)
    W, S, Z, v = weights(rng, (N,), K, fmt, group, zeros)
    X, x = bf16(rng.standard_normal((M, K)))
    close(fg.w4_gemv(X, W, S, Z), x @ v.T, np.abs(x) @ np.abs(v).T)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 24600, 256), (16, 24580, 640), (3, 131100, 128), (2, 25000, 1408)])
def test_w4_a_tile_per_wave(M, N, K, fmt, group, zeros):
    """Many short rows: waves with tiles of their own, the last one ragged."""
    rng = np.random.default_rng(M * N + K)
    W, S, Z, v = weights(rng, (N,), K, fmt, group, zeros)
    X, x = bf16(rng.standard_normal((M, K)))
    y = fg.w4_gemv(X, W, S, Z)
    assert not fg.last_config().endswith("tiles_per_wave=0")
    close(y, x @ v.T, np.abs(x) @ np.abs(v).T)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K,swiglu", [(16, 8, 8, 40, 4224, True), (12, 2, 3, 34, 9344, False), (16, 4, 40, 3000, 256, True),
                                              (8, 3, 24, 5600, 128, False), (16, 2, 4, 32, 8192, False)])
def test_w4_experts_long_and_many(T, k, E, N, K, swiglu, fmt, group, zeros):
    """Experts with X by chunks, in several passes over a crowded expert, and with tiles of a wave's own."""
    rng = np.random.default_rng(T * N + K)
    W, S, Z, v = weights(rng, (E, N), K, fmt, group, zeros)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[:, 0] = E - 1                                  # every token picks one of them
    ids[1, 0] = -1
    X, x = bf16(rng.standard_normal((T, K)))
    y = fg.w4_gemv_experts(X, W, S, dev(ids), Z, swiglu=swiglu)
    close(y, *expert_reference(x, v, ids, 0, False, swiglu))
