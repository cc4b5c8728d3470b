"""GPU: moving rows between token order and expert order (dispatch, combine and the combine's
gradients) against plain implementations.

Rows, counts and indices have to be equal.  The dispatched rows are the 1x128 quantiser's codes and
scales, bit for bit the oracle's.  Combine: k terms summed in fp32 and one rounding to bf16, so
|error| <= 2^-8 |ref| + 2^-22 sum |w y| (k <= 32 additions); dweights: H products over 256 threads,
|error| <= 2^-19 sum |d y| for H up to 2^14; dY: one product, one rounding."""
import numpy as np
import pytest

import oracle
import workloads as W

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

SENT = 0x7F          # an E4M3 NaN: the library never writes it


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


def tokens(T, H, seed):
    rng = np.random.default_rng(seed)
    bits = W.bf16_bits((rng.standard_normal((T, H)) * np.exp2(rng.integers(-6, 7, (T, H // 128)).repeat(128, 1)))
                       .astype(np.float32))
    return bits, dev(bits.view(np.int16)).view(torch.bfloat16)


def pick(T, k, E, seed, holes=True):
    """ids with popular and unpopular experts, repeats between tokens, and (holes) picks that are not there."""
    rng = np.random.default_rng(seed)
    like = rng.standard_normal((1, E)) + rng.standard_normal((T, E))
    ids = np.argsort(-like, axis=1)[:, :k].astype(np.int32)
    if holes and T * k > 3:
        flat = ids.reshape(-1)
        flat[rng.integers(0, T * k, max(1, T * k // 10))] = -1
        flat[rng.integers(0, T * k)] = E + 5
        flat[rng.integers(0, T * k)] = np.iinfo(np.int32).min
        flat[rng.integers(0, T * k)] = np.iinfo(np.int32).max
    return ids


def ranks(ids, G, first):
    """(local expert or -1, rank) of each pair, and the experts' counts."""
    count = np.zeros(G, np.int64)
    e = ids.astype(np.int64).reshape(-1) - first
    e[(ids.reshape(-1) < 0) | (e < 0) | (e >= G)] = -1
    rank = np.zeros_like(e)
    for p, x in enumerate(e):
        if x >= 0:
            rank[p] = count[x]
            count[x] += 1
    return e, rank, count


CASES = [(1, 1, 1, 128, 1, 0), (1, 8, 16, 256, 1, 0), (3, 2, 5, 384, 2, 1), (130, 8, 24, 256, 64, 0), (256, 8, 64, 128, 30, 3),
         (257, 8, 33, 2176, 70, 0), (700, 6, 256, 128, 12, 100), (5000, 3, 7, 128, 2000, 0), (1500, 8, 1000, 128, 40, 20),
         (400, 32, 40, 128, 500, 0)]


@pytest.mark.parametrize("T,k,G,H,M_max,first", CASES)
def test_dispatch_masked(T, k, G, H, M_max, first):
    """One launch and four, ragged and crowded experts, other ranks' experts, rows past the capacity."""
    bits, X = tokens(T, H, T + G)
    ids = pick(T, k, max(G + 2 * first, k), seed=T * k)
    e, rank, count = ranks(ids, G, first)
    codes = torch.full((G, M_max, H), SENT, dtype=torch.uint8, device="cuda")
    scales = torch.full((G, H // 128, M_max), float("nan"), device="cuda")
    fg.read_device_error()
    _, _, mm, rows = fg.moe_dispatch_masked(X, dev(ids), G, M_max, first_expert=first, codes=codes, scales=scales)
    assert np.array_equal(mm.cpu().numpy(), np.minimum(count, M_max))
    ref_rows = np.where((e >= 0) & (rank < M_max), e * M_max + rank, -1)
    assert np.array_equal(rows.cpu().numpy().reshape(-1), ref_rows)
    assert (fg.read_device_error() & fg.DEVERR_BAD_COUNT != 0) == bool((count > M_max).any())
    co, so = oracle.quantize_1x128(bits)
    want = np.full((G * M_max, H), SENT, np.uint8)
    want_s = np.full((G * M_max, H // 128), np.nan, np.float32)
    on = ref_rows >= 0
    want[ref_rows[on]] = co[np.arange(T).repeat(k)[on]]
    want_s[ref_rows[on]] = so[np.arange(T).repeat(k)[on]]
    assert np.array_equal(codes.cpu().numpy().reshape(G * M_max, H), want)
    assert np.array_equal(scales.cpu().numpy().transpose(0, 2, 1).reshape(G * M_max, -1), want_s, equal_nan=True)


@pytest.mark.parametrize("T,k,G,H,M_max,first", CASES)
def test_dispatch_contiguous(T, k, G, H, M_max, first):
    bits, X = tokens(T, H, T + G)
    ids = pick(T, k, max(G + 2 * first, k), seed=T * k)
    e, rank, count = ranks(ids, G, first)
    room = -(-(T * k + 127 * min(G, T * k)) // 128) * 128
    start = np.concatenate([[0], np.cumsum(-(-count // 128) * 128)])
    for total in (room, max(1, int(start[-1]) - 100)):      # all of it fits; the last rows do not
        codes = torch.full((total, H), SENT, dtype=torch.uint8, device="cuda")
        scales = torch.full((H // 128, total), float("nan"), device="cuda")
        fg.read_device_error()
        _, _, mi, rows = fg.moe_dispatch_contiguous(X, dev(ids), G, M_total=total, first_expert=first, codes=codes, scales=scales)
        row = np.where(e >= 0, start[np.maximum(e, 0)] + rank, -1)
        ref_rows = np.where(row < total, row, -1)
        want_mi = np.full(total, -1, np.int32)
        for g in range(G):
            want_mi[start[g]:start[g] + count[g]] = g
        assert np.array_equal(mi.cpu().numpy(), want_mi)
        assert np.array_equal(rows.cpu().numpy().reshape(-1), ref_rows)
        assert (fg.read_device_error() & fg.DEVERR_BAD_COUNT != 0) == bool((row >= total).any())
        co, so = oracle.quantize_1x128(bits)
        want = np.full((total, H), SENT, np.uint8)
        want_s = np.full((total, H // 128), np.nan, np.float32)
        on = ref_rows >= 0
        want[ref_rows[on]] = co[np.arange(T).repeat(k)[on]]
        want_s[ref_rows[on]] = so[np.arange(T).repeat(k)[on]]
        assert np.array_equal(codes.cpu().numpy(), want)
        assert np.array_equal(scales.cpu().numpy().T, want_s, equal_nan=True)


def test_dispatch_without_tokens():
    X = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    _, _, mm, rows = fg.moe_dispatch_masked(X, ids, 5, 16, masked_m=torch.full((5,), 9, dtype=torch.int32, device="cuda"))
    assert mm.tolist() == [0] * 5 and rows.shape == (0, 4)
    _, _, mi, _ = fg.moe_dispatch_contiguous(X, ids, 5, M_total=300)
    assert (mi == -1).all()


def test_dispatch_quantiser_edges():
    """Zero blocks, subnormals, signed zeros and the largest magnitudes code as the quantiser codes them."""
    x = np.zeros((4, 256), np.float32)
    x[0, :128] = -0.0
    x[1, 3] = 3e38
    x[1, 200] = -1e-40
    x[2] = np.float32(2.0) ** np.arange(-128, 128)
    x[3] = -x[2][::-1]
    bits = W.bf16_bits(x)
    X = dev(bits.view(np.int16)).view(torch.bfloat16)
    ids = dev(np.zeros((4, 1), np.int32))
    codes, scales, mm, _ = fg.moe_dispatch_masked(X, ids, 1, 4)
    a, s = fg.quantize_1x128(X)
    assert torch.equal(codes.view(torch.uint8)[0], a.view(torch.uint8)) and torch.equal(scales[0], s)
    assert mm.item() == 4


def rows_for(T, k, R, seed):
    rng = np.random.default_rng(seed)
    rows = rng.permutation(R)[:T * k].reshape(T, k).astype(np.int32)
    rows.reshape(-1)[rng.integers(0, T * k, max(1, T * k // 8))] = -1
    rows[0] = -1                                            # a token with nothing
    return rows


COMBINES = [(1, 1, 8), (1, 8, 128), (3, 5, 2056), (130, 8, 2048), (65, 32, 136), (300, 6, 7168), (33, 9, 4104)]


@pytest.mark.parametrize("T,k,H", COMBINES)
def test_combine(T, k, H):
    rng = np.random.default_rng(T + H)
    R = T * k + 7
    Y, y = bf16(rng.standard_normal((R, H)))
    w = rng.standard_normal((T, k)).astype(np.float32)
    for rows, weights in ((rows_for(T, k, R, T), w), (rows_for(T, k, R, T + 1), None), (None, w)):
        out = fg.moe_combine(Y, None if weights is None else dev(weights), None if rows is None else dev(rows))
        r = np.arange(T * k).reshape(T, k) if rows is None else rows
        terms = np.where((r >= 0)[:, :, None], y[np.maximum(r, 0)].astype(np.float64), 0.0)
        if weights is not None:
            terms = terms * weights[:, :, None].astype(np.float64)
        ref = terms.sum(1)
        err = np.abs(out.float().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * np.abs(terms).sum(1)).all()
        if rows is not None:
            assert (out[0] == 0).all()


@pytest.mark.parametrize("T,k,H", COMBINES)
def test_combine_backward(T, k, H):
    rng = np.random.default_rng(T + H)
    R = T * k + 7
    Y, y = bf16(rng.standard_normal((R, H)))
    D, d = bf16(rng.standard_normal((T, H)))
    w = rng.standard_normal((T, k)).astype(np.float32)
    rows = rows_for(T, k, R, T)
    dY = torch.full((R, H), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = fg.moe_combine_backward(D, Y, dev(w), dev(rows), dY=dY)
    on = rows >= 0
    got = dY.float().cpu().numpy()
    untouched = np.setdiff1d(np.arange(R), rows[on])
    assert (got[untouched] == 7.0).all()
    t, j = np.nonzero(on)
    ref = w[t, j].astype(np.float64)[:, None] * d[t]
    assert (np.abs(got[rows[t, j]] - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-37).all()
    prod = d[t].astype(np.float64) * y[rows[t, j]]
    gw = dw.cpu().numpy()
    assert (gw[~on] == 0).all()
    assert (np.abs(gw[t, j] - prod.sum(1)) <= 2.0 ** -19 * np.abs(prod).sum(1)).all()


def test_combine_gradient_against_differences():
    """The loss <dout, combine> is linear in Y and w, so whole-step differences are exact up to the
    bf16 rounding of combine's output (2^-8 of each output)."""
    rng = np.random.default_rng(4)
    T, k, H, R = 2, 3, 16, 9
    Y, y = bf16(rng.standard_normal((R, H)))
    D, d = bf16(rng.standard_normal((T, H)))
    w = rng.random((T, k)).astype(np.float32)
    rows = np.array([[0, 4, -1], [8, 2, 3]], np.int32)
    _, dw = fg.moe_combine_backward(D, Y, dev(w), dev(rows))

    def loss(wv):
        out = fg.moe_combine(Y, dev(wv), dev(rows)).double().cpu().numpy()
        return (out * d).sum(), 2.0 ** -8 * np.abs(out * d).sum()
    base, slack = loss(w)
    for t in range(T):
        for j in range(k):
            step = w.copy()
            step[t, j] += 1.0
            up, more = loss(step)
            assert abs((up - base) - dw[t, j].item()) <= slack + more


def test_combine_bad_rows_and_other_forms():
    rng = np.random.default_rng(6)
    Y, y = bf16(rng.standard_normal((4, 8, 64)))             # [G, M_max, H]
    rows = np.array([[0, 31], [32, 40]], np.int32)
    fg.read_device_error()
    out = fg.moe_combine(Y, None, dev(rows))
    assert fg.read_device_error() & fg.DEVERR_BAD_INDEX
    flat = y.reshape(32, 64)
    assert (out[1] == 0).all()
    assert np.allclose(out[0].float().cpu().numpy(), flat[0] + flat[31], rtol=2.0 ** -8)
    D, _ = bf16(rng.standard_normal((2, 64)))
    dY, _ = fg.moe_combine_backward(D, Y, None, dev(rows))
    assert fg.read_device_error() & fg.DEVERR_BAD_INDEX
    assert torch.equal(dY.view(32, 64)[31], D[0]) and (dY.view(32, 64)[1:31] == 0).all()
    with pytest.raises(ValueError):
        fg.moe_combine(Y)
    with pytest.raises(TypeError):
        fg.moe_combine(Y.float(), None, dev(rows))
    with pytest.raises(ValueError):
        fg.moe_combine(Y, torch.ones(3, 2, device="cuda"), dev(rows))
    # NaN in rows that no pair names stays out
    Y.view(32, 64)[5] = float("nan")
    assert torch.isfinite(fg.moe_combine(Y, None, dev(rows[:1]))).all()


def test_dispatch_combine_round_trip_on_a_captured_stream():
    """Dispatch and combine in a graph on a stream of their own: replays, with eager
    work and other ids between them, equal the eager calls."""
    T, k, G, H = 600, 4, 20, 256
    bits, X = tokens(T, H, 9)
    ids = dev(pick(T, k, G, 1))
    w = torch.rand((T, k), device="cuda")
    cap = 512
    bufs = dict(codes=torch.zeros((G, cap, H), dtype=torch.uint8, device="cuda"),
                scales=torch.zeros((G, H // 128, cap), device="cuda"),
                masked_m=torch.zeros(G, dtype=torch.int32, device="cuda"),
                row_map=torch.zeros((T, k), dtype=torch.int32, device="cuda"))
    Y = torch.randn((G, cap, H), device="cuda").to(torch.bfloat16)
    out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    fg.prepare_stream(s)
    torch.cuda.synchronize()

    def go():
        fg.moe_dispatch_masked(X, ids, G, cap, **bufs)
        fg.moe_combine(Y, w, bufs["row_map"], out=out)
    with torch.cuda.stream(s):
        go()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            go()
    for i in range(4):
        ids.copy_(dev(pick(T, k, G, 20 + i)))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            go()
        s.synchronize()
        want = [bufs["masked_m"].clone(), bufs["row_map"].clone(), out.clone()]
        bufs["row_map"].fill_(-7)
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        for a, b in zip(want, (bufs["masked_m"], bufs["row_map"], out)):
            assert torch.equal(a, b)
