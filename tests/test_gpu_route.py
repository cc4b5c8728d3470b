"""GPU: the expert router (route_topk) and its gradient against plain 64-bit implementations written
from the definition.

The picks have to be equal.  A row whose choice hangs on a difference below 2^-18 of the values has
no one answer in 32 bits, so such rows are drawn again before the kernel sees them; exact ties stay.
Weights: exp and the reciprocal are within 2 units in the last place each, a sum of up to 1024
positive terms in 16 lanes and 64 steps adds less than 7, the quotient 1: relative error below
2^-19.  Gradients: the same factors in a difference of two sums of at most 33 terms, so absolute
error below 2^-18 of the terms' magnitudes (2^-8 relative more where the result is bf16)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402

BIG = float(np.finfo(np.float32).max)
INF = np.inf


def clean(x):
    return np.clip(np.where(np.isnan(x), -INF, x.astype(np.float64)), -INF, BIG)


def scores(logits, score):
    x = clean(logits)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return x, 1 / (1 + np.exp(-x))
        m = x.max(1, keepdims=True)
        e = np.where(x == -INF, 0.0, np.exp(x - np.where(m == -INF, 0.0, m)))
        t = e.sum(1, keepdims=True)
        return x, np.divide(e, t, out=np.zeros_like(e), where=t > 0)


def choices(logits, bias, score, n_group, topk_group, group_top):
    """(scores, choice values, sorted group scores), choice values outside the kept groups at -inf.
    Without a bias the choice goes by the logits: scores order as they do, but saturate."""
    x, s = scores(logits, score)
    c = x if bias is None else s + clean(bias)
    c = np.where(x == -INF, -INF, c)
    if n_group == 1 or topk_group == n_group:
        return s, c, None
    T, E = c.shape
    per = c.reshape(T, n_group, -1)
    if bias is None and group_top == 2:
        per = np.where(per == -INF, -INF, s.reshape(T, n_group, -1))
    gs = np.sort(per, axis=2)[:, :, ::-1][:, :, :group_top].sum(2)
    order = np.argsort(-gs, axis=1, kind="stable")
    keep = np.zeros_like(gs, dtype=bool)
    np.put_along_axis(keep, order[:, :topk_group], True, axis=1)
    return s, np.where(keep.repeat(E // n_group, 1), c, -INF), -np.sort(-gs, axis=1)


def reference(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    s, c, _ = choices(logits, bias, score, n_group, topk_group, group_top)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    there = np.take_along_axis(c, ids, 1) > -INF
    w = np.where(there, np.take_along_axis(s, ids, 1), 0.0)
    if renorm:
        t = w.sum(1, keepdims=True)
        w = np.divide(w, t, out=np.zeros_like(w), where=t > 0)
    return np.where(there, ids, -1), w * scale


def undecided(logits, bias, score, n_group, topk_group, group_top, k):
    _, c, gs = choices(logits, bias, score, n_group, topk_group, group_top)

    def close(v):
        a, b = v[:, :-1], v[:, 1:]
        fine = (b > -INF)
        d = np.where(fine, a, 0.0) - np.where(fine, b, 0.0)
        return ((d > 0) & (d < 2.0 ** -18 * np.abs(np.where(fine, a, 1.0)))).any(1)
    bad = close(-np.sort(-c, axis=1)[:, :k + 1])
    if gs is not None:
        bad |= close(gs[:, topk_group - 1:topk_group + 1])
    return bad


def to_dtype(x, dtype):
    """float32 values that the type can hold."""
    return x if dtype == "float32" else torch.from_numpy(x).to(torch.bfloat16).float().numpy()


def draw(T, E, dtype, seed, bias, score, n_group, topk_group, group_top, k, sigma=1.5):
    rng = np.random.default_rng(seed)
    logits = to_dtype(rng.standard_normal((T, E)).astype(np.float32) * np.float32(sigma), dtype)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    for _ in range(100):
        bad = undecided(logits, b, score, n_group, topk_group, group_top, k)
        if not bad.any():
            return logits, b
        logits[bad] = to_dtype(rng.standard_normal((int(bad.sum()), E)).astype(np.float32) * np.float32(sigma), dtype)
    raise AssertionError("no decided rows")


def dev(x, dtype="float32"):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(getattr(torch, dtype))


def check(logits, k, dtype="float32", bias=None, **kw):
    ids, w = fg.route_topk(dev(logits, dtype), k, bias=None if bias is None else dev(bias), **kw)
    ri, rw = reference(logits, k, bias=bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -19, atol=1e-37)
    return ids, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 7), (5, 64, 8), (17, 65, 3), (33, 128, 16), (66, 160, 6), (129, 256, 8),
                                   (7, 257, 17), (9, 511, 32), (5, 1000, 5), (4, 1024, 32)])
def test_picks_and_weights(T, E, k, dtype, score):
    for renorm, scale, bias in ((True, 1.0, False), (False, 2.5, True)):
        logits, b = draw(T, E, dtype, T + E, bias, score, 1, 1, 1, k)
        check(logits, k, dtype, bias=b, score=score, renorm=renorm, scale=scale)


@pytest.mark.parametrize("E,n_group,topk_group,group_top,k", [
    (256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (60, 4, 2, 2, 4), (72, 3, 2, 2, 5), (64, 64, 9, 1, 9), (30, 5, 1, 2, 6),
    (512, 16, 3, 2, 8), (1000, 8, 2, 2, 16), (520, 40, 7, 2, 8), (12, 6, 6, 2, 4), (96, 2, 1, 2, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, n_group, topk_group, group_top, k, score):
    """Groups that fit the lanes' chunks, straddle them, or hold one expert; every group kept."""
    for bias in (False, True):
        logits, b = draw(70, E, "float32", E + n_group, bias, score, n_group, topk_group, group_top, k)
        check(logits, k, bias=b, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top, scale=2.5)


def test_ties_go_to_the_lowest_index():
    for E, n_group in ((256, 1), (256, 8), (100, 4), (40, 1), (700, 7)):
        logits = np.zeros((3, E), np.float32)
        logits[1, 5::7] = 1.0
        logits[2] = -np.arange(E) // 9
        for score in ("softmax", "sigmoid"):
            check(logits, 8, score=score, n_group=n_group, topk_group=max(1, n_group // 2))
            check(logits, 8, "bfloat16", score=score, n_group=n_group, topk_group=max(1, n_group // 2), group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group", [1, 4])
def test_masked_and_special_logits(score, n_group):
    """-inf, NaN, +inf and the type's lowest value; rows with nothing or too little to choose."""
    rng = np.random.default_rng(5)
    E, k = 48, 6
    logits = rng.permuted(np.tile(np.arange(E, dtype=np.float32) / 8 - 3, (12, 1)), axis=1)
    logits[0] = -INF
    logits[1, 3:] = -INF
    logits[2] = np.nan
    logits[3, :40] = np.nan
    logits[4, 7] = INF
    logits[5, [9, 30]] = INF
    logits[6, 1:] = -BIG
    logits[7] = -BIG
    logits[8, ::2] = -INF
    logits[9, :44] = -INF
    kw = dict(score=score, n_group=n_group, topk_group=max(1, n_group // 2), group_top=1)
    check(logits, k, **kw)
    ids, w = fg.route_topk(dev(logits), k, renorm=False, **kw)
    assert ids[0].tolist() == [-1] * k and w[0].abs().sum() == 0
    assert torch.isfinite(w).all()
    bias = np.zeros(E, np.float32)
    bias[:40] = -INF
    bias[41] = np.nan
    ids, _ = check(logits, k, bias=bias, **kw)
    assert not np.isin(ids.cpu().numpy(), list(range(40)) + [41]).any()
    bias[44] = INF                                     # forced in wherever its logit allows it
    ids, _ = check(logits[10:], 1, bias=bias, **kw)
    assert (ids == 44).all()


def test_wide_range_of_logits():
    """Scores that underflow where the others are: weights stay finite and sum to the scale."""
    logits = np.linspace(-80, 80, 64, dtype=np.float32)[None].repeat(2, 0)
    for score in ("softmax", "sigmoid"):
        ids, w = check(logits, 4, score=score, scale=3.0)
        np.testing.assert_allclose(w.sum(1).cpu().numpy(), 3.0, rtol=1e-6)


@pytest.mark.parametrize("dtype,offset", [("float32", 1), ("bfloat16", 1), ("bfloat16", 3)])
def test_unaligned_logits(dtype, offset):
    logits, _ = draw(9, 130, dtype, 3, False, "sigmoid", 1, 1, 1, 4)
    flat = torch.zeros(9 * 130 + offset, dtype=getattr(torch, dtype), device="cuda")
    view = flat[offset:].view(9, 130)
    view.copy_(dev(logits, dtype))
    ids, w = fg.route_topk(view, 4, score="sigmoid")
    ri, rw = reference(logits, 4, score="sigmoid")
    assert np.array_equal(ids.cpu().numpy(), ri)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -19)
    dx = fg.route_topk_backward(view, ids, torch.ones_like(w), score="sigmoid", renorm=False)
    assert dx.shape == view.shape


def weights64(x, ids, score, renorm, scale):
    """The picked experts' weights from logits in 64 bits (ids fixed)."""
    _, s = scores(x, score)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        w = w / w.sum(1, keepdims=True)
    return w * scale


def gradient(x, ids, g, score, renorm, scale):
    """(dlogits, magnitude of the terms it is a difference of)."""
    _, s = scores(x, score)
    T, E = x.shape
    g = np.where(ids >= 0, g * scale, 0.0)
    p = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    dx, mag = np.zeros((T, E)), np.zeros((T, E))
    rows = np.arange(T)[:, None]
    if renorm:
        t = p.sum(1, keepdims=True)
        p = p / t
        d, m = g - (g * p).sum(1, keepdims=True), np.abs(g) + (np.abs(g) * p).sum(1, keepdims=True)
        f = p * (1 - p * t) if score == "sigmoid" else p
        for j in range(ids.shape[1]):
            ok = ids[:, j] >= 0
            dx[ok, ids[ok, j]], mag[ok, ids[ok, j]] = (d * f)[ok, j], (m * f)[ok, j]
    elif score == "sigmoid":
        for j in range(ids.shape[1]):
            ok = ids[:, j] >= 0
            dx[ok, ids[ok, j]] = (g * p * (1 - p))[ok, j]
        mag = np.abs(dx)
    else:
        spread = np.zeros((T, E))
        for j in range(ids.shape[1]):
            ok = ids[:, j] >= 0
            spread[ok, ids[ok, j]] = g[ok, j]
        dx = s * (spread - (g * p).sum(1, keepdims=True))
        mag = s * (np.abs(spread) + (np.abs(g) * p).sum(1, keepdims=True))
    del rows
    return dx, mag


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 8, 2, "float32"), (5, 1, 1, "float32"), (33, 160, 6, "bfloat16"),
                                         (70, 256, 8, "float32"), (9, 257, 17, "bfloat16"), (6, 1000, 32, "float32"),
                                         (11, 65, 5, "bfloat16"), (4, 512, 16, "float32")])
def test_backward(T, E, k, dtype, score, renorm):
    rng = np.random.default_rng(T * E)
    x = to_dtype(rng.standard_normal((T, E)).astype(np.float32) * 2, dtype)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if k > 2:
        ids[::3, 1] = -1                                # picks that are not there
    g = rng.standard_normal((T, k)).astype(np.float32)
    dx = fg.route_topk_backward(dev(x, dtype), dev(ids, "int32"), dev(g), score=score, renorm=renorm, scale=2.5)
    ref, mag = gradient(x, ids, g, score, renorm, 2.5)
    got = dx.float().cpu().numpy()
    tol = 2.0 ** -18 * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0) + 1e-37
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(score, renorm):
    """The kernel's gradient against central differences of the 64-bit weights (step 1e-5: error about
    1e-10 from the third derivative, 1e-11 from rounding), to the kernel's 32-bit tolerance."""
    rng = np.random.default_rng(8)
    T, E, k, h = 3, 20, 4, 1e-5
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids = reference(x, k, score=score)[0].astype(np.int32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    dx = fg.route_topk_backward(dev(x), dev(ids, "int32"), dev(g), score=score, renorm=renorm, scale=1.5).cpu().numpy()
    for e in range(E):
        up, down = x.astype(np.float64), x.astype(np.float64)
        up[:, e] += h
        down[:, e] -= h
        d = ((weights64(up, ids, score, renorm, 1.5) - weights64(down, ids, score, renorm, 1.5)) * g).sum(1) / (2 * h)
        np.testing.assert_allclose(dx[:, e], d, rtol=2.0 ** -16, atol=2.0 ** -18 * np.abs(g).max() * 1.5)


def test_given_outputs_other_stream_and_refusals():
    logits, b = draw(40, 96, "float32", 2, True, "sigmoid", 1, 1, 1, 4)
    x = dev(logits)
    ids = torch.full((40, 4), 77, dtype=torch.int32, device="cuda")
    w = torch.full((40, 4), 77.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fg.route_topk(x, 4, bias=dev(b), score="sigmoid", ids=ids, weights=w, stream=s)
    s.synchronize()
    assert got[0] is ids and got[1] is w
    assert np.array_equal(ids.cpu().numpy(), reference(logits, 4, bias=b, score="sigmoid")[0])
    e = fg.route_topk(x[:0], 4)
    assert e[0].shape == (0, 4)
    with pytest.raises(TypeError):
        fg.route_topk(x.double(), 4)
    with pytest.raises(ValueError):
        fg.route_topk(x.t(), 4)
    with pytest.raises(ValueError):
        fg.route_topk(x, 4, score="relu")
    with pytest.raises(ValueError):
        fg.route_topk(x, 4, bias=dev(b[:5]))
    with pytest.raises(fg.Fp8GemmError):
        fg.route_topk(x, 97)
    with pytest.raises(fg.Fp8GemmError):
        fg.route_topk(x, 4, n_group=5)


@pytest.mark.parametrize("E,n_group,topk_group,group_top,k", [(266, 2, 1, 2, 10), (376, 8, 3, 2, 32), (20, 2, 1, 1, 10),
                                                              (28, 4, 2, 2, 12), (208, 16, 5, 1, 20), (999, 3, 2, 2, 6)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_groups_of_odd_sizes(E, n_group, topk_group, group_top, k, dtype):
    """Groups with lanes to themselves and places left free, odd sizes, more picks than a group has."""
    for score in ("softmax", "sigmoid"):
        logits, b = draw(37, E, dtype, E + k, True, score, n_group, topk_group, group_top, k)
        logits[3, E // 2:] = -np.inf                   # a row with whole groups masked
        check(logits, k, dtype, bias=b, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_one_renormalised_pick_has_no_gradient(score, dtype):
    """Its weight is the scale whatever the logits are: the gradient is zero, not rounding noise."""
    rng = np.random.default_rng(2)
    logits = dev(rng.standard_normal((500, 96)).astype(np.float32), dtype)
    ids, w = fg.route_topk(logits, 1, score=score, scale=2.5)
    dx = fg.route_topk_backward(logits, ids, dev(rng.standard_normal((500, 1)).astype(np.float32)), score=score, scale=2.5)
    assert bool((w == 2.5).all()) and bool((dx == 0).all())
