"""GPU: the router where little can be chosen, where scores are tiny, and where the choice is close,
against the 64-bit implementation of the operator's own tests.

Scores are within 4 units in the last place (2^-21) of the exact ones, a share of renormalised weights
adds a sum of at most 32 terms and a quotient: relative error below 2^-19.  A score below 2^-126 is
rounded to a multiple of 2^-149."""
import numpy as np
import pytest

from test_gpu_route import INF, check, dev, gradient, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402


@pytest.mark.parametrize("E,n_group", [(64, 4), (60, 4), (128, 4), (100, 4), (256, 8), (160, 8), (512, 8), (376, 8), (1024, 8),
                                       (600, 5), (520, 40), (999, 3)])
@pytest.mark.parametrize("topk_group,group_top", [(1, 1), (1, 2), (2, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_kept_groups_run_out(E, n_group, topk_group, group_top, bias):
    """The kept groups hold fewer experts than there are picks, the others are live: the rest of the picks
    are not there, whichever groups were dropped and however many picks are missing."""
    size, k = E // n_group, 8
    rng = np.random.default_rng(E)
    logits = (rng.permuted(np.tile(np.arange(E, dtype=np.float32), (3 * n_group, 1)), axis=1) / E - 2).astype(np.float32)
    for r in range(3 * n_group):
        best = [(r + i) % n_group for i in range(topk_group)]
        for i, g in enumerate(best):
            live = min(size, group_top + (r // n_group if i == 0 else 0))   # experts of the group that can be chosen
            at = g * size + rng.permutation(size)
            logits[r, at] = -INF
            logits[r, at[:live]] = 3 + np.arange(live, dtype=np.float32) / 4 + i
    b = (rng.permutation(E) / (64.0 * E)).astype(np.float32) if bias else None
    for score in ("softmax", "sigmoid"):
        ids, w = check(logits, min(k, topk_group * size), bias=b, score=score, n_group=n_group, topk_group=topk_group,
                       group_top=group_top, scale=2.5)
        missing = ids < 0
        assert bool(missing.any()) and bool((w[missing] == 0).all())


@pytest.mark.parametrize("scale", [1.0, 2.5, 16.0])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_renormalised_weights_of_tiny_scores(scale, dtype):
    """Sigmoid scores down to the smallest that are not 0, and picks far below experts out of service: the
    weights are the picks' shares, finite and summing to the scale."""
    rows = np.float32(np.linspace(-80, -102, 45))[:, None]
    logits = rows - np.arange(16, dtype=np.float32)[None] / 8
    logits = torch.from_numpy(logits).to(getattr(torch, dtype)).float().numpy()
    for k in (1, 4, 16):
        ids, w = check(logits, k, dtype, score="sigmoid", scale=scale)
        assert bool(torch.isfinite(w).all())
        np.testing.assert_allclose(w.sum(1).cpu().numpy(), scale, rtol=2.0 ** -19)
    wide = np.concatenate([np.zeros((45, 4), np.float32), logits], axis=1)
    bias = np.zeros(20, np.float32)
    bias[:4] = -INF
    ids, w = fg.route_topk(dev(wide, dtype), 16, bias=dev(bias), score="softmax", scale=scale)
    x = np.take_along_axis(wide.astype(np.float64), ids.long().cpu().numpy(), 1)
    assert (ids >= 4).all()
    share = np.exp(x - x.max(1, keepdims=True))
    np.testing.assert_allclose(w.cpu().numpy(), share / share.sum(1, keepdims=True) * scale, rtol=2.0 ** -19)


def test_scores_below_the_type_are_zero():
    """Where every pick's score rounds to 0 in 32 bits the weights are 0; scores below 2^-126 are kept."""
    logits = np.full((2, 8), -150.0, np.float32)
    for renorm in (False, True):
        ids, w = fg.route_topk(dev(logits), 3, score="sigmoid", renorm=renorm)
        assert ids[0].tolist() == [0, 1, 2] and bool((w == 0).all())
    logits = (-86 - np.arange(64, dtype=np.float32) / 4)[None]
    for scale in (1.0, 16.0):
        ids, w = fg.route_topk(dev(logits), 32, score="sigmoid", renorm=False, scale=scale)
        ref = reference(logits, 32, score="sigmoid", renorm=False, scale=scale)[1]
        assert (np.abs(w.cpu().numpy() - ref) <= 2.0 ** -19 * ref + (scale + 1) * 2.0 ** -149).all()


def test_gradient_of_tiny_scores():
    """Renormalised sigmoid weights keep their gradient where the scores are below 2^-126."""
    rng = np.random.default_rng(3)
    x = (-84 - 16 * rng.random((40, 24))).astype(np.float32)
    ids = np.argsort(rng.random((40, 24)), axis=1)[:, :6].astype(np.int32)
    g = rng.standard_normal((40, 6)).astype(np.float32)
    dx = fg.route_topk_backward(dev(x), dev(ids, "int32"), dev(g), score="sigmoid", renorm=True, scale=2.5)
    ref, mag = gradient(x, ids, g, "sigmoid", True, 2.5)
    assert (np.abs(dx.cpu().numpy() - ref) <= 2.0 ** -18 * mag).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_between_close_values(score):
    """One expert with a tiny score against one whose bias is that score 1.5e-6 of it up or down: three
    times the scores' and the sum's rounding (4.8e-7 + 0.6e-7), so the choice is decided."""
    rng = np.random.default_rng(4)
    R = 120
    x = (-50 - 36 * rng.random(R)).astype(np.float32)
    E = 2 * R + 1                                       # the last is out of service, softmax's largest
    logits = np.full((R, E), -INF, np.float32)
    bias = np.zeros(E, np.float32)
    s = 1 / (1 + np.exp(-x.astype(np.float64))) if score == "sigmoid" else np.exp(x.astype(np.float64)) / (1 + np.exp(x.astype(np.float64)))
    side = np.where(rng.random(R) < 0.5, 1.0, -1.0)
    at = np.arange(R)
    logits[at, 2 * at] = x
    logits[at, 2 * at + 1] = -103.0                     # its own score is below 1e-8 of the other's
    bias[2 * at + 1] = (s * (1 + 1.5e-6 * side)).astype(np.float32)
    logits[:, E - 1] = 0.0
    bias[E - 1] = -INF
    ids, _ = fg.route_topk(dev(logits), 2, bias=dev(bias), score=score)
    want = np.where(side > 0, 2 * at + 1, 2 * at)
    assert np.array_equal(ids[:, 0].cpu().numpy(), want)


def test_choice_between_close_values_far_below_the_largest():
    """The same for softmax below a largest logit that is not 0: the score's two powers and the quotient make
    7e-7 at most, less than half of the difference."""
    rng = np.random.default_rng(5)
    R = 120
    x = (-46 - 24 * rng.random(R)).astype(np.float32)
    E = 2 * R + 1
    top = np.float32(11.7)
    logits = np.full((R, E), -INF, np.float32)
    bias = np.zeros(E, np.float32)
    s = np.exp(x.astype(np.float64)) / (np.exp(x.astype(np.float64)) + np.exp(float(top)))
    side = np.where(rng.random(R) < 0.5, 1.0, -1.0)
    at = np.arange(R)
    logits[at, 2 * at] = x
    logits[at, 2 * at + 1] = -100.0
    bias[2 * at + 1] = (s * (1 + 1.5e-6 * side)).astype(np.float32)
    logits[:, E - 1] = top
    bias[E - 1] = -INF
    ids, _ = fg.route_topk(dev(logits), 2, bias=dev(bias), score="softmax")
    assert np.array_equal(ids[:, 0].cpu().numpy(), np.where(side > 0, 2 * at + 1, 2 * at))
