"""GPU: the router where little can be chosen, against the 64-bit implementation of the operator's own
tests, with its tolerances."""
import numpy as np
import pytest

from test_gpu_route import INF, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)


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
