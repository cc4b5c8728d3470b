"""GPU: the combine's gradient with respect to the rows alone (dweights and Y NULL), through the C ABI."""
import numpy as np
import pytest

from test_gpu_permute import COMBINES, bf16, dev, rows_for

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402


@pytest.mark.parametrize("T,k,H", COMBINES)
@pytest.mark.parametrize("weighted,mapped", [(True, True), (False, True), (True, False)])
def test_rows_alone(T, k, H, weighted, mapped):
    """The same bits as with the weights' gradient; other rows untouched."""
    rng = np.random.default_rng(T + H)
    R = T * k + 7
    Y, _ = bf16(rng.standard_normal((R, H)))
    D, _ = bf16(rng.standard_normal((T, H)))
    w = dev(rng.standard_normal((T, k)).astype(np.float32))
    rows = dev(rows_for(T, k, R, T)) if mapped else None
    want = torch.full((R, H), 7.0, dtype=torch.bfloat16, device="cuda")
    fg.moe_combine_backward(D, Y, w if weighted else None, rows, dY=want)
    got = torch.full((R, H), 7.0, dtype=torch.bfloat16, device="cuda")
    st = fg.lib().fp8gemm_moe_combine_backward(D.data_ptr(), None, w.data_ptr() if weighted else None,
                                               rows.data_ptr() if mapped else None, got.data_ptr(), None, T, H, k, R,
                                               torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(got, want)
