"""GPU: the gated block and its gradients on matrices that start beside 128-byte lines."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_gpu_ffn import bits, off_by  # noqa: E402
from test_gpu_gated import normal  # noqa: E402

bf16 = torch.bfloat16


@pytest.mark.parametrize("M,I,K", [(8, 2816, 4480), (64, 2048, 2048), (300, 1408, 1024), (500, 512, 7168), (1000, 1408, 2048), (2048, 512, 1024)])
def test_the_same_bits_anywhere(M, I, K):
    X, W, dH = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I)
    results = []
    for chunks in (0, 1, 6):
        x, w, d = off_by(X, chunks), off_by(W, 7 * chunks % 8), off_by(dH, chunks)
        pre, dpre = (off_by(torch.zeros((M, 2 * I), dtype=bf16, device="cuda"), chunks) for _ in range(2))
        H = fg.gated_ffn(x, w, pre=pre)
        out = [H, pre]
        for kept in (pre, None):
            out += fg.gated_ffn_backward(d, x, w, pre=kept, dpre=dpre) + (dpre.clone(),)
        results.append([bits(t) for t in out])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
