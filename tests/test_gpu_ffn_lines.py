"""GPU: the gated block and its gradients on matrices that start beside 128-byte lines."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_gpu_ffn import bits, off_by  # noqa: E402
from test_gpu_gated import backward_close, forward_close, normal  # noqa: E402

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


@pytest.mark.parametrize("chunks", [0, 1, 4, 7])
@pytest.mark.parametrize("K", [2056, 2080, 2104, 2112])
@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("tile,M,I", [("128x128", 1500, 456), ("64x64", 700, 520)])
def test_by_lines(tile, M, I, split, K, chunks, monkeypatch):
    """Loads by whole lines, as the configuration says, with every kind of K's end: 1, 4 and 7 chunks of 16 bytes, and a
    whole slice."""
    monkeypatch.setenv("FP8GEMM_FORCE_CONFIG", "product:%s:%d" % (tile, split))
    X, W, dH = off_by(normal(1, M, K), chunks), off_by(normal(2, 2 * I, K, scale=K ** -0.5), 7 * chunks % 8), normal(3, M, I)
    pre, dpre = torch.zeros((M, 2 * I), dtype=bf16, device="cuda"), off_by(torch.zeros((M, 2 * I), dtype=bf16, device="cuda"), chunks)
    H = fg.gated_ffn(X, W, pre=pre)
    lines = chunks > 0 or K % 64 > 0
    assert fg.last_config().endswith("tile=%s split=%d lines=%d" % (tile, split, lines))
    forward_close(X, W, "silu", H, pre)
    dX, dW = fg.gated_ffn_backward(dH, X, W, dpre=dpre)
    words = fg.last_config()
    assert "dX tile=%sx4 split=%d lines=1 " % (tile, split) in words and words.endswith("products tile=%sx4 split=%d lines=%d" % (tile, split, lines))
    backward_close(dH, X, W, "silu", None, dpre, dX, dW)
