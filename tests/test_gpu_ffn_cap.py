"""GPU: the gated block, its gradients and the adapters with launch shapes sized for fewer CUs."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_gpu_gated import backward_close, forward_close, normal  # noqa: E402
from test_gpu_lora import case, check  # noqa: E402


@pytest.fixture(params=[1, 24, 100])
def cap(request):
    fg.set_num_cus(request.param)
    yield request.param
    fg.set_num_cus(0)


@pytest.mark.parametrize("M,I,K", [(3, 128, 512), (40, 72, 1024), (300, 264, 712), (1023, 336, 456)])
def test_gated_block(cap, M, I, K):
    X, W, dH = normal(M, M, K), normal(I, 2 * I, K, scale=K ** -0.5), normal(K, M, I)
    pre, dpre = (torch.empty((M, 2 * I), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    forward_close(X, W, "silu", fg.gated_ffn(X, W, pre=pre), pre)
    for kept in (pre, None):
        dX, dW = fg.gated_ffn_backward(dH, X, W, pre=kept, dpre=dpre)
        backward_close(dH, X, W, "silu", kept, dpre, dX, dW)


@pytest.mark.parametrize("T,L,R,K,N", [(20, 4, 16, 640, 264), (70, 9, 16, 2560, 520), (70, 9, 104, 4360, 520), (1500, 4, 32, 1608, 520)])
def test_adapters(cap, T, L, R, K, N):
    c = case(T, L, R, K, N, seed=T)
    check(c, fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"]))
