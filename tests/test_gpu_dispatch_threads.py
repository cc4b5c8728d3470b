"""GPU: large dispatches and products that split K, from several host threads on one stream.  Each call's
launches stay together on it, so every call gives the same bits as the same calls made one at a time."""
import threading

import numpy as np
import pytest

import workloads as W
from test_gpu_permute import dev, pick, tokens

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402


def make_calls():
    """Calls without arguments, each with its own outputs, which it returns."""
    calls = []
    for T, k, G, H, seed in ((2000, 8, 40, 256, 1), (9000, 1, 7, 640, 2), (1500, 8, 300, 128, 3)):
        _, X = tokens(T, H, seed)
        ids = dev(pick(T, k, G, seed))
        calls.append(lambda X=X, ids=ids, G=G: fg.moe_dispatch_contiguous(X, ids, G))
        calls.append(lambda X=X, ids=ids, G=G, n=T * k: fg.moe_dispatch_masked(X, ids, G, n // G * 4))
    for M, N, K, seed in ((64, 2112, 7168, 5), (128, 2112, 7168, 6)):
        d = W.dense(M, N, K, seed=seed)
        ops = (dev(d.A), dev(np.swapaxes(d.sa, -1, -2)), dev(d.B), dev(d.sb))
        calls.append(lambda ops=ops: (fg.gemm_nt(*ops),))
    return calls


def bits(outs):
    return [t.contiguous().view(torch.uint8).cpu() for t in outs]


def test_threads_on_one_stream_match_sequential_calls():
    calls = make_calls()
    want = []
    for c in calls:
        want.append(bits(c()))
    fg.read_device_error()
    results, errors = [], []

    def worker(n):
        try:
            done = [((n * 3 + r) % len(calls), calls[(n * 3 + r) % len(calls)]()) for r in range(8)]
            results.extend(done)
        except Exception as e:  # reported below, in the main thread
            errors.append(repr(e))
    threads = [threading.Thread(target=worker, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    torch.cuda.synchronize()
    fg.read_device_error()
    assert len(results) == 32
    for i, outs in results:
        for a, b in zip(want[i], bits(outs)):
            assert torch.equal(a, b), i
