"""Refusals of the gated block, its gradients and the low-rank adapters: bad arguments are rejected on the host before
any device work; and their host code's use of the stream's workspace, run against recorded HIP calls.  CPU only."""
import os
import sys
import threading

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_workspace_order import FAKE, Recorded, in_a_process  # noqa: E402

NULL, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fg.library_path()):
        from fp8_block_scaled_x128_amd import build
        build.build()
    return fg.lib()


SHAPES = (dict(M=-1), dict(I=0), dict(I=12), dict(I=-8), dict(K=0), dict(K=4), dict(act=2), dict(act=-1))
TOO_LARGE = (dict(K=(1 << 20) + 8), dict(I=(1 << 19) + 8), dict(M=1 << 31), dict(M=1 << 30, K=512), dict(M=1 << 30, I=256))


def test_gated_refusals(lib):
    def call(X=FAKE, W=FAKE, H=FAKE, pre=None, M=4, I=64, K=128, act=0):
        return lib.fp8gemm_gated_ffn(X, W, H, pre, M, I, K, act, None)
    assert call(M=0) == 0 and call(M=0, X=None, W=None, H=None) == 0
    for bad in SHAPES:
        assert call(**bad) == SHAPE, bad
    for bad in TOO_LARGE:
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=None), dict(W=None), dict(H=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(X=FAKE + 8), dict(W=FAKE + 2), dict(H=FAKE + 4), dict(pre=FAKE + 8)):
        assert call(**bad) == ALIGN, bad


def test_gated_backward_refusals(lib):
    def call(dH=FAKE, X=FAKE, W=FAKE, pre=FAKE, dpre=FAKE, dX=FAKE, dW=FAKE, M=4, I=64, K=128, act=1):
        return lib.fp8gemm_gated_ffn_backward(dH, X, W, pre, dpre, dX, dW, M, I, K, act, None)
    assert call(M=0, dW=None) == 0
    assert call(M=0, dH=None, X=None, W=None, pre=None, dpre=None, dX=None, dW=None) == 0
    for bad in SHAPES:
        assert call(**bad) == SHAPE, bad
    for bad in TOO_LARGE:
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(dH=None), dict(dpre=None), dict(X=None), dict(W=None), dict(X=None, pre=None, dW=None),
                dict(W=None, pre=None, dX=None)):
        assert call(**bad) == NULL, bad
    for name in ("dH", "X", "W", "pre", "dpre", "dX", "dW"):
        assert call(**{name: FAKE + 8}) == ALIGN, name


def test_lora_refusals(lib):
    def call(Y=FAKE, X=FAKE, A=FAKE, B=FAKE, ids=FAKE, order=None, scales=None, out=FAKE, T=4, L=3, R=16, K=128, N=64, ldx=128,
             ldy=64, ldo=64):
        return lib.fp8gemm_lora_add(Y, X, A, B, ids, order, scales, out, T, L, R, K, N, ldx, ldy, ldo, None)
    assert call(T=0) == 0 and call(N=0) == 0 and call(T=0, Y=None, X=None, ids=None, out=None) == 0
    for bad in (dict(T=-1), dict(L=0), dict(R=0), dict(R=12), dict(K=0), dict(K=20), dict(N=-8), dict(N=4), dict(ldx=120),
                dict(ldy=56), dict(ldo=0), dict(ldx=132), dict(ldy=68), dict(ldo=-64)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(R=136), dict(K=(1 << 20) + 8, ldx=1 << 21), dict(N=(1 << 20) + 8, ldy=1 << 21, ldo=1 << 21), dict(T=1 << 31),
                dict(ldx=1 << 40), dict(ldy=1 << 40), dict(ldo=1 << 60), dict(L=1 << 30), dict(T=1 << 30, ldx=1 << 11)):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("Y", "X", "A", "B", "ids", "out"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(Y=FAKE + 8), dict(X=FAKE + 2), dict(A=FAKE + 8), dict(B=FAKE + 4), dict(out=FAKE + 8), dict(ids=FAKE + 2),
                dict(order=FAKE + 1), dict(scales=FAKE + 2)):
        assert call(**bad) == ALIGN, bad


def test_lora_in_place_has_one_stride(lib):
    """Rows of the result over rows of Y at another stride would be read after they are written."""
    def call(Y, out, ldy, ldo, T=4, scales=FAKE + 2):          # (the scales' alignment is refused after the strides)
        return lib.fp8gemm_lora_add(Y, FAKE, FAKE, FAKE, FAKE, None, scales, out, T, 3, 16, 128, 64, 128, ldy, ldo, None)
    assert call(FAKE, FAKE, 64, 72) == SHAPE and call(FAKE, FAKE, 80, 64) == SHAPE
    assert call(FAKE, FAKE, 72, 72) == ALIGN and call(FAKE, FAKE + (1 << 20), 64, 72) == ALIGN
    assert call(FAKE, FAKE, 64, 72, T=1) == ALIGN              # one row has no stride


def test_binding_rejects_bad_tensors():
    import torch
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    h = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):          # host tensors are refused: no CPU path exists
        fg.gated_ffn(x, w)
    with pytest.raises(ValueError):
        fg.gated_ffn(x, w, act="relu", out=h)
    with pytest.raises(ValueError):
        fg.gated_ffn(x, w[:31], out=h)
    with pytest.raises(ValueError):
        fg.gated_ffn_backward(h, x, w)
    with pytest.raises(ValueError):
        fg.lora_add(h, x, torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 8, dtype=torch.bfloat16),
                    torch.zeros(4, dtype=torch.int32))


def test_short_path_refuses_anything():
    import torch
    calls = fg._calls()
    host = torch.zeros(4, 8)
    for name, n in (("gated_ffn", 6), ("gated_ffn_backward", 9), ("lora_add", 9)):
        f = getattr(calls, name)
        for count in (0, 1, n - 1, n, n + 1):
            for value in (None, 3, "x", host, torch.zeros(0), torch.zeros(1, 1, 1), 1 << 70, float("nan")):
                assert f(*[value] * count) == -1


class Calls(Recorded):
    def gated(self, stream, M=64, I=256, K=7168, pre=None):
        return self.lib.fp8gemm_gated_ffn(FAKE, FAKE, FAKE, pre, M, I, K, 0, stream)

    def backward(self, stream, M=256, I=512, K=1024, pre=None, dX=FAKE, dW=FAKE):
        return self.lib.fp8gemm_gated_ffn_backward(FAKE, FAKE, FAKE, pre, FAKE, dX, dW, M, I, K, 0, stream)

    def lora(self, stream, T=16, L=3, R=16, K=7168, N=4096):
        return self.lib.fp8gemm_lora_add(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, T, L, R, K, N, K, N, N, stream)

    def count(self, f, *args, **kw):
        before = len(self.launches())
        assert f(*args, **kw) == 0
        return len(self.launches()) - before


def _threads_on_one_stream(so):
    r = Calls(so)
    stream, calls = 0x1230, 12
    os.environ["FP8GEMM_FORCE_CONFIG"] = "product:128x128:2"      # K splits in every product
    work = [(f, r.count(f, stream)) for f in (r.lora, r.backward, r.gated, r.lora)]
    assert [n for _, n in work] == [2, 2, 1, 2]
    start, bad, owner = len(r.launches()), [], {}

    def run(f, n):
        owner[threading.get_native_id()] = n
        for _ in range(calls):
            if f(stream) != 0:
                bad.append(f)
    threads = [threading.Thread(target=run, args=a) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not bad
    log = r.launches(start)
    assert len(log) == calls * sum(n for _, n in work)
    at, turns = 0, 0
    while at < len(log):
        tid = log[at][0]
        assert [x[0] for x in log[at:at + owner[tid]]] == [tid] * owner[tid], "launch %d: another thread's launch within a call" % at
        turns += at > 0 and log[at - 1][0] != tid
        at += owner[tid]
    assert turns >= 3                                             # the threads did take turns


def test_launches_of_a_call_are_not_separated(tmp_path):
    in_a_process(tmp_path, "_threads_on_one_stream", __file__)


def _workspace_limits(so):
    """No workspace where none is needed; more than it holds is refused before a launch, or taken in passes."""
    r = Calls(so)
    r.hip.record_pause(0)
    before = r.hip.record_allocations()
    assert r.count(r.gated, 0x10, M=1) == 1 and r.count(r.gated, 0x10, M=4096, I=2048) == 1
    assert r.count(r.backward, 0x10, M=4096, I=2048, K=7168) in (2, 3)
    assert r.count(r.lora, 0x10, T=45, R=8, K=1544, N=2112) == 1
    assert r.hip.record_allocations() == before
    assert r.count(r.lora, 0x10) == 2
    assert r.hip.record_allocations() == before + 2
    assert r.count(r.lora, 0x10, T=140000, R=128, K=64, N=64) == 4        # 128 MiB hold 131072 rows of 128 and their halves
    assert r.count(r.lora, 0x10, T=70000, L=5000, R=8, K=64, N=64) == 4   # tiles of 16 rows, 4096 a launch
    assert r.count(r.gated, 0x10, M=1 << 29, I=8, K=8) == 1                # few tiles in one launch, of as many rows as it takes
    assert r.count(r.backward, 0x10, M=1 << 29, I=8, K=8) in (2, 3)
    os.environ["FP8GEMM_FORCE_CONFIG"] = "product:256x256:2"
    n = len(r.launches())
    assert r.gated(0x10, M=4096, I=4096) == UNSUPPORTED
    assert r.backward(0x10, M=4096, I=4096, K=4096) == UNSUPPORTED
    assert len(r.launches()) == n
    os.environ["FP8GEMM_FORCE_CONFIG"] = "product:256x256:1"
    assert r.gated(0x10, M=1 << 21, I=1 << 18, K=64) == UNSUPPORTED       # 2^13 x 2^11 tiles
    assert r.backward(0x10, M=8, I=1 << 19, K=1 << 20, dX=None) == UNSUPPORTED
    assert len(r.launches()) == n


def test_workspace_limits(tmp_path):
    in_a_process(tmp_path, "_workspace_limits", __file__)


if __name__ == "__main__":
    globals()[sys.argv[1]](sys.argv[2])
