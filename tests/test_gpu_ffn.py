"""GPU: the gated block, its gradients and the low-rank adapters where calls can go wrong beside their sizes: every tile and
K split, graphs, streams and threads, operands past 2^32 bytes, values that are not finite, and the three run together.
Tolerances are those of the operators' own tests (test_gpu_gated.py, test_gpu_lora.py)."""
import os
import sys
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402
from test_gpu_gated import act64, backward_close, forward_close, normal, within  # noqa: E402
from test_gpu_lora import case, check, rows_apart  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
bf16 = torch.bfloat16


def bits(t):
    return t.detach().contiguous().view(torch.int16).clone()


@pytest.mark.parametrize("act,kept", [("silu", True), ("gelu_tanh", False)])
@pytest.mark.parametrize("split", [1, 2, 3, 5])
@pytest.mark.parametrize("tile", ["256x256", "128x256", "128x128", "64x64", "64x64x2"])
def test_every_tile_and_split(tile, split, act, kept, monkeypatch):
    monkeypatch.setenv("FP8GEMM_FORCE_CONFIG", "product:%s:%d" % (tile, split))
    M, I, K = 333, 264, 712
    X, W, dH = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I)
    pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    H = fg.gated_ffn(X, W, act=act, pre=pre)
    assert tile in fg.last_config() or tile == "64x64x2"     # (a shape of the gradients)
    forward_close(X, W, act, H, pre)
    dpre = torch.empty_like(pre)
    for need in ((True, True), (True, False), (False, True)):
        dX, dW = fg.gated_ffn_backward(dH, X, W, pre=pre if kept else None, act=act, dpre=dpre, need_dX=need[0], need_dW=need[1])
        backward_close(dH, X, W, act, pre if kept else None, dpre, dX, dW)
    for n in (2, 64):                      # fewer rows than any tile, fewer slices of dW's sum than splits
        dX, dW = fg.gated_ffn_backward(dH[:n], X[:n], W, pre=pre[:n] if kept else None, act=act, dpre=dpre[:n])
        backward_close(dH[:n], X[:n], W, act, pre[:n] if kept else None, dpre[:n], dX, dW)


def test_no_rows():
    X, W = torch.empty((0, 72), dtype=bf16, device="cuda"), normal(1, 48, 72)
    assert fg.gated_ffn(X, W).shape == (0, 24)
    dW = torch.full((48, 72), float("nan"), dtype=bf16, device="cuda")
    dX, got = fg.gated_ffn_backward(X.new_empty((0, 24)), X, W, dW=dW)
    assert dX.shape == (0, 72) and got is dW and (dW == 0).all()
    c = case(4, 2, 8, 64, 72, seed=1)
    assert fg.lora_add(c["Y"][:0], c["X"][:0], c["A"], c["B"], c["ids"][:0]).shape == (0, 72)
    assert fg.lora_add(c["Y"][:, :0].contiguous(), c["X"], c["A"], c["B"][:, :0].contiguous(), c["ids"]).shape == (4, 0)


def test_refusals_of_device_tensors():
    X, W = normal(1, 6, 64), normal(2, 32, 64)
    dH = normal(3, 6, 16)
    bad = [lambda: fg.gated_ffn(X.float(), W), lambda: fg.gated_ffn(X, W[:, :56].contiguous()), lambda: fg.gated_ffn(X.t(), W),
           lambda: fg.gated_ffn(X, W, pre=X), lambda: fg.gated_ffn(X, W, out=dH[:5]), lambda: fg.gated_ffn(X[:, :60].contiguous(), W[:, :60].contiguous()),
           lambda: fg.gated_ffn(X.cpu(), W), lambda: fg.gated_ffn_backward(dH[:, :8], X, W), lambda: fg.gated_ffn_backward(dH, X, W, dX=W)]
    c = case(6, 2, 8, 64, 72, seed=1)
    Y, A, B, ids = c["Y"], c["A"], c["B"], c["ids"]
    bad += [lambda: fg.lora_add(Y, c["X"], A, B, ids.long()), lambda: fg.lora_add(Y, c["X"], A, B, ids, order=ids[:5]),
            lambda: fg.lora_add(Y, c["X"], A, B, ids, scales=c["scales"].double()), lambda: fg.lora_add(Y, c["X"].t().contiguous().t(), A, B, ids),
            lambda: fg.lora_add(Y[:1].expand(6, 72), c["X"], A, B, ids), lambda: fg.lora_add(Y, c["X"], A[:, :, :56], B, ids),
            lambda: fg.lora_add(Y, c["X"], A, B[:1], ids), lambda: fg.lora_add(Y[:, :64], c["X"], A, B, ids),
            lambda: fg.lora_add(Y, c["X"], A, B, ids, out=torch.empty((6, 76), dtype=bf16, device="cuda")[:, 1:73])]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, fg.Fp8GemmError)):
            f()
            pytest.fail("call %d was taken" % i)


# a kernel of few rows, tiles with and without K splits; adapters by row, a few rows a workgroup, 64 rows
GATED = [(3, 128, 512), (40, 72, 1024), (300, 264, 712), (1023, 336, 456)]
LORA = [(20, 4, 16, 640, 264), (70, 9, 16, 2560, 520), (70, 9, 16, 4360, 520), (1500, 4, 32, 328, 520)]


def test_graphs():
    """Captured together, replayed with the program's own work between, beside a second graph of the same stream."""
    s = torch.cuda.Stream()
    todo, outs = [], []
    for M, I, K in GATED:
        X, W, dH = normal(M, M, K), normal(I, 2 * I, K, scale=K ** -0.5), normal(K, M, I)
        o = [torch.zeros(n, dtype=bf16, device="cuda") for n in ((M, I), (M, 2 * I), (M, 2 * I), (M, K), (2 * I, K))]
        outs += o

        def both(X=X, W=W, dH=dH, o=o):
            fg.gated_ffn(X, W, pre=o[1], out=o[0], stream=s)
            fg.gated_ffn_backward(dH, X, W, pre=o[1], dpre=o[2], dX=o[3], dW=o[4], stream=s)
        todo.append(both)
    for T, L, R, K, N in LORA:
        c = case(T, L, R, K, N, seed=T)
        o = torch.zeros((T, N), dtype=bf16, device="cuda")
        outs.append(o)
        todo.append(lambda c=c, o=o: fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"], out=o, stream=s))
    fg.prepare_stream(s)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for f in todo:
            f()
    s.synchronize()
    ref = [bits(t) for t in outs]
    graphs = []
    for run in (todo, todo[::-1]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for f in run:
                f()
        graphs.append(g)
    for r in range(4):
        for t in outs:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graphs[r % 2].replay()
        torch.cuda.synchronize()
        for i, t in enumerate(outs):
            assert torch.equal(bits(t), ref[i]), "replay %d, output %d" % (r, i)
    assert fg.read_device_error() == 0


def test_capture_on_an_unprepared_stream(monkeypatch):
    """What needs the stream's workspace is refused while the stream captures and has none, the rest is taken."""
    M, I, K = 40, 72, 1024
    X, W, dH = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I)
    c = case(20, 4, 16, 640, 264, seed=2)
    big = case(20, 4, 16, 4608, 264, seed=2)
    o = [torch.zeros(n, dtype=bf16, device="cuda") for n in ((M, 2 * I), (M, K), (2 * I, K), (20, 264))]
    fg.gated_ffn(X, W)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    H = torch.zeros((M, I), dtype=bf16, device="cuda")
    with torch.cuda.graph(g, stream=s):
        monkeypatch.setenv("FP8GEMM_FORCE_CONFIG", "product:64x64:2")
        with pytest.raises(fg.Fp8GemmError):
            fg.gated_ffn(X, W, out=H, stream=s)
        monkeypatch.delenv("FP8GEMM_FORCE_CONFIG")
        with pytest.raises(fg.Fp8GemmError):
            fg.lora_add(big["Y"], big["X"], big["A"], big["B"], big["ids"], out=o[3], stream=s)
        fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], out=o[3], stream=s)
        fg.gated_ffn(X[:2], W, out=H[:2], stream=s)
    g.replay()
    torch.cuda.synchronize()
    check(c, o[3], scales=False)
    forward_close(X[:2], W, "silu", H[:2], None)


def test_threads_on_their_own_streams():
    """Concurrent calls give the bits of calls made one at a time."""
    jobs = []
    for M, I, K in GATED[1:]:
        X, W, dH = normal(M, M, K), normal(I, 2 * I, K, scale=K ** -0.5), normal(K, M, I)
        jobs.append(lambda s, X=X, W=W: (fg.gated_ffn(X, W, stream=s),))
        jobs.append(lambda s, X=X, W=W, dH=dH: fg.gated_ffn_backward(dH, X, W, stream=s))
    for T, L, R, K, N in LORA:
        c = case(T, L, R, K, N, seed=T)
        jobs.append(lambda s, c=c: (fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"], stream=s),))
    want = [[bits(t) for t in f(None)] for f in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(n):
        s = torch.cuda.Stream()
        for r in range(3):
            for i in range(len(jobs)):
                j = (i + n) % len(jobs)
                with torch.cuda.stream(s):
                    got = jobs[j](s)
                s.synchronize()
                if not all(torch.equal(bits(t), w) for t, w in zip(got, want[j])):
                    bad.append((n, r, j))
    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and not bad, bad


def test_threads_on_one_stream():
    """Two threads' calls on one stream share its workspace and keep apart."""
    s = torch.cuda.Stream()
    c = case(70, 9, 16, 4360, 520, seed=70)
    X, W, dH = normal(1, 40, 1024), normal(2, 144, 1024, scale=2.0 ** -5), normal(3, 40, 72)
    jobs = [lambda: (fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"], stream=s),),
            lambda: (fg.gated_ffn(X, W, stream=s),) + fg.gated_ffn_backward(dH, X, W, stream=s)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        want = [[bits(t) for t in f()] for f in jobs]
    s.synchronize()
    got = [[], []]

    def work(n):
        with torch.cuda.stream(s):
            for _ in range(20):
                got[n].append(jobs[n]())
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    for n in range(2):
        assert len(got[n]) == 20 and all(torch.equal(bits(t), w) for call in got[n] for t, w in zip(call, want[n]))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,I,K", [(5, 40, 72), (70, 72, 136)])
def test_large_values(M, I, K, act):
    """Gates from tiny to 1e15 of both signs: no exponential's overflow reaches a result."""
    size = (10.0 ** torch.linspace(-8, 15, M, device="cuda"))[:, None]
    X = (normal(1, M, K).float() * size).to(bf16)
    W, dH = normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I)
    pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    forward_close(X, W, act, fg.gated_ffn(X, W, act=act, pre=pre), pre)
    dpre = torch.empty_like(pre)
    for p in (pre, None):
        dX, dW = fg.gated_ffn_backward(dH, X, W, pre=p, act=act, dpre=dpre)
        backward_close(dH, X, W, act, p, dpre, dX, dW)


@pytest.mark.parametrize("M,I,K", [(6, 40, 72), (70, 72, 136), (300, 136, 200)])
def test_values_that_are_not_finite(M, I, K):
    """A row of X, a pair of W's rows and a row of dH that are not finite change their own results only, and what
    stands behind the last row changes none."""
    X = torch.full((M + 70, K), float("nan"), dtype=bf16, device="cuda")
    W, dH = normal(2, 2 * I, K, scale=K ** -0.5), torch.full((M + 70, I), float("nan"), dtype=bf16, device="cuda")
    X[:M], dH[:M] = normal(1, M, K), normal(3, M, I)
    X, dH = X[:M], dH[:M]
    H = fg.gated_ffn(X, W)
    dpre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    dX, dW = fg.gated_ffn_backward(dH, X, W, dpre=dpre)
    forward_close(X, W, "silu", H, None)
    backward_close(dH, X, W, "silu", None, dpre, dX, dW)
    X2, W2, dH2 = X.clone(), W.clone(), dH.clone()
    X2[3], W2[11] = float("nan"), float("inf")
    H2 = fg.gated_ffn(X2, W2)
    rows, cols = torch.arange(M, device="cuda") != 3, torch.arange(I, device="cuda") != 11
    assert torch.equal(H2[rows][:, cols], H[rows][:, cols]) and H2[3].isnan().all()
    dH2[5] = float("nan")
    dp2 = torch.empty_like(dpre)
    dX2, dW2 = fg.gated_ffn_backward(dH2, X, W, dpre=dp2)
    rows = torch.arange(M, device="cuda") != 5
    assert torch.equal(dp2[rows], dpre[rows]) and torch.equal(dX2[rows], dX[rows])
    assert dX2[5].isnan().all() and dW2.isnan().all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(act):
    """dX and dW along their own signs against central differences in 64 bits of <dH, H>.  Each gradient is off by
    2^-8 of itself and by 2^-8 sum |dpre| |w| through dpre's rounding (twice that where g and u are rounded too)."""
    M, I, K = 41, 72, 136
    X, W, dH = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5), normal(3, M, I)
    pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    fg.gated_ffn(X, W, act=act, pre=pre)
    dpre = torch.empty_like(pre)
    dX, dW = (t.double() for t in fg.gated_ffn_backward(dH, X, W, act=act, dpre=dpre))

    def loss(x, w):
        g, u = (x @ w.t()).chunk(2, dim=1)
        return (dH.double() * act64(g, act)[0] * u).sum()
    x, w, h, r = X.double(), W.double(), 1e-6, dpre.double().abs()
    for grad, at, off in ((dX, lambda e: loss(x + e * dX.sign(), w), r @ w.abs()), (dW, lambda e: loss(x, w + e * dW.sign()), r.t() @ x.abs())):
        diff = float((at(h) - at(-h)) / (2 * h))
        got = float(grad.abs().sum())
        tol = 2.0 ** -8 * float(grad.abs().sum() + off.sum()) + 1e-6 * abs(got)
        assert tol < 0.25 * got and abs(got - diff) <= tol, (got, diff, tol)


def test_x_past_4gib():
    """dX's and X's rows on both sides of 2^32 bytes; dH is zero but in some rows, so that dW's sums are short."""
    M, I, K = (1 << 20) + 37, 8, 2056
    X = torch.randn((M, K), dtype=bf16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    W = normal(2, 2 * I, K, scale=K ** -0.5)
    edge = (1 << 32) // (2 * K)
    rows = torch.tensor([0, 1, 777, edge - 1, edge, edge + 1, M - 65, M - 2, M - 1], device="cuda")
    dH = torch.zeros((M, I), dtype=bf16, device="cuda")
    dH[rows] = normal(3, len(rows), I)
    H = fg.gated_ffn(X, W)
    forward_close(X[rows], W, "silu", H[rows], None)
    dpre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    dX, dW = fg.gated_ffn_backward(dH, X, W, dpre=dpre)
    backward_close(dH[rows], X[rows], W, "silu", None, dpre[rows], dX[rows], dW)
    other = torch.ones(M, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert not dX[other].any()


@pytest.mark.parametrize("M", [3, 70])
def test_w_past_4gib(M):
    """W's and dW's rows past 2^32 bytes; dH is zero but in some columns."""
    I, K = (1 << 17) + 40, 8200
    W = torch.randn((2 * I, K), dtype=bf16, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 2.0 ** -6
    X = normal(2, M, K)
    edge = (1 << 32) // (2 * K) - I                                  # an up row
    cols = torch.tensor([0, 9, edge - 1, edge, edge + 1, I // 2, I - 65, I - 1], device="cuda")
    both = torch.cat((cols, I + cols))
    dH = torch.zeros((M, I), dtype=bf16, device="cuda")
    dH[:, cols] = normal(3, M, len(cols))
    pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    H = fg.gated_ffn(X, W, pre=pre)
    forward_close(X, W[both], "silu", H[:, cols], pre[:, both])
    dpre = torch.empty_like(pre)
    dX, dW = fg.gated_ffn_backward(dH, X, W, pre=pre, dpre=dpre)
    backward_close(dH[:, cols], X, W[both], "silu", pre[:, both], dpre[:, both], dX, dW[both])
    other = torch.ones(2 * I, dtype=torch.bool, device="cuda")
    other[both] = False
    assert not any(part.any() for part in (dW[:I][other[:I]], dW[I:][other[I:]]))


def test_pre_past_4gib():
    """dpre and pre past 2^32 bytes, with and without the products kept."""
    M, I, K = (1 << 15) + 5, (1 << 15) + 8, 8
    X, W = normal(1, M, K), normal(2, 2 * I, K, scale=K ** -0.5)
    rows = torch.tensor([0, 5, (1 << 32) // (4 * I) - 1, (1 << 32) // (4 * I), M - 1], device="cuda")
    dH = torch.zeros((M, I), dtype=bf16, device="cuda")
    dH[rows] = normal(3, len(rows), I)
    pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    H = fg.gated_ffn(X, W, pre=pre)
    forward_close(X[rows], W, "silu", H[rows], pre[rows])
    dpre = torch.empty_like(pre)
    for p in (pre, None):
        dX, dW = fg.gated_ffn_backward(dH, X, W, pre=p, dpre=dpre)
        backward_close(dH[rows], X[rows], W, "silu", None if p is None else p[rows], dpre[rows], dX[rows], dW)


@pytest.mark.parametrize("T,R,K,N", [(300, 16, 136, 264), (300, 16, 2568, 264), (300, 16, 4168, 264), (1100, 16, 136, 264)])
def test_adapters_rows_past_4gib(T, R, K, N):
    """Rows of X, Y and the result so far apart that they pass 2^32 bytes."""
    c = case(T, 3, R, K, N, seed=T)
    want = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"])
    step = 1 << 23 if T <= 300 else 1 << 21
    wide = torch.empty((T, step), dtype=bf16, device="cuda")
    assert 2 * wide.numel() > 1 << 32
    X, Y, out = wide[:, :K], wide[:, 8192:8192 + N], wide[:, 12288:12288 + N]
    X.copy_(c["X"])
    Y.copy_(c["Y"])
    assert torch.equal(fg.lora_add(Y, X, c["A"], c["B"], c["ids"], c["scales"], out=out), want)
    check(c, want)


@pytest.mark.parametrize("T,R,K,N", [(40, 16, 4096, 4096), (40, 16, 2048, 2048), (1300, 16, 4096, 4096), (1300, 128, 1 << 18, 72),
                                     (1300, 128, 72, 1 << 18)])
def test_adapters_past_4gib(T, R, K, N):
    """Adapters on both sides of 2^32 bytes of A, of B, or of both."""
    L = (1 << 31) // (R * max(K, N)) + 9
    gen = torch.Generator("cuda").manual_seed(1)
    A = torch.randn((L, R, K), dtype=bf16, device="cuda", generator=gen) * 2.0 ** -6
    B = torch.randn((L, N, R), dtype=bf16, device="cuda", generator=gen) * 0.25
    named = torch.tensor([0, 1, L - 10, L - 9, L - 8, L - 1], device="cuda")
    small = torch.arange(T, device="cuda") % len(named)
    c = dict(X=normal(2, T, K), Y=normal(3, T, N), A=A[named], B=B[named], ids=small.int(), scales=torch.ones(len(named), device="cuda"))
    check(c, fg.lora_add(c["Y"], c["X"], A, B, named[small].int()), scales=False)


@pytest.mark.parametrize("T,L,R,K,N", [(140000, 30, 128, 64, 72), (70000, 5000, 8, 64, 72)])
def test_adapters_in_several_passes(T, L, R, K, N):
    """More rows than the workspace holds, with and without an order of the rows."""
    c = case(T, L, R, K, N, seed=1)
    got = fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"])
    s, x = c["scales"].double(), c["X"].double()
    live = c["ids"] >= 0
    assert torch.equal(got[~live], c["Y"][~live])
    pick = live.nonzero().squeeze(1)[::37]
    a = c["ids"][pick].long()
    Ad, Bd = c["A"].double(), c["B"].double()
    v = torch.bmm(Ad[a], x[pick][:, :, None])
    ref = c["Y"][pick].double() + s[a][:, None] * torch.bmm(Bd[a], v)[:, :, 0]
    low = 2.0 ** -18 * torch.bmm(Ad[a].abs(), x[pick].abs()[:, :, None]) + 2.0 ** -15 * v.abs()
    within(got[pick], ref, s[a].abs()[:, None] * torch.bmm(Bd[a].abs(), low)[:, :, 0] + 2.0 ** -22 * ref.abs())
    order = c["ids"].argsort(stable=True).int()
    assert torch.equal(fg.lora_add(c["Y"], c["X"], c["A"], c["B"], c["ids"], c["scales"], order=order), got)
    assert fg.read_device_error() == 0


@pytest.mark.parametrize("T,L,R,K,N", [(20, 4, 24, 264, 136), (40, 4, 16, 2568, 136), (40, 4, 16, 4168, 136), (70, 4, 104, 1200, 136), (1100, 4, 16, 200, 264), (700, 3, 72, 136, 136)])
def test_adapters_in_every_kernel(T, L, R, K, N):
    """By row, a few rows a workgroup, and 64 rows: apart, in place, in another order, ids and orders out of range, neighbours
    that are not finite, an infinite A x."""
    c = case(T, L, R, K, N, seed=T + K)
    c["ids"][[1, 2, 3]] = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def call(ids=c["ids"], **kw):
        v = dict(c, ids=ids, **{k: kw.pop(k) for k in list(kw) if k in c})
        return fg.lora_add(v["Y"], v["X"], v["A"], v["B"], v["ids"], v["scales"], **kw)
    want = call()
    check(c, want)
    wide = rows_apart(c["Y"], 40)
    assert torch.equal(call(Y=wide, X=rows_apart(c["X"], 8), out=wide), want)
    perm = torch.randperm(T, generator=torch.Generator("cuda").manual_seed(1), device="cuda").int()
    assert torch.equal(call(order=perm), want)
    fg.read_device_error()
    ids = c["ids"].clone()
    ids[5], ids[T - 1] = L, 2 ** 31 - 1
    out = call(ids=ids)
    assert fg.read_device_error() == fg.DEVERR_BAD_INDEX
    ids[5] = ids[T - 1] = -(2 ** 31)
    check(c, out, ids=ids)
    order = perm.clone()
    order[3], order[T - 2] = T, -7
    kept = call(order=order, out=torch.full_like(want, 3.0))
    assert fg.read_device_error() == fg.DEVERR_BAD_INDEX
    named = torch.ones(T, dtype=torch.bool, device="cuda")
    named[perm[[3, T - 2]].long()] = False
    assert torch.equal(kept[named], want[named]) and (kept[~named] == 3).all()
    A, B, X = c["A"].clone(), c["B"].clone(), c["X"].clone()
    A[2], B[2] = float("inf"), float("nan")
    X[c["ids"] < 0] = float("nan")
    rows = c["ids"] != 2
    got = call(A=A, B=B, X=X)
    assert torch.equal(got[rows], want[rows]) and got[~rows].isnan().all()
    # A x of infinity, B without zeros: the infinity of the formula, with its sign
    A, B = c["A"].clone(), c["B"].clone()
    X = c["X"].clone()
    A[1], B[1], X[2] = 3e38, 0.0, 0.0
    A[1, 0], B[1, :, 0], X[2, :8] = 3e38, -2.0, 8.0
    A[1, 1:] = 0.0
    scales = c["scales"].clone()
    scales[1] = 1.5
    got = call(A=A, B=B, X=X, scales=scales)
    assert (got[2] == -float("inf")).all()
    assert torch.equal(got[c["ids"] != 1], want[c["ids"] != 1])


@pytest.mark.parametrize("T,hidden,inter,L,R,act", [(1, 256, 128, 2, 8, "silu"), (77, 512, 256, 5, 16, "gelu_tanh"), (1300, 256, 384, 3, 40, "silu")])
def test_served_block(T, hidden, inter, L, R, act):
    """Gated layer, quantisation, FP8 product and adapters: the low-rank part against 64 bits, on the bf16 results that
    the program itself has in between."""
    from gated_ffn import Block
    block = Block(hidden, inter, L, R, act=act)
    x = normal(5, T, hidden)
    ids = torch.tensor(np.random.default_rng(T).integers(-1, L, T), dtype=torch.int32, device="cuda")
    got = block.serve(x, ids)
    h = fg.gated_ffn(x, block.w1, act=act)
    forward_close(x, block.w1, act, h, None)
    y = fg.gemm_nt(*fg.quantize_1x128(h), block.w2, block.s2)
    check(dict(X=h, Y=y, A=block.a, B=block.b, ids=ids, scales=block.scales), got)


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,I,K", [(3, 64, 128), (130, 72, 264)])
def test_autograd(M, I, K, act, keep):
    """The autograd function's gradients against the formula's, through a gradient that is not contiguous and
    with one gradient not needed."""
    from gated_ffn import GatedFfn
    X, W, dH = normal(1, M, K).requires_grad_(), normal(2, 2 * I, K, scale=K ** -0.5).requires_grad_(), normal(3, I, M).t()
    h = GatedFfn.apply(X, W, act, keep)
    dX, dW = torch.autograd.grad(h, (X, W), dH)
    pre = None
    x, w = X.detach(), W.detach()
    if keep:
        pre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
        fg.gated_ffn(x, w, act=act, pre=pre)
    dpre = torch.empty((M, 2 * I), dtype=bf16, device="cuda")
    wantX, wantW = fg.gated_ffn_backward(dH.contiguous(), x, w, pre=pre, act=act, dpre=dpre)
    assert torch.equal(dX, wantX) and torch.equal(dW, wantW)
    backward_close(dH, x, w, act, pre, dpre, dX, dW)
    (alone,) = torch.autograd.grad(GatedFfn.apply(x, W, act, keep), W, dH)
    backward_close(dH, x, w, act, pre, dpre, None, alone)


def test_training_runs():
    from gated_ffn import Block
    losses = Block(256, 128, 2, 8).train(normal(1, 96, 256), torch.zeros((96, 128), device="cuda"), 3)
    assert len(losses) == 3 and all(np.isfinite(losses))


def off_by(x, chunks):
    """The same matrix `chunks` x 16 bytes behind a 512-byte boundary, between NaN."""
    t = torch.full((x.numel() + 512,), float("nan"), dtype=bf16, device="cuda")
    v = t[8 * chunks:8 * chunks + x.numel()].view(x.shape)
    v.copy_(x)
    assert v.data_ptr() % 128 == 16 * (chunks % 8)
    return v


@pytest.mark.parametrize("chunks", [0, 1, 6])
@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("tile,M,I,K", [("128x128", 777, 1032, 2056), ("64x64", 777, 1032, 2064), ("128x128", 1300, 456, 2080),
                                        ("64x64", 1300, 456, 2112), ("64x64x2", 300, 264, 1032), ("128x256", 300, 264, 1032), ("256x256", 300, 264, 1032)])
def test_rows_off_the_lines(tile, M, I, K, split, chunks, monkeypatch):
    """Rows and matrices that start at any 16 bytes, with loads enough that the tiles take them by whole lines."""
    monkeypatch.setenv("FP8GEMM_FORCE_CONFIG", "product:%s:%d" % (tile, split))
    X, W, dH = off_by(normal(1, M, K), chunks), off_by(normal(2, 2 * I, K, scale=K ** -0.5), 7 * chunks % 8), off_by(normal(3, M, I), chunks)
    pre, dpre = off_by(torch.zeros((M, 2 * I), dtype=bf16, device="cuda"), chunks), off_by(torch.zeros((M, 2 * I), dtype=bf16, device="cuda"), chunks)
    H = fg.gated_ffn(X, W, pre=pre, out=off_by(torch.zeros((M, I), dtype=bf16, device="cuda"), chunks))
    forward_close(X, W, "silu", H, pre)
    for kept in (pre, None):
        dX, dW = fg.gated_ffn_backward(dH, X, W, pre=kept, dpre=dpre)
        backward_close(dH, X, W, "silu", kept, dpre, dX, dW)
