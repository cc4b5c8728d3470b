"""Refusals of the routing, token permutation and 4-bit product entry points: bad arguments are
rejected on the host before any device work.  CPU only (no GPU needed, no compute calls)."""
import os

import pytest

import fp8_block_scaled_x128_amd as fg

FAKE = 1 << 20          # aligned non-null address; never dereferenced by the validation paths
NULL, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fg.library_path()):
        from fp8_block_scaled_x128_amd import build
        build.build()
    return fg.lib()


def test_route_refusals(lib):
    def call(logits=FAKE, bias=None, ids=FAKE, w=FAKE, T=4, E=64, k=8, dtype=0, score=0, n_group=1, topk_group=1,
             group_top=1, renorm=1, scale=1.0):
        return lib.fp8gemm_route_topk(logits, bias, ids, w, T, E, k, dtype, score, n_group, topk_group, group_top, renorm,
                                      scale, None)
    assert call(T=0) == 0 and call(T=0, logits=None, ids=None, w=None) == 0
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=65), dict(dtype=2), dict(score=2), dict(n_group=0), dict(n_group=5),
                dict(topk_group=0), dict(n_group=4, topk_group=5), dict(n_group=8, topk_group=1, k=9), dict(scale=float("nan")),
                dict(n_group=8, topk_group=2, group_top=3), dict(n_group=8, topk_group=2, group_top=0),
                dict(n_group=64, topk_group=16, group_top=2)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(E=1025), dict(E=256, k=33), dict(E=128, n_group=128, topk_group=64)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=None), dict(ids=None), dict(w=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(logits=FAKE + 2), dict(logits=FAKE + 1, dtype=1), dict(bias=FAKE + 2), dict(ids=FAKE + 1), dict(w=FAKE + 3)):
        assert call(**bad) == ALIGN, bad


def test_route_backward_refusals(lib):
    def call(logits=FAKE, ids=FAKE, dw=FAKE, dx=FAKE, T=4, E=64, k=8, dtype=0, score=0, renorm=1, scale=1.0):
        return lib.fp8gemm_route_topk_backward(logits, ids, dw, dx, T, E, k, dtype, score, renorm, scale, None)
    assert call(T=0) == 0
    for bad in (dict(T=-1), dict(E=0), dict(k=65), dict(dtype=3), dict(score=-1), dict(scale=float("inf"))):
        assert call(**bad) == SHAPE, bad
    assert call(E=2000) == UNSUPPORTED
    for bad in (dict(logits=None), dict(ids=None), dict(dw=None), dict(dx=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(logits=FAKE + 2), dict(dx=FAKE + 1, dtype=1), dict(ids=FAKE + 2), dict(dw=FAKE + 2)):
        assert call(**bad) == ALIGN, bad


@pytest.mark.parametrize("name", ["masked", "contiguous"])
def test_dispatch_refusals(lib, name):
    f = getattr(lib, "fp8gemm_moe_dispatch_" + name)

    def call(X=FAKE, ids=FAKE, A=FAKE, sa=FAKE, where=FAKE, rows=FAKE, T=4, H=256, k=2, G=4, cap=128, first=0):
        return f(X, ids, A, sa, where, rows, T, H, k, G, cap, first, None)
    for bad in (dict(T=-1), dict(H=0), dict(H=200), dict(k=0), dict(G=0), dict(cap=-1), dict(first=-1)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(k=33), dict(G=1025), dict(T=1 << 30), dict(T=1 << 62), dict(H=1 << 25), dict(cap=1 << 31),
                dict(cap=1 << 40)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=None), dict(ids=None), dict(A=None), dict(sa=None), dict(where=None), dict(rows=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(X=FAKE + 8), dict(A=FAKE + 8), dict(sa=FAKE + 2), dict(ids=FAKE + 2), dict(where=FAKE + 1),
                dict(rows=FAKE + 2)):
        assert call(**bad) == ALIGN, bad


def test_combine_refusals(lib):
    def call(Y=FAKE, w=FAKE, rows=FAKE, out=FAKE, T=4, H=64, k=2, R=100):
        return lib.fp8gemm_moe_combine(Y, w, rows, out, T, H, k, R, None)
    assert call(T=0) == 0
    for bad in (dict(T=-1), dict(H=0), dict(H=12), dict(k=0), dict(R=-1), dict(rows=None, R=7)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(k=33), dict(T=1 << 62), dict(R=1 << 31), dict(H=1 << 25)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(Y=None) == NULL and call(out=None) == NULL
    for bad in (dict(Y=FAKE + 8), dict(out=FAKE + 8), dict(w=FAKE + 2), dict(rows=FAKE + 2)):
        assert call(**bad) == ALIGN, bad

    def back(dout=FAKE, Y=FAKE, w=FAKE, rows=FAKE, dY=FAKE, dw=FAKE, T=4, H=64, k=2, R=100):
        return lib.fp8gemm_moe_combine_backward(dout, Y, w, rows, dY, dw, T, H, k, R, None)
    assert back(T=0) == 0
    for bad in (dict(dout=None), dict(Y=None), dict(dY=None)):
        assert back(**bad) == NULL, bad
    for bad in (dict(dout=FAKE + 8), dict(dY=FAKE + 4), dict(dw=FAKE + 2)):
        assert back(**bad) == ALIGN, bad
    assert back(H=20) == SHAPE


def test_w4_refusals(lib):
    def call(X=FAKE, W=FAKE, s=FAKE, z=None, Y=FAKE, M=1, N=64, K=256, fmt=1, group=64):
        return lib.fp8gemm_w4_gemv(X, W, s, z, Y, M, N, K, fmt, group, None)
    assert call(M=0) == 0 and call(N=0) == 0
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=96), dict(fmt=2), dict(group=16), dict(group=256), dict(fmt=0, group=64),
                dict(fmt=0, group=32, z=FAKE), dict(fmt=0, group=32, K=48)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(K=1 << 23), dict(M=(1 << 20) + 1), dict(N=1 << 25), dict(M=1 << 62)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=None), dict(W=None), dict(s=None), dict(Y=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(X=FAKE + 8), dict(W=FAKE + 8), dict(Y=FAKE + 8), dict(s=FAKE + 2), dict(z=FAKE + 1)):
        assert call(**bad) == ALIGN, bad

    def experts(X=FAKE, W=FAKE, s=FAKE, z=None, ids=FAKE, Y=FAKE, T=2, k=2, E=4, N=64, K=256, fmt=1, group=64, first=0,
                per_pair=0, swiglu=0):
        return lib.fp8gemm_w4_gemv_experts(X, W, s, z, ids, Y, T, k, E, N, K, fmt, group, first, per_pair, swiglu, None)
    assert experts(T=0) == 0
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(first=-1), dict(N=63, swiglu=1), dict(K=100)):
        assert experts(**bad) == SHAPE, bad
    for bad in (dict(T=1 << 30, k=2), dict(E=65535), dict(T=1 << 22, K=1 << 10, group=128)):
        assert experts(**bad) == UNSUPPORTED, bad
    assert experts(ids=None) == NULL and experts(ids=FAKE + 2) == ALIGN


def test_binding_rejects_bad_tensors():
    import torch
    with pytest.raises(ValueError):          # host tensors are refused: no CPU path exists
        fg.route_topk(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        fg.w4_gemv(torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.uint8),
                   torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        fg.moe_dispatch_masked(torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32), 2, 8)


def test_short_path_refuses_anything():
    """The compiled calls take any arguments without touching memory: wrong counts, types and host tensors
    come back as a refusal."""
    import torch
    calls = fg._calls()
    host = torch.zeros(4, 8)
    for name, n in (("route_topk", 12), ("route_topk_backward", 8), ("moe_dispatch", 11), ("moe_combine", 5),
                    ("moe_combine_backward", 7), ("w4_gemv", 6), ("w4_gemv_experts", 9)):
        f = getattr(calls, name)
        for count in (0, 1, n - 1, n, n + 1):
            for value in (None, 3, "x", host, torch.zeros(0), 1 << 70, float("nan")):
                assert f(*[value] * count) == -1
