"""GPU: the gated feed-forward block in bf16 and its gradients against a plain 64-bit implementation.

Tolerances.  A rounding to bf16 is off by 2^-9 of the value at most where it is not at the end of its binade
(2^-8 bounds it everywhere).  A sum of n products in fp32, in any order the kernels use, is off by n 2^-24 sum |x w|
at most; with errors of either sign that is some sqrt(n) 2^-24 in practice, and 2^-18 sum |x w| bounds it for the
lengths here (the matrix cores keep at least fp32's 24 bits in a step of 32 products).  The activations move with
their argument by at most 1.13 (gelu) or 1.1 (silu), and are formed within 2^-21 of |g|.
Gradients: dg = dh u act'(g) moves by |dh| |act'| per u (|act'| <= 1.13) and by |dh u| |act''| per g (|act''| <= 1.2);
dpre is rounded to bf16, so a sum over it is off by 2^-8 sum |dpre| |w| at most, which 2^-9 sum + the tolerance of
independent roundings would leave far below; the bound is used as it stands."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU runs deselect these with -m "not gpu"
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_block_scaled_x128_amd as fg  # noqa: E402

SUM = 2.0 ** -18


def normal(seed, *shape, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def act64(g, act):
    """act(g) and act'(g) in 64 bits."""
    if act == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        a = 2 * np.sqrt(2 / np.pi)
        z, dz = a * (g + 0.044715 * g ** 3), a * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(z)
    return g * s, s + g * s * (1 - s) * dz


def within(got, ref, tol):
    assert torch.isfinite(got).all()
    err = (got.double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + tol + 1e-30).all(), float((err / (ref.abs() + tol + 1e-30)).max())


def products(X, W):
    """g, u and the sums of their terms' sizes."""
    x, w = X.double(), W.double()
    return (x @ w.t()).chunk(2, dim=1), (x.abs() @ w.abs().t()).chunk(2, dim=1)


def forward_close(X, W, act, H, pre):
    (g, u), (sg, su) = products(X, W)
    a, _ = act64(g, act)
    within(H, a * u, SUM * (1.13 * sg * u.abs() + a.abs() * su) + 2.0 ** -20 * (g * u).abs())
    if pre is not None:
        within(pre, torch.cat((g, u), 1), SUM * torch.cat((sg, su), 1))


# few rows (a kernel of its own up to 64), and tiles with every kind of end
SIZES = [(1, 8, 8), (1, 2048, 512), (2, 40, 72), (3, 24, 1000), (16, 64, 128), (17, 16, 320), (33, 104, 200), (64, 8, 2056),
         (65, 72, 136), (100, 512, 64), (128, 128, 8), (257, 136, 1032), (300, 1416, 456), (1000, 264, 520)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,I,K", SIZES)
def test_forward(M, I, K, act):
    X, W = normal(M, M, K), normal(I, 2 * I, K, scale=K ** -0.5)
    pre = torch.full((M + 1, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((M + 1, I), 7.0, dtype=torch.bfloat16, device="cuda")
    fg.gated_ffn(X, W, act=act, pre=pre[:M], out=out[:M])
    forward_close(X, W, act, out[:M], pre[:M])
    assert (pre[M:] == 7).all() and (out[M:] == 7).all()           # rows behind the last stay
    alone = fg.gated_ffn(X, W, act=act)
    assert torch.equal(alone, out[:M])


def backward_close(dH, X, W, act, pre, dpre, dX, dW):
    (g, u), (sg, su) = products(X, W)
    tg, tu = SUM * sg, SUM * su
    if pre is not None:
        g, u = pre.double().chunk(2, dim=1)
        tg = tu = torch.zeros_like(g)
    d = dH.double()
    a, da = act64(g, act)
    dp = torch.cat((d * u * da, d * a), 1)
    dtol = torch.cat((d.abs() * (1.13 * tu + 1.2 * u.abs() * tg) + 2.0 ** -20 * (d * u).abs() * (1 + g.abs()),
                      d.abs() * (1.13 * tg) + 2.0 ** -20 * (d * g).abs()), 1)
    within(dpre, dp, dtol)
    # the sums are over dpre as it was rounded
    r = dpre.double()
    if dX is not None:
        within(dX, r @ W.double(), SUM * (r.abs() @ W.double().abs()))
    if dW is not None:
        within(dW, r.t() @ X.double(), SUM * (r.abs().t() @ X.double().abs()))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("M,I,K", SIZES)
def test_backward(M, I, K, act, kept):
    X, W, dH = normal(M, M, K), normal(I, 2 * I, K, scale=K ** -0.5), normal(K, M, I)
    pre = None
    if kept:
        pre = torch.empty((M, 2 * I), dtype=torch.bfloat16, device="cuda")
        fg.gated_ffn(X, W, act=act, pre=pre)
    full = {n: torch.full((r + 1, c), 7.0, dtype=torch.bfloat16, device="cuda")
            for n, r, c in (("dpre", M, 2 * I), ("dX", M, K), ("dW", 2 * I, K))}
    o = {n: t[:-1] for n, t in full.items()}
    dX, dW = fg.gated_ffn_backward(dH, X, W, pre=pre, act=act, **o)
    backward_close(dH, X, W, act, pre, o["dpre"], dX, dW)
    assert all((t[-1] == 7).all() for t in full.values())
    # one gradient alone, and dpre in the place of pre
    only, none = fg.gated_ffn_backward(dH, X, W, pre=pre, act=act, need_dW=False)
    assert none is None
    backward_close(dH, X, W, act, pre, o["dpre"], only, None)
    place = None if pre is None else pre.clone()
    none, only = fg.gated_ffn_backward(dH, X, W, pre=place, act=act, dpre=place, need_dX=False)
    assert none is None and (place is None or torch.equal(place, o["dpre"]))
    backward_close(dH, X, W, act, pre, o["dpre"], None, only)
