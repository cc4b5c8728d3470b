"""The autograd function of examples/gated_ffn.py, with the library's calls replaced by plain ones.  CPU only."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_ffn  # noqa: E402


class Plain:
    """silu, without a graph, as the library's calls are."""

    @staticmethod
    def gated_ffn(x, w, act, pre=None):
        with torch.no_grad():
            p = x @ w.t()
            if pre is not None:
                pre.copy_(p)
            g, u = p.chunk(2, dim=1)
            return torch.nn.functional.silu(g) * u

    @staticmethod
    def gated_ffn_backward(dh, x, w, pre=None, act="silu", need_dX=True, need_dW=True):
        with torch.no_grad():
            g, u = (x @ w.t()).chunk(2, dim=1)
            s = torch.sigmoid(g)
            dp = torch.cat((dh * u * (s + g * s * (1 - s)), dh * g * s), 1)
            return dp @ w if need_dX else None, dp.t() @ x if need_dW else None


@pytest.mark.parametrize("keep", [True, False])
def test_a_second_derivative_is_refused(keep, monkeypatch):
    """The gradients have no graph of their own: what would be differentiated through them raises, instead of leaving out
    their part of it."""
    monkeypatch.setattr(gated_ffn, "fg", Plain)
    gen = torch.Generator().manual_seed(1)
    x, w = (torch.randn(s, generator=gen, dtype=torch.float64).requires_grad_() for s in ((3, 8), (16, 8)))
    assert torch.autograd.gradcheck(lambda a, b: gated_ffn.GatedFfn.apply(a, b, "silu", keep), (x, w))
    h = gated_ffn.GatedFfn.apply(x, w, "silu", keep)
    dx, dw = torch.autograd.grad(h.sum(), (x, w), create_graph=True)
    for grad, at in ((dx, x), (dw, w)):
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad((grad * at).sum(), at)
