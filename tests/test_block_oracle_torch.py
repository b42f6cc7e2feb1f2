"""oracle/block_oracle.py against torch's own float64 layer norm and automatic
gradients (host only)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O

DOUBLE = dict(rtol=1e-11, atol=1e-11)      # both sides in float64: sums of a few dozen terms


@pytest.mark.parametrize("affine", [True, False])
def test_layernorm(affine):
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(7, 33, generator=gen, dtype=torch.float64).mul_(2).add_(0.5).requires_grad_()
    w, b = (torch.randn(33, generator=gen, dtype=torch.float64).requires_grad_() if affine else None for _ in range(2))
    dy, add = (torch.randn(7, 33, generator=gen, dtype=torch.float64) for _ in range(2))
    y = torch.nn.functional.layer_norm(x, (33,), w, b, eps=1e-5)
    ((y * dy).sum() + (x * add).sum()).backward()
    n = lambda t: None if t is None else t.detach().numpy()  # noqa: E731
    ry, mean, rstd = O.layernorm_fwd(n(x), n(w), n(b), 1e-5)
    np.testing.assert_allclose(ry, n(y), **DOUBLE)
    dx, dw, db = O.layernorm_bwd(n(dy), n(x), n(w), mean, rstd, n(add))
    np.testing.assert_allclose(dx, n(x.grad), **DOUBLE)
    if affine:
        np.testing.assert_allclose(dw, n(w.grad), **DOUBLE)
        np.testing.assert_allclose(db, n(b.grad), **DOUBLE)


def test_gated_ffn():
    gen = torch.Generator().manual_seed(1)
    x, w1, w3, w2 = (torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()
                     for s in ((6, 16), (16, 24), (16, 24), (24, 16)))
    dout, add = (torch.randn(6, 16, generator=gen, dtype=torch.float64) for _ in range(2))
    y = (torch.nn.functional.silu(x @ w1) * (x @ w3)) @ w2 + add
    (y * dout).sum().backward()
    n = lambda t: t.detach().numpy()  # noqa: E731
    ry, H, _ = O.ffn_fwd(n(x), n(w1), n(w3), n(w2), n(add))
    np.testing.assert_allclose(ry, n(y), **DOUBLE)
    g = O.ffn_bwd(n(dout), n(x), n(w1), n(w3), n(w2), H)
    for name, t in (("dx", x), ("dw1", w1), ("dw3", w3), ("dw2", w2)):
        np.testing.assert_allclose(g[name], n(t.grad), err_msg=name, **DOUBLE)


@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout_keeps_the_expected_value_of_the_gradient(p):
    """The gradient through the oracle's mask is the mask times its scale, as autograd has it."""
    keep = O.dropout_keep(3, 4, 0, 500, p)
    x = torch.randn(500, generator=torch.Generator().manual_seed(2), dtype=torch.float64).requires_grad_()
    scale = 65536.0 / (65536.0 - O.dropout_threshold(p))
    out = torch.where(torch.from_numpy(keep), x * scale, torch.zeros((), dtype=torch.float64))
    out.sum().backward()
    np.testing.assert_allclose(O.dropout(x.detach().numpy(), keep, p), out.detach().numpy(), **DOUBLE)
    np.testing.assert_allclose(O.dropout(np.ones(500), keep, p), x.grad.numpy(), **DOUBLE)
