"""Pins of oracle/block_oracle.py: gradients against central differences, the
generator against its authors' known answers, the mask's layout by hand."""
import numpy as np
import pytest

from oracle import block_oracle as O


def _num_grad(fn, a, eps=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + eps
        hi = fn()
        a[i] = keep - eps
        lo = fn()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_philox_known_answers():
    # the generator's published known-answer vectors (4x32, 10 rounds)
    assert O.philox4x32_10([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert O.philox4x32_10([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert O.philox4x32_10([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344],
                           [0xA4093822, 0x299F31D0]) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_takes_16_bits_per_element_low_half_first():
    # block 0 of seed 0, offset 0: the words of the first known answer
    draws = [0xE8D5, 0x6627, 0xC58D, 0xE169, 0xAC4C, 0xBC57, 0xDBD8, 0x9B00]
    for p in (0.0, 0.25, 0.5, 0.75, 1.0):
        want = [d >= round(p * 65536) for d in draws]
        assert O.dropout_keep(0, 0, 0, 8, p).tolist() == want
    assert O.dropout_keep(0, 0, 3, 5, 0.75).tolist() == [d >= 49152 for d in draws[3:]]


def test_mask_rate_and_mean():
    p = 0.3
    keep = O.dropout_keep(7, 1, 0, 40000, p)
    q = O.dropout_threshold(p) / 65536
    assert abs((1 - keep.mean()) - q) < 5 * np.sqrt(q * (1 - q) / keep.size)
    x = np.ones(keep.size)
    assert abs(O.dropout(x, keep, p).mean() - 1) < 5 * np.sqrt(q / (1 - q) / keep.size)
    assert (O.dropout(x, np.zeros(keep.size, bool), 1.0) == 0).all()


@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_gradient(affine):
    r = np.random.default_rng(0)
    x, dy = r.normal(size=(3, 5)), r.normal(size=(3, 5))
    w = r.normal(size=5) if affine else None
    b = r.normal(size=5) if affine else None
    add = r.normal(size=(3, 5))
    loss = lambda: float((O.layernorm_fwd(x, w, b, 1e-5)[0] * dy).sum() + (x * add).sum())  # noqa: E731
    y, mean, rstd = O.layernorm_fwd(x, w, b, 1e-5)
    dx, dw, db = O.layernorm_bwd(dy, x, w, mean, rstd, add)
    np.testing.assert_allclose(dx, _num_grad(loss, x), rtol=1e-6, atol=1e-8)
    if affine:
        np.testing.assert_allclose(dw, _num_grad(loss, w), rtol=1e-6, atol=1e-8)
        np.testing.assert_allclose(db, _num_grad(loss, b), rtol=1e-6, atol=1e-8)


def test_ffn_gradient():
    r = np.random.default_rng(1)
    x, w1, w3, w2 = (r.normal(size=s) for s in ((3, 4), (4, 5), (4, 5), (5, 4)))
    add, dout = r.normal(size=(3, 4)), r.normal(size=(3, 4))
    loss = lambda: float((O.ffn_fwd(x, w1, w3, w2, add)[0] * dout).sum())  # noqa: E731
    _, H, _ = O.ffn_fwd(x, w1, w3, w2, add)
    g = O.ffn_bwd(dout, x, w1, w3, w2, H)
    for name, a in (("dx", x), ("dw1", w1), ("dw3", w3), ("dw2", w2)):
        np.testing.assert_allclose(g[name], _num_grad(loss, a), rtol=1e-6, atol=1e-8, err_msg=name)
    np.testing.assert_allclose(O.ffn_bwd(dout, x, w1, w3, w2, H, add)["dx"], g["dx"] + add)


def test_silu_of_large_values_stays_finite():
    one = np.ones((1, 1))
    y, H, a = O.ffn_fwd(np.array([[-1000.0]]), one, one, one)
    assert a[0, 0] == 0.0 and np.isfinite(y).all()
