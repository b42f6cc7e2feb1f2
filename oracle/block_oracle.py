"""CPU oracle of the operators around the routed experts (test infrastructure
only): layer norm, counter-based dropout and the shared gated feed-forward
block, forward and backward, in numpy float64 from their formulas.  It shares
no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ layer norm
def layernorm_fwd(x, weight, bias, eps):
    """y, mean, rstd of each row; weight / bias None: ones / zeros."""
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layernorm_bwd(dy, x, weight, mean, rstd, addend=None):
    """dx, dweight, dbias."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    if addend is not None:
        dx = dx + addend
    return dx, (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------------ dropout
def philox4x32_10(counter, key):
    """The generator of Salmon et al. (2011), one block, in Python integers:
    counter of four and key of two 32-bit words -> four 32-bit words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_threshold(p):
    return int(np.rint(p * 65536.0))


def dropout_keep(seed, offset, first, count, p):
    """Which of the elements first .. first + count - 1 are kept."""
    thr = dropout_threshold(p)
    words = {}
    out = np.zeros(count, bool)
    lo = 0xFFFFFFFF
    for n in range(count):
        i = first + n
        b = i >> 3
        if b not in words:
            words[b] = philox4x32_10((b & lo, b >> 32, offset & lo, (offset >> 32) & lo),
                                     (seed & lo, (seed >> 32) & lo))
        out[n] = ((words[b][(i & 7) >> 1] >> (16 * (i & 1))) & 0xFFFF) >= thr
    return out


def dropout(x, keep, p, residual=None):
    """residual + keep * x / (1 - q), q the threshold's share of 65536."""
    thr = dropout_threshold(p)
    out = np.zeros_like(x)
    if thr < 65536:
        out[keep] = x[keep] * (65536.0 / (65536.0 - thr))
    return out if residual is None else out + residual


# ------------------------------------------------------------------ gated FFN
def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def ffn_fwd(x, w1, w3, w2, addend=None):
    """H = [x W1 | x W3], A = silu(H1) * H3, y = A W2 (+ addend): y, H, A."""
    h1, h3 = x @ w1, x @ w3
    a = h1 * _sigmoid(h1) * h3
    y = a @ w2
    return (y if addend is None else y + addend), np.concatenate([h1, h3], 1), a


def ffn_bwd(dout, x, w1, w3, w2, H, addend=None):
    """Gradients from dout and H = [H1 | H3] as given."""
    f = w1.shape[1]
    h1, h3 = H[:, :f], H[:, f:]
    s = _sigmoid(h1)
    a = h1 * s * h3
    da = dout @ w2.T
    dh1, dh3 = da * h3 * s * (1.0 + h1 * (1.0 - s)), da * h1 * s
    dx = dh1 @ w1.T + dh3 @ w3.T
    return dict(dx=dx if addend is None else dx + addend, dw1=x.T @ dh1, dw3=x.T @ dh3,
                dw2=a.T @ dout, a=a, da=da, dh1=dh1, dh3=dh3)
