"""The block step (norm, routed and shared experts, dropout, residual) as it is
used: forward and backward against the oracles in 64 bits, and as a graph."""
import numpy as np
import pytest
import torch

from helpers import assert_close, f64
from mixture_experts_layer_59_b200 import binding as B
from mixture_experts_layer_59_b200.layer import MoEBlockStep
from oracle import block_oracle as O
from oracle import moe_oracle as M

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5


def bf(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.float32).to(BF).to(torch.float64).numpy()


def inputs(T, d, f, E, fs, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0, dt=BF: (torch.randn(*s, generator=g) * std + mean).to(dt).cuda()  # noqa: E731
    return dict(x=n(T, d, std=2.0, mean=0.3), dy=n(T, d), ln=(n(d, std=0.1, mean=1.0, dt=torch.float32),
                                                             n(d, std=0.1, dt=torch.float32)),
                experts=(n(d, E, std=0.05), n(E, d, f, std=0.05), n(E, d, f, std=0.05), n(E, f, d, std=0.05)),
                shared=(n(d, fs, std=0.05), n(d, fs, std=0.05), n(fs, d, std=0.05)),
                logits=torch.randn(T, E, generator=g).cuda(), rng=torch.tensor([99, 7], device="cuda"))


@pytest.mark.parametrize("T,d,f,E,k,fs,p", [(384, 256, 256, 8, 2, 192, 0.1), (1, 128, 128, 4, 2, 72, 0.0),
                                            (700, 256, 128, 16, 4, 520, 0.3)])
def test_block_step(T, d, f, E, k, fs, p):
    c = inputs(T, d, f, E, fs, T + d)
    step = MoEBlockStep(T, d, f, E, k, fs, p=p, eps=EPS)
    y = step.forward(c["x"], c["ln"], c["experts"], c["shared"], c["rng"], logits_override=c["logits"])
    g = step.backward(c["dy"])
    B.moe_check_status()
    x, dy = f64(c["x"]), f64(c["dy"])
    w, b = map(f64, c["ln"])
    n, mean, rstd = O.layernorm_fwd(x, w, b, EPS)
    n = bf(n)
    fwd = M.layer_fwd(n, *map(f64, c["experts"]), k, logits_override=f64(c["logits"]), staged=True)
    sw = tuple(map(f64, c["shared"]))
    h, H, _ = O.ffn_fwd(n, *sw)
    m = bf(h + bf(fwd["out"]))
    keep = O.dropout_keep(99, 7, 0, T * d, p).reshape(T, d)
    assert_close(y, O.dropout(m, keep, p, x), "y")
    dm = bf(O.dropout(dy, keep, p))
    bwd = M.layer_bwd(dm, n, *map(f64, c["experts"]), fwd, staged=True, router_grad_on=False)
    # staged as the kernels store it: A and dH in bf16
    sb = O.ffn_bwd(dm, n, *sw, bf(H))
    d1, d3 = bf(sb["dh1"]), bf(sb["dh3"])
    sb = dict(dw1=n.T @ d1, dw3=n.T @ d3, dw2=bf(sb["a"]).T @ dm,
              dx=d1 @ sw[0].T + d3 @ sw[1].T + bf(bwd["dx"]))
    # the rounded n on both sides may differ in its last bit where the norm sits
    # between two bf16 values: the gradients then differ by rounding alone
    for name in ("dw1", "dw3", "dw2"):
        assert_close(g[name], bwd[name], name)
        assert_close(g["shared_" + name[1:]], sb[name], "shared " + name)
    dx, dw, db = O.layernorm_bwd(bf(sb["dx"]), x, w, mean, rstd, dy)
    # dn went through three bf16 sums (experts, shared, its store): half a step
    # each of 2^-8 in the mean is 3 x 0.35 x 2^-8 = 4e-3 of dn's magnitude
    assert_close(g["dx"], dx, "dx", (2e-2, 5e-3))
    # sums over T tokens of independent roundings of dn (and of n): for T = 1 that of one
    assert_close(g["ln_weight"], dw, "ln_weight", (2e-2, 8e-3))
    assert_close(g["ln_bias"], db, "ln_bias", (2e-2, 8e-3))


def test_block_capture_and_rng():
    T, d, f, E, k, fs = 300, 256, 128, 8, 2, 256
    c = inputs(T, d, f, E, fs, 3)
    args = (c["x"], c["ln"], c["experts"], c["shared"], c["rng"])
    eager = MoEBlockStep(T, d, f, E, k, fs, p=0.2)
    step = MoEBlockStep(T, d, f, E, k, fs, p=0.2)
    graph = step.capture(*args, c["dy"])
    last = None
    for offset in (1, 2, 1):
        c["rng"][1] = offset
        graph.replay()
        y = eager.forward(*args)
        g = eager.backward(c["dy"])
        torch.cuda.synchronize()
        assert torch.equal(step.y, y) and torch.equal(step.ln_grads["dx"], g["dx"])
        assert torch.equal(step.ffn_grads["dw2"], g["shared_w2"])
        assert torch.equal(step.moe.grads["dw1"], g["dw1"])
        assert last is None or not torch.equal(y, last)
        last = y.clone()
    B.moe_check_status()


def test_block_on_two_streams_at_once():
    """Two steps with their own buffers, in flight together, each as alone."""
    T, d, f, E, k, fs = 900, 256, 128, 8, 2, 512
    cs = [inputs(T, d, f, E, fs, s) for s in (4, 5)]
    steps = [MoEBlockStep(T, d, f, E, k, fs, p=0.2) for _ in cs]
    want = []
    for c, s in zip(cs, steps):
        y = s.forward(c["x"], c["ln"], c["experts"], c["shared"], c["rng"])
        g = s.backward(c["dy"])
        want.append((y.clone(), g["dx"].clone(), g["shared_w1"].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        for c, s, st in zip(cs, steps, streams):
            s.forward(c["x"], c["ln"], c["experts"], c["shared"], c["rng"], stream=st)
        for c, s, st in zip(cs, steps, streams):
            s.backward(c["dy"], stream=st)
        torch.cuda.synchronize()
        for s, (y, dx, w1) in zip(steps, want):
            assert torch.equal(s.y, y) and torch.equal(s.ln_grads["dx"], dx)
            assert torch.equal(s.ffn_grads["dw1"], w1)
    B.moe_check_status()
