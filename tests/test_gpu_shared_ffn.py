"""The shared gated FFN against the oracle in 64 bits.

Three kinds of checks.
 - Exact: inputs whose every intermediate is a small integer (times 32), so
   that all sums are exact in fp32 and all results in bf16; a wrong or missing
   index anywhere changes a result.  W1 = 32 makes silu(h1) = 32 and
   silu'(h1) = 1 exactly (the sigmoid of 32 rounds to 1 in fp32).
 - Staged: random inputs, the oracle rounding H, A and dH to bf16 where the
   kernels do; the tolerance the library states for bf16, 1e-2 of the largest
   value and 2e-3 of the mean magnitude.
 - Bound: random inputs against the unstaged formulas, element by element.
   h = 2^-8 (1 + 2^-7) bounds a bf16 rounding of a value that already carries
   small errors; an accumulation of K products errs by at most
   ACC(K) = (K / 16 + 16) 2^-22 times the sum of the products' magnitudes;
   |silu'| <= 1.1; the fast sigmoid is within 2^-18 relative.
"""
import numpy as np
import pytest
import torch

from helpers import BF16_TOL, assert_close
from mixture_experts_layer_59_b200 import binding as B
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H_ = 2.0 ** -8 * (1 + 2.0 ** -7)

SHAPES = [(1, 8, 8), (1, 2048, 1024), (2, 64, 72), (5, 16, 264), (31, 136, 200), (64, 1152, 320), (96, 2048, 512),
          (127, 128, 128), (128, 256, 256), (129, 264, 136), (200, 512, 1024), (300, 1000, 680), (513, 2048, 256),
          (1500, 1000, 680), (2500, 384, 1024), (4000, 640, 128)]


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def acc(k):
    return (k / 16 + 16) * 2.0 ** -22


def bf(a):
    """Round a numpy array to bf16 (nearest even) and back."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.float32).to(BF).to(torch.float64).numpy()


def sparse_int(gen, *shape, density, values=(-1.0, 1.0)):
    v = torch.tensor(values)[torch.randint(len(values), shape, generator=gen)]
    return (v * (torch.rand(*shape, generator=gen) < density)).to(BF).cuda()


def exact_case(T, d, f, seed):
    """x one-hot, W1 = 32, W3, W2, dout in {-1, 0, 1}."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, d)
    x[torch.arange(T), torch.randint(d, (T,), generator=g)] = 1
    w1 = torch.full((d, f), 32.0)
    dens = min(1.0, 64.0 / f)
    return dict(x=x.to(BF).cuda(), w1=w1.to(BF).cuda(), w3=sparse_int(g, d, f, density=0.7),
                w2=sparse_int(g, f, d, density=dens), dout=sparse_int(g, T, d, density=min(1.0, 32.0 / d)),
                add=(32 * torch.randint(-3, 4, (T, d), generator=g)).to(BF).cuda())


@pytest.mark.parametrize("T,d,f", SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_exact(T, d, f, add):
    c = exact_case(T, d, f, T + d + f)
    w = (c["w1"], c["w3"], c["w2"])
    addend = c["add"] if add else None
    y, H = B.moe_shared_ffn_fwd(c["x"], *w, addend=addend)
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=addend)
    B.moe_check_status()
    ry, rH, _ = O.ffn_fwd(f64(c["x"]), *map(f64, w), f64(addend))
    r = O.ffn_bwd(f64(c["dout"]), f64(c["x"]), *map(f64, w), rH, f64(addend))
    np.testing.assert_array_equal(f64(H), rH)
    for name, got, ref in [("y", y, ry)] + [(n, g[n], r[n]) for n in ("dx", "dw1", "dw3", "dw2")]:
        ref = np.rint(ref)          # the oracle's sigmoid is a hair below 1
        ok = bf(ref) == ref         # (a rare sum past 8 bits rounds: compared rounded)
        assert ok.mean() > 0.99, name
        np.testing.assert_array_equal(f64(got), bf(ref), err_msg=name)
    y2, H2 = B.moe_shared_ffn_fwd(c["x"], *w, addend=addend, save=False)
    assert H2 is None and torch.equal(y2, y)


@pytest.mark.parametrize("T,d,f", [(10000, 2048, 640), (3000, 1024, 2048), (5000, 2048, 512), (8000, 512, 512),
                                   (4321, 1992, 1352), (19000, 256, 136)])
def test_exact_many_rows(T, d, f):
    """The sizes that CTA pairs compute, with shared last tiles in every product."""
    c = exact_case(T, d, f, T + d + f)
    y, H = B.moe_shared_ffn_fwd(c["x"], c["w1"], c["w3"], c["w2"], addend=c["add"])
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], c["w1"], c["w3"], c["w2"], H, addend=c["add"])
    B.moe_check_status()
    x, w1, w3, w2, do, add = (c[n].double() for n in ("x", "w1", "w3", "w2", "dout", "add"))
    h1, h3 = x @ w1, x @ w3                       # h1 = 32: silu 32, its slope 1
    da = do @ w2.T
    d1, d3, A = da * h3, da * 32, 32 * h3
    assert d1.abs().max() <= 256                  # dH is exact in bf16
    ref = dict(y=A @ w2 + add, dx=d1 @ w1.T + d3 @ w3.T + add, dw1=x.T @ d1, dw3=x.T @ d3, dw2=A.T @ do)
    assert torch.equal(H.double(), torch.cat([h1, h3], 1))
    for n, got in dict(g, y=y).items():
        assert ((ref[n].to(BF).double() == ref[n]).double().mean()) > 0.99, n
        assert torch.equal(got, ref[n].to(BF)), n
    # the results where the addends were, and without an addend
    w = (c["w1"], c["w3"], c["w2"])
    a = c["add"].clone()
    assert torch.equal(B.moe_shared_ffn_fwd(c["x"], *w, addend=a, y=a, save=False)[0], y)
    a = c["add"].clone()
    again = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=a, out=dict(dx=a))
    assert all(torch.equal(again[n], g[n]) for n in g)
    y = B.moe_shared_ffn_fwd(c["x"], *w)[0]
    dx = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H)["dx"]
    assert torch.equal(y, (A @ w2).to(BF)) and torch.equal(dx, (d1 @ w1.T + d3 @ w3.T).to(BF))


def test_exact_offsets_past_32_bits():
    """H and dH of more than 2^31 elements."""
    T, d, f = 600000, 8, 2048
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    c = exact_case(T, d, f, 1)
    y, H = B.moe_shared_ffn_fwd(c["x"], c["w1"], c["w3"], c["w2"], addend=c["add"])
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], c["w1"], c["w3"], c["w2"], H, addend=c["add"])
    B.moe_check_status()
    w1, w3, w2 = (c[n].double() for n in ("w1", "w3", "w2"))
    dw = dict.fromkeys(("dw1", "dw3", "dw2"), 0.0)
    for i in range(0, T, 50000):                  # as in test_exact_many_rows, rows by rows
        r = slice(i, i + 50000)
        x, do, add = (c[n][r].double() for n in ("x", "dout", "add"))
        h1, h3 = x @ w1, x @ w3
        da = do @ w2.T
        d1, d3, A = da * h3, da * 32, 32 * h3
        assert torch.equal(H[r].double(), torch.cat([h1, h3], 1)), i
        assert torch.equal(y[r], (A @ w2 + add).to(BF)), i
        assert torch.equal(g["dx"][r], (d1 @ w1.T + d3 @ w3.T + add).to(BF)), i
        dw = dict(dw1=dw["dw1"] + x.T @ d1, dw3=dw["dw3"] + x.T @ d3, dw2=dw["dw2"] + A.T @ do)
    for n, ref in dw.items():
        assert torch.equal(g[n], ref.to(BF)), n


def random_case(T, d, f, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF).cuda()  # noqa: E731
    return dict(x=n(T, d), w1=n(d, f, std=scale * d ** -0.5), w3=n(d, f, std=d ** -0.5), w2=n(f, d, std=f ** -0.5),
                dout=n(T, d), add=n(T, d))


@pytest.mark.parametrize("T,d,f", SHAPES)
def test_staged_and_bound(T, d, f):
    c = random_case(T, d, f, 7 * T + d + f, scale=3.0)
    w = (c["w1"], c["w3"], c["w2"])
    y, H = B.moe_shared_ffn_fwd(c["x"], *w, addend=c["add"])
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=c["add"])
    B.moe_check_status()
    X, W1, W3, W2, DO, ADD = (f64(c[n]) for n in ("x", "w1", "w3", "w2", "dout", "add"))
    _, rH, _ = O.ffn_fwd(X, W1, W3, W2, ADD)
    # H: one accumulation, one rounding
    eH = acc(d) * (np.abs(X) @ np.abs(np.concatenate([W1, W3], 1))) + H_ * np.abs(rH)
    assert (np.abs(f64(H) - rH) <= eH).all()
    # y, staged: A is rounded once, from the unrounded H
    ry, _, A = O.ffn_fwd(X, W1, W3, W2, ADD)
    assert_close(y, bf(bf(A) @ W2 + ADD), "y", BF16_TOL)
    # y, unstaged, element by element
    e13 = acc(d) * (np.abs(X) @ np.abs(W1)), acc(d) * (np.abs(X) @ np.abs(W3))
    sl = np.abs(rH[:, :f]) * O._sigmoid(rH[:, :f])
    eA = 1.1 * e13[0] * (np.abs(rH[:, f:]) + e13[1]) + sl * e13[1] + (H_ + 2.0 ** -17) * np.abs(A)
    ey = eA @ np.abs(W2) + acc(f) * ((np.abs(A) + eA) @ np.abs(W2)) + 2.0 ** -22 * np.abs(ADD) + 2 * H_ * np.abs(ry)
    assert (np.abs(f64(y) - ry) <= ey + H_ * ey).all()
    # backward from the kernel's own H, staged
    h1, h3 = f64(H)[:, :f], f64(H)[:, f:]
    sg = O._sigmoid(h1)
    A = h1 * sg * h3
    sA, eA = bf(A), (H_ + 2.0 ** -17) * np.abs(A)
    r = O.ffn_bwd(DO, X, W1, W3, W2, f64(H), ADD)
    d1, d3 = bf(r["dh1"]), bf(r["dh3"])
    staged = dict(dx=bf(d1 @ W1.T + d3 @ W3.T + ADD), dw1=bf(X.T @ d1), dw3=bf(X.T @ d3), dw2=bf(sA.T @ DO))
    for n, ref in staged.items():
        assert_close(g[n], ref, n, BF16_TOL)
    # backward, unstaged, element by element
    eda = acc(d) * (np.abs(DO) @ np.abs(W2).T)
    gd1, gd3 = h3 * sg * (1 + h1 * (1 - sg)), h1 * sg
    # 1 - sigmoid of the fast sigmoid carries its error undamped: |h3 h1| 2^-18 more
    e1 = eda * np.abs(gd1) + (np.abs(r["da"]) + eda) * np.abs(h3) * (1 + np.abs(h1)) * 2.0 ** -17 + 2 * H_ * np.abs(r["dh1"])
    e3 = eda * np.abs(gd3) + (np.abs(r["da"]) + eda) * np.abs(gd3) * 2.0 ** -17 + 2 * H_ * np.abs(r["dh3"])
    m1, m3 = np.abs(r["dh1"]) + e1, np.abs(r["dh3"]) + e3
    bounds = dict(dx=e1 @ np.abs(W1).T + e3 @ np.abs(W3).T + 2 * acc(f) * (m1 @ np.abs(W1).T + m3 @ np.abs(W3).T)
                  + 2.0 ** -22 * np.abs(ADD),
                  dw1=np.abs(X).T @ e1 + acc(T) * (np.abs(X).T @ m1), dw3=np.abs(X).T @ e3 + acc(T) * (np.abs(X).T @ m3),
                  dw2=eA.T @ np.abs(DO) + acc(T) * ((np.abs(A) + eA).T @ np.abs(DO)))
    for n, e in bounds.items():
        assert (np.abs(f64(g[n]) - r[n]) <= (e + 2 * H_ * np.abs(r[n])) * (1 + H_)).all(), n


def test_gradient_against_differences():
    """The kernels' gradients against differences of the kernels' own forward pass
    along random directions (bf16 results: a loose but independent check)."""
    T, d, f = 160, 128, 192
    c = random_case(T, d, f, 11)
    names = ("x", "w1", "w3", "w2")
    y, H = B.moe_shared_ffn_fwd(*(c[n] for n in names))
    g = B.moe_shared_ffn_bwd(c["dout"], *(c[n] for n in names), H)
    grads = dict(x=g["dx"], w1=g["dw1"], w3=g["dw3"], w2=g["dw2"])
    loss = lambda a: float((B.moe_shared_ffn_fwd(*a)[0].double() * c["dout"].double()).sum())  # noqa: E731
    for i, n in enumerate(names):
        gen = torch.Generator().manual_seed(20 + i)
        # along the gradient itself plus noise: the derivative is then far from zero
        step = (grads[n].float() / grads[n].float().norm()
                + 0.1 * torch.randn(c[n].shape, generator=gen).cuda() / c[n].numel() ** 0.5)
        size = 0.02 * c[n].float().norm()
        args = [c[m] for m in names]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = (c[n].float() + size * step).to(BF), (c[n].float() - size * step).to(BF)
        num = loss(hi) - loss(lo)
        ana = float((grads[n].double() * (hi[i].double() - lo[i].double())).sum())
        # rounding: each y is off by 2^-8 at most, summed over T d terms at random
        noise = 4 * 2.0 ** -8 * float((y.double().abs() * c["dout"].double().abs()).square().sum().sqrt())
        assert abs(num - ana) <= 0.05 * abs(ana) + noise, (n, num, ana, noise)


def test_no_rows_and_outputs_in_place():
    c = random_case(70, 256, 128, 3)
    w = (c["w1"], c["w3"], c["w2"])
    y, H = B.moe_shared_ffn_fwd(c["x"], *w, addend=c["add"])
    a = c["add"].clone()
    assert torch.equal(B.moe_shared_ffn_fwd(c["x"], *w, addend=a, y=a)[0], y)
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=c["add"])
    a = c["add"].clone()
    assert torch.equal(B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=a, out=dict(dx=a))["dx"], g["dx"])
    e = c["x"][:0]
    y0, H0 = B.moe_shared_ffn_fwd(e, *w)
    assert y0.shape == (0, 256) and H0.shape == (0, 256)
    out = dict(dw1=torch.ones(256, 128, device="cuda", dtype=BF))
    g0 = B.moe_shared_ffn_bwd(e, e, *w, H0, out=out)
    assert not any(g0[n].any() for n in ("dw1", "dw3", "dw2")) and g0["dx"].shape == (0, 256)


def test_bad_rows_stay_their_own():
    """NaN and infinite rows of x spoil their own row of y and dx only."""
    c = random_case(150, 200, 136, 4)
    w = (c["w1"], c["w3"], c["w2"])
    clean = B.moe_shared_ffn_fwd(c["x"], *w)
    gclean = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, clean[1])
    x = c["x"].clone()
    x[17, 3], x[140, 199] = float("nan"), float("inf")
    y, H = B.moe_shared_ffn_fwd(x, *w)
    good = [i for i in range(150) if i not in (17, 140)]
    assert torch.equal(y[good], clean[0][good]) and torch.isnan(y[17]).all()
    g = B.moe_shared_ffn_bwd(c["dout"], x, *w, H)
    assert torch.equal(g["dx"][good], gclean["dx"][good])


@pytest.mark.parametrize("T,d,f", [(3, 136, 72), (130, 264, 200), (700, 256, 384)])
def test_guard_bands_and_dirty_workspaces(T, d, f):
    """Nothing is written outside the outputs and the workspace, and what the
    workspace holds beforehand (NaN here) does not reach the results."""
    c = random_case(T, d, f, 5)
    w = (c["w1"], c["w3"], c["w2"])

    def guarded(*shape):
        n = int(np.prod(shape))
        big = torch.full((n + 256,), 77.0, device="cuda", dtype=BF)
        return big, big[128:128 + n].view(*shape)

    def dirty(n):
        return torch.full((n + 512,), 0xFF, device="cuda", dtype=torch.uint8)

    y, H = B.moe_shared_ffn_fwd(c["x"], *w)
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H)
    bufs = {n: guarded(*s) for n, s in (("y", (T, d)), ("H", (T, 2 * f)), ("dx", (T, d)), ("dw1", (d, f)),
                                        ("dw3", (d, f)), ("dw2", (f, d)))}
    n1 = B.lib().moe_shared_ffn_fwd_workspace_size(T, d, f, B.MOE_BF16)
    n2 = B.lib().moe_shared_ffn_bwd_workspace_size(T, d, f, B.MOE_BF16)
    ws1, ws2 = dirty(n1), dirty(n2)
    B.moe_shared_ffn_fwd(c["x"], *w, H=bufs["H"][1], y=bufs["y"][1], ws=ws1[:n1])
    B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, bufs["H"][1],
                         out={n: bufs[n][1] for n in ("dx", "dw1", "dw3", "dw2")}, ws=ws2[:n2])
    B.moe_check_status()
    for n, ref in dict(g, y=y, H=H).items():
        big, view = bufs[n]
        assert torch.equal(view, ref), n
        assert (big[:128] == 77).all() and (big[-128:] == 77).all(), n
    assert (ws1[n1:] == 0xFF).all() and (ws2[n2:] == 0xFF).all()


@pytest.mark.parametrize("T,d,f", [(1, 256, 128), (260, 512, 256), (3000, 1024, 2048)])
def test_captured_graph_replays_on_new_inputs_and_another_stream(T, d, f):
    a, b = random_case(T, d, f, 6), random_case(T, d, f, 7)
    names = ("x", "w1", "w3", "w2")
    wsf = torch.empty(B.lib().moe_shared_ffn_fwd_workspace_size(T, d, f, B.MOE_BF16), device="cuda", dtype=torch.uint8)
    wsb = torch.empty(B.lib().moe_shared_ffn_bwd_workspace_size(T, d, f, B.MOE_BF16), device="cuda", dtype=torch.uint8)
    want = []
    for c in (a, b):
        y, H = B.moe_shared_ffn_fwd(*(c[n] for n in names), addend=c["add"])
        want.append((y, B.moe_shared_ffn_bwd(c["dout"], *(c[n] for n in names), H, addend=c["add"])))
    s = {n: t.clone() for n, t in a.items()}
    H, y = torch.empty(T, 2 * f, device="cuda", dtype=BF), torch.empty(T, d, device="cuda", dtype=BF)
    out = dict(dx=torch.empty(T, d, device="cuda", dtype=BF), dw1=torch.empty(d, f, device="cuda", dtype=BF),
               dw3=torch.empty(d, f, device="cuda", dtype=BF), dw2=torch.empty(f, d, device="cuda", dtype=BF))

    def step():
        B.moe_shared_ffn_fwd(*(s[n] for n in names), addend=s["add"], H=H, y=y, ws=wsf)
        B.moe_shared_ffn_bwd(s["dout"], *(s[n] for n in names), H, addend=s["add"], out=out, ws=wsb)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        step()
    for c, (wy, wg) in ((b, want[1]), (a, want[0])):
        for n in s:
            s[n].copy_(c[n])
        graph.replay()
        assert torch.equal(y, wy) and all(torch.equal(out[n], wg[n]) for n in out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        y2, H2 = B.moe_shared_ffn_fwd(*(b[n] for n in names), addend=b["add"], stream=side)
        g2 = B.moe_shared_ffn_bwd(b["dout"], *(b[n] for n in names), H2, addend=b["add"], stream=side)
        junk = [torch.full((T, 2 * f), float("nan"), device="cuda", dtype=BF) for _ in range(6)]
        side.synchronize()
        assert torch.equal(y2, want[1][0]) and all(torch.equal(g2[n], want[1][1][n]) for n in g2)
        del junk


def test_bounded_wait_expires_then_next_call_is_clean():
    c = random_case(300, 256, 256, 8)
    w = (c["w1"], c["w3"], c["w2"])
    y, _ = B.moe_shared_ffn_fwd(c["x"], *w)
    assert B.lib().moe_debug_expire_next_wait(5_000_000) == 0
    B.moe_shared_ffn_fwd(c["x"], *w)
    with pytest.raises(B.MoEError) as e:
        B.moe_check_status()
    assert e.value.code == B.MOE_ERR_DEVICE_TIMEOUT
    assert torch.equal(B.moe_shared_ffn_fwd(c["x"], *w)[0], y)
    B.moe_check_status()
