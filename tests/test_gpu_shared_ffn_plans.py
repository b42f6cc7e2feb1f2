"""The shared FFN at every cut that its planner can choose for each product
(tests/test_shared_ffn_plan.py asserts that the sizes here cover them):
exact results, outputs in place of the addends, guard bands, workspaces full
of NaN."""
import numpy as np
import pytest
import torch

from ffn_plans import EXACT_SIZES, GUARD_SIZES
from mixture_experts_layer_59_b200 import binding as B
from test_gpu_shared_ffn import exact_case, random_case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
GRADS = ("dx", "dw1", "dw3", "dw2")


@pytest.mark.parametrize("T,d,f", EXACT_SIZES)
def test_exact(T, d, f):
    """One-hot rows of x, W1 = 32, small integers elsewhere: H, A and dH are
    integers that bf16 holds, every sum stays an integer below 2^24, so a result
    is the exact sum rounded once.  A wrong, missing or doubled part of a tile
    changes it."""
    c = exact_case(T, d, f, T + d + f)
    w = (c["w1"], c["w3"], c["w2"])
    y, H = B.moe_shared_ffn_fwd(c["x"], *w, addend=c["add"])
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=c["add"])
    B.moe_check_status()
    x, w1, w3, w2, do, add = (c[n].double() for n in ("x", "w1", "w3", "w2", "dout", "add"))
    h1, h3 = x @ w1, x @ w3                       # h1 = 32: silu 32, its slope 1
    da = do @ w2.T
    d1, d3, A = da * h3, da * 32, 32 * h3
    assert torch.equal(d1.to(BF).double(), d1) and torch.equal(d3.to(BF).double(), d3)
    ref = dict(y=A @ w2, dx=d1 @ w1.T + d3 @ w3.T, dw1=x.T @ d1, dw3=x.T @ d3, dw2=A.T @ do)
    assert max(float(r.abs().max()) for r in ref.values()) < 2 ** 24
    plain = {n: ref[n].to(BF) for n in ("y", "dx")}
    ref["y"], ref["dx"] = ref["y"] + add, ref["dx"] + add
    assert torch.equal(H.double(), torch.cat([h1, h3], 1))
    for n, got in dict(g, y=y).items():
        assert torch.equal(got, ref[n].to(BF)), n
    # the results where the addends were, H not written; without an addend
    a = c["add"].clone()
    assert torch.equal(B.moe_shared_ffn_fwd(c["x"], *w, addend=a, y=a, save=False)[0], y)
    a = c["add"].clone()
    again = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=a, out=dict(dx=a))
    assert all(torch.equal(again[n], g[n]) for n in g)
    assert torch.equal(B.moe_shared_ffn_fwd(c["x"], *w)[0], plain["y"])
    assert torch.equal(B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H)["dx"], plain["dx"])
    B.moe_check_status()


def guarded(*shape, fill=77.0):
    n = int(np.prod(shape))
    big = torch.full((n + 256,), fill, device="cuda", dtype=BF)
    return big, big[128:128 + n].view(*shape)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,d,f", GUARD_SIZES)
def test_guard_bands_and_dirty_workspaces(T, d, f, add):
    """Nothing is written outside the outputs and the workspace; NaN in the
    workspace and in the outputs beforehand does not reach the results."""
    c = random_case(T, d, f, 5)
    w = (c["w1"], c["w3"], c["w2"])
    addend = c["add"] if add else None
    y, H = B.moe_shared_ffn_fwd(c["x"], *w, addend=addend)
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=addend)
    bufs = {n: guarded(*s) for n, s in (("y", (T, d)), ("H", (T, 2 * f)), ("dx", (T, d)), ("dw1", (d, f)),
                                        ("dw3", (d, f)), ("dw2", (f, d)))}
    for _, view in bufs.values():
        view.fill_(float("nan"))
    n1, n2 = B.moe_shared_ffn_fwd_workspace_size(T, d, f), B.moe_shared_ffn_bwd_workspace_size(T, d, f)
    ws1, ws2 = (torch.full((n + 4096,), 0xFF, device="cuda", dtype=torch.uint8) for n in (n1, n2))
    for _ in range(2):          # the second time over what the first left
        B.moe_shared_ffn_fwd(c["x"], *w, addend=addend, H=bufs["H"][1], y=bufs["y"][1], ws=ws1[:n1])
        B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, bufs["H"][1], addend=addend,
                             out={n: bufs[n][1] for n in GRADS}, ws=ws2[:n2])
        B.moe_check_status()
        for n, ref in dict(g, y=y, H=H).items():
            big, view = bufs[n]
            assert torch.equal(view, ref), n
            assert (big[:128] == 77).all() and (big[-128:] == 77).all(), n
        assert (ws1[n1:] == 0xFF).all() and (ws2[n2:] == 0xFF).all()
