"""Bounded device waits of the operators around the experts: a wait that runs out
(the producer issues no copies, every wait has 5 ms) ends the kernel, shows in
moe_check_status, writes nothing outside the outputs, and the next call is clean."""
import time

import pytest
import torch

from ffn_plans import PRODUCTS, kind, plan
from mixture_experts_layer_59_b200 import binding as B
from test_gpu_shared_ffn import random_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def expires(call, skip):
    """Runs `call` with its launch number `skip` (of those that wait) starved."""
    B.moe_check_status()
    assert B.lib().moe_debug_expire_later_wait(skip, 5_000_000) == 0
    start = time.monotonic()
    try:
        call()
        with pytest.raises(B.MoEError) as e:
            B.moe_check_status()
    finally:
        B.lib().moe_debug_expire_next_wait(0)  # not left for another test, should nothing have taken it
    assert e.value.code == B.MOE_ERR_DEVICE_TIMEOUT
    assert time.monotonic() - start < 1.0
    B.moe_check_status()                       # the report is taken once


def guarded(t):
    big = torch.full((t.numel() + 512,), 77.0, device="cuda", dtype=t.dtype)
    return big, big[256:256 + t.numel()].view(t.shape)


def intact(bufs):
    return all((big[:256] == 77).all() and (big[-256:] == 77).all() for big, _ in bufs.values())


@pytest.mark.parametrize("T,d,f", [(1493, 4104, 2056), (700, 7168, 2048), (300, 1000, 680), (200, 4096, 2048)])
def test_shared_ffn(T, d, f):
    c = random_case(T, d, f, 8)
    w = (c["w1"], c["w3"], c["w2"])
    y, H = B.moe_shared_ffn_fwd(c["x"], *w, addend=c["add"])
    g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=c["add"])
    ws1, ws2 = (torch.empty(n, device="cuda", dtype=torch.uint8) for n in
                (B.moe_shared_ffn_fwd_workspace_size(T, d, f), B.moe_shared_ffn_bwd_workspace_size(T, d, f)))
    fb = {n: guarded(t) for n, t in (("y", y), ("H", H))}
    gb = {n: guarded(t) for n, t in g.items()}

    def fwd():
        B.moe_shared_ffn_fwd(c["x"], *w, addend=c["add"], H=fb["H"][1], y=fb["y"][1], ws=ws1)

    def bwd():
        B.moe_shared_ffn_bwd(c["dout"], c["x"], *w, H, addend=c["add"], out={n: v for n, (_, v) in gb.items()}, ws=ws2)

    for skip in range(2):
        expires(fwd, skip)
        fwd()
        B.moe_check_status()
        assert torch.equal(fb["y"][1], y) and torch.equal(fb["H"][1], H) and intact(fb), PRODUCTS[skip]
    for skip in range(3):
        expires(bwd, skip)
        bwd()
        B.moe_check_status()
        assert all(torch.equal(gb[n][1], g[n]) for n in g) and intact(gb), PRODUCTS[2 + skip]


def test_sizes_cover_pairs_with_shares_and_clusters():
    kinds = {kind(plan(*s, i)) for s in [(1493, 4104, 2056), (700, 7168, 2048), (300, 1000, 680), (200, 4096, 2048)]
             for i in range(5)}
    assert kinds >= {"shared alike", "shared anywhere", "whole", "split 128 cluster", "split 256 cluster"}


@pytest.mark.parametrize("T,d,dtype", [(5000, 2048, BF), (3000, 1037, BF), (2600, 7168, BF), (2500, 7017, BF),
                                       (1300, 8192, F32), (2500, 601, F32)])
def test_layernorm_backward(T, d, dtype):
    gen = torch.Generator().manual_seed(T + d)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, dy, add, w = n(T, d).to(dtype), n(T, d).to(dtype), n(T, d).to(dtype), n(d)
    _, mean, rstd = B.moe_layernorm_fwd(x, w)
    want = B.moe_layernorm_bwd(dy, x, w, mean, rstd, addend=add)
    bufs = {k: guarded(t) for k, t in want.items()}
    ws = torch.empty(B.moe_layernorm_bwd_workspace_size(T, d), device="cuda", dtype=torch.uint8)

    def call():
        B.moe_layernorm_bwd(dy, x, w, mean, rstd, addend=add, out={k: v for k, (_, v) in bufs.items()}, ws=ws)

    for _ in range(2):
        expires(call, 0)
        call()
        B.moe_check_status()
        assert all(torch.equal(bufs[k][1], want[k]) for k in want) and intact(bufs)
