"""Host-side checks of the operators around the experts: bad arguments are
refused before anything is launched (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from mixture_experts_layer_59_b200 import binding as B
from mixture_experts_layer_59_b200.layer import MoEBlockStep

F = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)


def ln_fwd(**kw):
    a = dict(x=F, ldx=256, w=F, b=F, T=4, d=256, dt=B.MOE_BF16, wdt=B.MOE_F32, eps=1e-5, y=F, mean=F, rstd=F)
    a.update(kw)
    return B.lib().moe_layernorm_fwd(*a.values(), None)


def ln_bwd(**kw):
    a = dict(dy=F, lddy=256, x=F, ldx=256, w=F, mean=F, rstd=F, add=None, ldadd=0, T=4, d=256, dt=B.MOE_BF16,
             wdt=B.MOE_F32, dx=F, dw=F, db=F, ws=F, wsb=1 << 30)
    a.update(kw)
    return B.lib().moe_layernorm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), -2), (dict(wdt=-1), -2), (dict(T=-1), -1), (dict(d=0), -1), (dict(eps=-1.0), -1),
    (dict(eps=math.nan), -1), (dict(mean=None), -1), (dict(x=None), -1), (dict(y=None), -1),
    (dict(ldx=255), -1), (dict(x=ODD), -1), (dict(w=ODD), -1), (dict(T=0, x=None, y=None), 0),
])
def test_layernorm_fwd_refusals(kw, code):
    assert ln_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), -2), (dict(wdt=9), -2), (dict(T=-1), -1), (dict(d=-3), -1), (dict(dy=None), -1),
    (dict(mean=None), -1), (dict(rstd=None), -1), (dict(dx=None), -1), (dict(lddy=255), -1),
    (dict(add=F, ldadd=10), -1), (dict(ws=None), -5), (dict(wsb=16), -5), (dict(dx=ODD), -1),
])
def test_layernorm_bwd_refusals(kw, code):
    assert ln_bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(p=-0.01), -1), (dict(p=1.01), -1), (dict(p=math.nan), -1), (dict(dt=3), -2),
    (dict(x=None), -1), (dict(rng=None), -1), (dict(out=None), -1), (dict(x=ODD), -1),
    (dict(rng=ctypes.c_void_p(260)), -1), (dict(n=0, x=None, out=None), 0),
])
def test_dropout_refusals(kw, code):
    a = dict(x=F, res=None, n=100, p=0.1, rng=F, dt=B.MOE_BF16, out=F)
    a.update(kw)
    assert B.lib().moe_dropout_fwd(*a.values(), None) == code
    del a["res"]
    assert B.lib().moe_dropout_bwd(*a.values(), None) == code


def test_binding_refuses_what_it_cannot_launch():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    rng = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: B.moe_layernorm_fwd(x, w),                       # not on a CUDA device
                 lambda: B.moe_layernorm_fwd(x[0], w),                    # not a matrix
                 lambda: B.moe_layernorm_fwd(x, w[:5]),                   # wrong width
                 lambda: B.moe_layernorm_fwd(x.t(), torch.zeros(4)),      # columns contiguous
                 lambda: B.moe_layernorm_fwd(x.half(), w),                # type
                 lambda: B.moe_layernorm_fwd(x, w, w.bfloat16()),         # two parameter types
                 lambda: B.moe_layernorm_bwd(x, x.bfloat16(), w, x[:, 0], x[:, 0]),
                 lambda: B.moe_dropout_fwd(x, 0.1, rng),
                 lambda: B.moe_dropout_fwd(x, 0.1, rng.int()),
                 lambda: B.moe_dropout_fwd(x.t(), 0.1, rng),
                 lambda: B.moe_dropout_fwd(x, 0.1, rng, residual=x[:2])):
        with pytest.raises(B.MoEError):
            call()


def ffn_fwd(**kw):
    a = dict(x=F, w1=F, w3=F, w2=F, add=None, T=4, d=256, f=128, dt=B.MOE_BF16, H=F, y=F, ws=F, wsb=1 << 30)
    a.update(kw)
    return B.lib().moe_shared_ffn_fwd(*a.values(), None)


def ffn_bwd(**kw):
    a = dict(dout=F, x=F, w1=F, w3=F, w2=F, H=F, add=None, T=4, d=256, f=128, dt=B.MOE_BF16, dx=F, dw1=F, dw3=F,
             dw2=F, ws=F, wsb=1 << 30)
    a.update(kw)
    return B.lib().moe_shared_ffn_bwd(*a.values(), None)


SHARED = [(dict(dt=B.MOE_F32), -2), (dict(T=-1), -1), (dict(d=12), -2), (dict(f=4), -2), (dict(d=0), -2),
          (dict(f=-8), -2), (dict(T=1 << 30, d=1 << 20), -2), (dict(d=1 << 20, f=1 << 20), -2), (dict(T=1, d=8, f=1 << 29), -2), (dict(x=None), -1), (dict(w1=None), -1), (dict(w3=None), -1),
          (dict(w2=None), -1), (dict(x=ctypes.c_void_p(264)), -1), (dict(w2=ctypes.c_void_p(258)), -1),
          (dict(add=ctypes.c_void_p(258)), -1), (dict(ws=None), -1), (dict(wsb=8), -5)]


@pytest.mark.parametrize("kw,code", SHARED + [(dict(y=None), -1), (dict(H=ODD), -1), (dict(T=0, x=None, y=None), 0)])
def test_shared_ffn_fwd_refusals(kw, code):
    assert ffn_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [(dict(dout=None), -1), (dict(H=None), -1), (dict(dx=None), -1),
                                              (dict(dw2=None), -1), (dict(dw1=ODD), -1)])
def test_shared_ffn_bwd_refusals(kw, code):
    assert ffn_bwd(**kw) == code


def test_shared_ffn_workspaces():
    for size in (B.lib().moe_shared_ffn_fwd_workspace_size, B.lib().moe_shared_ffn_bwd_workspace_size):
        assert size(0, 256, 128, B.MOE_BF16) == 0 and size(10, 256, 128, B.MOE_F32) == 0
        assert size(1 << 30, 1 << 20, 128, B.MOE_BF16) == 0 and size(10, 12, 128, B.MOE_BF16) == 0
        assert 0 < size(10, 256, 128, B.MOE_BF16) < size(10000, 256, 128, B.MOE_BF16)


def test_binding_refuses_ffn_arguments():
    bf = torch.bfloat16
    x, w1, w2 = torch.zeros(4, 16, dtype=bf), torch.zeros(16, 8, dtype=bf), torch.zeros(8, 16, dtype=bf)
    for call in (lambda: B.moe_shared_ffn_fwd(x, w1, w1, w2),                   # not on a CUDA device
                 lambda: B.moe_shared_ffn_fwd(x, w1, w2, w2),                   # shape
                 lambda: B.moe_shared_ffn_fwd(x, w1, w1, w1.t()),               # not contiguous
                 lambda: B.moe_shared_ffn_fwd(x.float(), w1, w1, w2),           # types differ
                 lambda: B.moe_shared_ffn_fwd(x, w1, w1, w2, addend=x[:2]),
                 lambda: B.moe_shared_ffn_bwd(x, x, w1, w1, w2, torch.zeros(4, 8, dtype=bf))):
        with pytest.raises(B.MoEError):
            call()


def test_layernorm_workspace_covers_every_launch_shape():
    # one partial row of 2 d floats per block: 4 blocks per SM, 6 for narrow rows
    size = B.lib().moe_layernorm_bwd_workspace_size
    assert size(0, 700) == 0
    for d in (1, 33, 256, 257, 700, 1037, 4096, 8192):
        assert size(5, d) == 5 * 2 * d * 4
        assert size(100000, d) == (888 if d <= 256 else 592) * 2 * d * 4
    assert size(1, 8193) == 64 * 2 * 8193 * 4


def test_shared_ffn_workspace_holds_the_activation():
    # the forward's A, the backward's dH and A, each [T, f] or [T, 2f] bf16 at 256-byte steps
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for T, d, f in ((1, 256, 128), (300, 72, 520), (16384, 2048, 1024)):
        assert B.moe_shared_ffn_fwd_workspace_size(T, d, f) >= up(T * f * 2)
        assert B.moe_shared_ffn_bwd_workspace_size(T, d, f) >= up(T * f * 4) + up(T * f * 2)


def test_sizes_past_32_bits_are_refused():
    # ctypes would wrap them; a meta tensor has the shape without the memory
    for shape in ((1 << 32, 8), (8, 1 << 31)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
        with pytest.raises(B.MoEError, match="2.31"):
            B.moe_layernorm_fwd(x)


def test_block_step_host_side():
    T, d, f, E, k, fs = 300, 256, 128, 8, 2, 72
    s = MoEBlockStep(T, d, f, E, k, fs, p=0.1, device="cpu", round_mode=B.MOE_ROUND_NONE)
    assert s.moe.round_mode == B.MOE_ROUND_NONE and s.n.dtype == torch.bfloat16
    assert tuple(s.Hs.shape) == (T, 2 * fs) and s.mean.dtype == torch.float32
    assert s.ws_fwd.numel() == B.moe_shared_ffn_fwd_workspace_size(T, d, fs) > 0
    assert s.ws_bwd.numel() == B.moe_shared_ffn_bwd_workspace_size(T, d, fs) > 0
    assert s.ws_ln.numel() == B.moe_layernorm_bwd_workspace_size(T, d) > 0
    assert tuple(s.ffn_grads["dw2"].shape) == (fs, d) and tuple(s.ln_grads["dbias"].shape) == (d,)
    with pytest.raises(ValueError, match="bf16"):
        MoEBlockStep(T, d, f, E, k, fs, device="cpu", dtype=torch.float32)
    for bad in (0, -8, 12):
        with pytest.raises(ValueError, match="multiples of 8"):
            MoEBlockStep(T, d, f, E, k, bad, device="cpu")
    x = torch.zeros(T, d, dtype=torch.bfloat16)
    with pytest.raises(B.MoEError, match="CUDA device"):
        s.forward(x, (None, None), (), (), torch.zeros(2, dtype=torch.int64))
