"""Calls of the operators around the experts that their documentation allows and
that are not part of a step: results in place, outputs left out, one tensor in
two places, very many rows, generator blocks past 2^32."""
import ctypes

import pytest
import torch

from mixture_experts_layer_59_b200 import binding as B
from oracle import block_oracle as O
from test_gpu_norm_dropout import check_ln
from test_gpu_shared_ffn import random_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def give_memory_back():
    """The large buffers of a test are not kept from those after it."""
    yield
    torch.cuda.empty_cache()


def need(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(4000, 1037), (3000, 7017), (5000, 33), (3000, 255), (2500, 2046), (3, 70001), (6000, 2048)])
def test_layernorm_in_place_of_many_rows(T, d, dtype):
    """Rows that share 16-byte units with their neighbours, each result where its row was."""
    gen = torch.Generator().manual_seed(d)
    x = (torch.randn(T, d, generator=gen) * 2 + 0.5).to(dtype).cuda()
    w, b = torch.randn(d, generator=gen).cuda(), torch.randn(d, generator=gen).cuda()
    y, mean, rstd = B.moe_layernorm_fwd(x, w, b)
    for _ in range(5):
        buf = torch.full((T * d + 64,), 5.0, device="cuda", dtype=dtype)
        off = x.data_ptr() % 16 // x.element_size() + 16
        z = buf[off:off + T * d].view(T, d).copy_(x)
        _, m, r = B.moe_layernorm_fwd(z, w, b, y=z)
        assert torch.equal(z, y) and torch.equal(m, mean) and torch.equal(r, rstd)
        assert (buf[:off] == 5).all() and (buf[off + T * d:] == 5).all()


@pytest.mark.parametrize("T,d", [(40, 384), (5000, 2048), (20, 9000)])
def test_layernorm_outputs_left_out(T, d):
    gen = torch.Generator().manual_seed(T)
    x, dy = (torch.randn(T, d, generator=gen).cuda() for _ in range(2))
    w = torch.randn(d, generator=gen).cuda()
    y, mean, rstd = B.moe_layernorm_fwd(x, w)
    want = B.moe_layernorm_bwd(dy, x, w, mean, rstd)
    y2 = torch.empty_like(y)
    assert B.lib().moe_layernorm_fwd(p(x), d, p(w), None, T, d, B.MOE_F32, B.MOE_F32, 1e-5, p(y2), None, None, stream()) == 0
    assert torch.equal(y2, y)
    ws = torch.empty(B.moe_layernorm_bwd_workspace_size(T, d), device="cuda", dtype=torch.uint8)
    for dw, db in ((True, False), (False, True), (False, False)):
        dx = torch.empty_like(x)
        gw, gb = torch.full((d,), 3.0, device="cuda"), torch.full((d,), 3.0, device="cuda")
        none = not (dw or db)
        rc = B.lib().moe_layernorm_bwd(p(dy), d, p(x), d, p(w), p(mean), p(rstd), None, 0, T, d, B.MOE_F32, B.MOE_F32,
                                       p(dx), p(gw) if dw else None, p(gb) if db else None, None if none else p(ws),
                                       0 if none else ws.numel(), stream())
        assert rc == 0
        assert torch.equal(dx, want["dx"])
        assert torch.equal(gw, want["dweight"]) if dw else bool((gw == 3).all())
        assert torch.equal(gb, want["dbias"]) if db else bool((gb == 3).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [2367, 2368, 2369])
def test_layernorm_where_the_launch_shape_changes(T, dtype):
    """Row counts around 16 warps per SM, widths around each share of a warp
    (tolerances: those of the norm's tests)."""
    gen = torch.Generator().manual_seed(T)
    for d in (30, 62, 64, 66, 126, 128, 254, 255, 256, 257, 258, 510, 512, 514, 1022, 1023, 1024, 1025):
        x = (torch.randn(T, d, generator=gen) * 2 + 0.5).to(dtype).cuda()
        check_ln(x, torch.randn(d, generator=gen).cuda(), torch.randn(d, generator=gen).cuda())


def test_layernorm_of_most_rows():
    """2^31 - 1 rows of one column: the variance is 0, y = bias exactly; the backward
    pass's xh = 0, so dx = dy w - mean(dy w) = 0 (times a finite rstd) and
    dweight = 0, dbias = the sum of dy = 1 in every third row."""
    T = (1 << 31) - 1
    need(60)
    x = torch.full((T, 1), 1.5, device="cuda", dtype=BF)
    b = torch.tensor([0.25], device="cuda")
    y, mean, rstd = B.moe_layernorm_fwd(x, None, b)
    step = 1 << 28
    for i in range(0, T, step):
        s = slice(i, i + step)
        assert bool((y[s] == 0.25).all()) and bool((mean[s] == 1.5).all()) and bool((rstd[s] == rstd[0]).all()), i
    dy = y.zero_()
    dy[::3] = 1
    dx = torch.full((T, 1), 7.0, device="cuda", dtype=BF)
    g = B.moe_layernorm_bwd(dy, x, None, mean, rstd, out=dict(dx=dx))
    for i in range(0, T, step):
        assert not g["dx"][i:i + step].any(), i
    # a thread's ones are a whole number below 2^24; the blocks' 888 sums and
    # their 32 columns join with fewer than 64 roundings
    n = (T + 2) // 3
    assert float(g["dweight"]) == 0.0 and abs(float(g["dbias"]) - n) <= 64 * 2.0 ** -24 * n


def test_shared_ffn_with_one_tensor_in_two_places():
    """w1 as w3 and x as dout and as the addend."""
    T, d, f = 300, 264, 136
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(T, d, generator=gen).to(BF).cuda()
    w1 = (torch.randn(d, f, generator=gen) * d ** -0.5).to(BF).cuda()
    w2 = (torch.randn(f, d, generator=gen) * f ** -0.5).to(BF).cuda()
    y, H = B.moe_shared_ffn_fwd(x, w1, w1, w2, addend=x)
    g = B.moe_shared_ffn_bwd(x, x, w1, w1, w2, H, addend=x)
    y2, H2 = B.moe_shared_ffn_fwd(x, w1, w1.clone(), w2, addend=x.clone())
    g2 = B.moe_shared_ffn_bwd(x.clone(), x, w1, w1.clone(), w2, H2, addend=x.clone())
    assert torch.equal(y, y2) and torch.equal(H, H2) and all(torch.equal(g[n], g2[n]) for n in g)
    assert torch.equal(H[:, :f], H[:, f:])


def test_dropout_blocks_past_32_bits():
    """More than 2^35 elements: generator blocks past 2^32, whose number's upper word
    is not zero.  In place (64 GB)."""
    n = (1 << 35) + 4099
    need(66)
    x = torch.ones(n, device="cuda", dtype=BF)
    rng = torch.tensor([123, 45], device="cuda")
    B.moe_dropout_bwd(x, 0.5, rng, dx=x)
    for lo, hi in ((0, 1000), ((1 << 32) - 500, (1 << 32) + 500), ((1 << 35) - 1000, (1 << 35) + 1000), (n - 3000, n)):
        keep = O.dropout_keep(123, 45, lo, hi - lo, 0.5)
        assert (x[lo:hi].double().cpu().numpy() == keep * 2.0).all(), lo
    # the blocks' upper word matters: those past 2^32 do not repeat the first ones
    assert not torch.equal(x[1 << 35:], x[:4099])
    # and by single elements
    y = x[1:n - 3]
    y.fill_(1.0)
    B.moe_dropout_fwd(y, 0.5, rng, out=y)
    m = y.numel()
    for lo, hi in ((0, 1000), ((1 << 35) - 1000, (1 << 35) + 1000), (m - 3000, m)):
        keep = O.dropout_keep(123, 45, lo, hi - lo, 0.5)
        assert (y[lo:hi].double().cpu().numpy() == keep * 2.0).all(), lo


def test_shared_ffns_and_norms_on_three_streams_at_once():
    """Pairs with shared tiles, clusters and a norm's backward pass in flight together,
    each with buffers of its own: the results they have alone."""
    jobs = []
    for T, d, f in ((1493, 4104, 2056), (300, 1000, 680), (700, 7168, 2048)):
        c = random_case(T, d, f, T)
        gen = torch.Generator().manual_seed(T)
        x, dy, w = (torch.randn(*s, generator=gen).cuda() for s in ((4000, 1037), (4000, 1037), (1037,)))

        def job(c=c, x=x, dy=dy, w=w, **at):
            ws = (c["w1"], c["w3"], c["w2"])
            y, H = B.moe_shared_ffn_fwd(c["x"], *ws, addend=c["add"], **at)
            g = B.moe_shared_ffn_bwd(c["dout"], c["x"], *ws, H, addend=c["add"], **at)
            n, mean, rstd = B.moe_layernorm_fwd(x, w, **at)
            return [y, H, n, *g.values(), *B.moe_layernorm_bwd(dy, x, w, mean, rstd, **at).values()]
        jobs.append((job, job(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [job(stream=s) for job, _, s in jobs]
        torch.cuda.synchronize()
        for (_, want, _), out in zip(jobs, got):
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    B.moe_check_status()
