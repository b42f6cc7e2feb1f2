"""Layer norm and dropout against the oracle in 64 bits.

Tolerances.  Let u = 2^-24 (half a step of fp32) and h = half a step of the
output type, finfo(t).eps / 2 (fp32 2^-24, bf16 2^-8).
 - A row's sums run over at most 64 terms in a thread, 5 shuffles and 32
   warps: fewer than 128 roundings, so mean and the sums of the backward pass
   are within 128 u of the sum of their terms' magnitudes, rstd within 128 u
   of itself (half of the variance's error plus the root and the division).
   Each result then takes a handful of further roundings: 256 u times the
   sum of the magnitudes of its terms bounds them all, plus h times the
   result for the last rounding.
 - dweight, dbias: a thread adds at most T / 64 rows, then at most 888 / 32
   partial rows and 32 column slices; with T <= 4000 fewer than 128
   roundings: 256 u times the sum of the terms' magnitudes.
 - dropout: the scale, the product and the sum round once each: 4 u times the
   magnitudes plus h times the result; the mask is exact.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_59_b200 import binding as B
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, tol, name):
    got = f64(got)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside; worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.2f} times the tolerance")


def draw(gen, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * std + mean).to(dtype).cuda()


def check_ln(x, w, b, eps=1e-5, dy=None, add=None):
    y, mean, rstd = B.moe_layernorm_fwd(x, w, b, eps=eps)
    X, Wt, Bi = f64(x), f64(w), f64(b)
    ry, rm, rr = O.layernorm_fwd(X, Wt, Bi, eps)
    absw = 1.0 if Wt is None else np.abs(Wt)
    absb = 0.0 if Bi is None else np.abs(Bi)
    mabs = np.abs(X).mean(1)
    within(mean, rm, 128 * U * mabs, "mean")
    # the mean's error shifts the centred values: second order in the variance, covered by mabs * rstd
    within(rstd, rr, 256 * U * rr * (1 + (mabs * rr * 128 * U)), "rstd")
    tol = 256 * U * (np.abs(ry) + 2 * absb + (mabs * rr)[:, None] * absw) + half_step(x.dtype) * np.abs(ry)
    within(y, ry, tol, "y")
    if dy is None:
        return
    g = B.moe_layernorm_bwd(dy, x, w, mean, rstd, addend=add)
    DY, A = f64(dy), f64(add)
    m, r = f64(mean), f64(rstd)
    dx, dw, db = O.layernorm_bwd(DY, X, Wt, m, r, A)
    xh = (X - m[:, None]) * r[:, None]
    G = DY * (1.0 if Wt is None else Wt)
    # xh itself is one difference and one product of fp32 values: |x| and |mean| enter its error
    axh = (np.abs(X) + np.abs(m)[:, None]) * r[:, None]
    mag = r[:, None] * (np.abs(G) + np.abs(G).mean(1, keepdims=True)
                        + axh * (np.abs(G) * axh).mean(1, keepdims=True))
    mag = mag + (0.0 if A is None else np.abs(A))
    within(g["dx"], dx, 256 * U * mag + half_step(x.dtype) * np.abs(dx), "dx")
    within(g["dweight"], dw, 256 * U * (np.abs(DY) * axh).sum(0), "dweight")
    within(g["dbias"], db, 256 * U * np.abs(DY).sum(0), "dbias")


SHAPES = [(1, 1), (1, 7168), (3, 2), (5, 31), (64, 33), (129, 128), (300, 250), (17, 1000), (37, 1037),
          (1000, 256), (450, 2048), (700, 1536), (40, 4096), (33, 4104), (20, 7168), (9, 8191),
          (12, 8192), (3, 8200), (2, 12345), (2, 70000), (4000, 64), (3001, 256), (2999, 1536), (1500, 2048),
          (2500, 2056), (800, 4096), (700, 7168), (650, 8192), (620, 8184), (5000, 2048), (4800, 512), (9500, 128), (2600, 7168), (1300, 8192),
          (9600, 33), (5000, 339), (3000, 1037), (3100, 1038), (2400, 2046), (1300, 4341), (2500, 7017), (1250, 8183)]


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,d", SHAPES)
def test_layernorm(T, d, dtype, wdtype):
    gen = torch.Generator().manual_seed(T * 100003 + d)
    x = draw(gen, T, d, dtype=dtype, std=2.0, mean=0.5)
    w, b = draw(gen, d, dtype=wdtype, std=0.2, mean=1.0), draw(gen, d, dtype=wdtype)
    dy = draw(gen, T, d, dtype=dtype)
    check_ln(x, w, b, dy=dy, add=draw(gen, T, d, dtype=dtype) if d % 3 else None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [1, 2, 3, 8, 15, 16, 17, 31, 32, 40, 63, 64, 72, 100, 128, 129, 130, 200, 255, 256])
def test_layernorm_many_narrow_rows(d, dtype):
    """Rows of less than a warp's width, several to a warp; the last warp not full."""
    gen = torch.Generator().manual_seed(d)
    for T in (2369, 4099):
        x, dy = draw(gen, T, d, dtype=dtype, std=2.0, mean=0.5), draw(gen, T, d, dtype=dtype)
        check_ln(x, draw(gen, d, std=0.2, mean=1.0), draw(gen, d), dy=dy, add=draw(gen, T, d, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_layernorm_without_weight_or_bias(dtype, w, b):
    gen = torch.Generator().manual_seed(5)
    x, dy = draw(gen, 100, 384, dtype=dtype), draw(gen, 100, 384, dtype=dtype)
    check_ln(x, draw(gen, 384) if w else None, draw(gen, 384) if b else None, dy=dy)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,pad,skip", [(256, 8, 0), (256, 8, 8), (256, 3, 1), (255, 2, 1), (128, 1, 0), (8200, 8, 0)])
def test_layernorm_row_strides_and_alignment(dtype, d, pad, skip):
    """Rows inside a wider matrix, starting at any element."""
    gen = torch.Generator().manual_seed(d + pad + skip)
    cut = lambda: draw(gen, 50, d + pad + skip, dtype=dtype)[:, skip:skip + d]  # noqa: E731
    check_ln(cut(), draw(gen, d), draw(gen, d), dy=cut(), add=cut())
    # weights that start at an odd element
    check_ln(cut(), draw(gen, d + 1)[1:], draw(gen, d + 1)[1:], dy=cut(), add=cut())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,pad,skip", [(9600, 128, 3, 1), (9601, 128, 8, 8), (5001, 16, 8, 0), (5001, 33, 5, 2),
                                          (4003, 200, 8, 4), (3000, 1000, 8, 4), (3000, 1001, 8, 3), (3000, 1001, 5, 0),
                                          (2500, 1029, 8, 3), (2500, 2053, 8, 7)])
def test_layernorm_many_rows_inside_a_wider_matrix(T, d, pad, skip, dtype):
    """Each array at an offset of its own, NaN all around the rows."""
    gen = torch.Generator().manual_seed(T + d + pad + skip)

    def cut(k):
        big = torch.full((T + 2, d + pad + 8), float("nan"), dtype=dtype, device="cuda")
        view = big[1:T + 1, k:k + d]
        view.copy_(draw(gen, T, d, dtype=dtype))
        return view

    check_ln(cut(skip), draw(gen, d), draw(gen, d), dy=cut((skip + 1) % 8), add=cut((2 * skip + 5) % 8))
    # x and y at the same offset in their 16 bytes
    x = cut(skip)
    if (x.stride(0) - d) % 8 == 0:
        buf = torch.full((T * d + 32,), 7.0, dtype=dtype, device="cuda")
        off = (x.data_ptr() - buf.data_ptr()) // x.element_size() % (16 // x.element_size())
        y = B.moe_layernorm_fwd(x, y=buf[off:off + T * d].view(T, d))[0]
        ref = O.layernorm_fwd(f64(x), None, None, 1e-5)[0]
        within(y, ref, 256 * U * (np.abs(ref) + 2) + half_step(dtype) * np.abs(ref), "y")
        assert (buf[:off] == 7).all() and (buf[off + T * d:] == 7).all()


@pytest.mark.parametrize("T,d", [(3000, 1002), (4000, 510), (2500, 2046), (1300, 3002), (1300, 7014)])
def test_layernorm_many_rows_at_even_offsets(T, d):
    """bf16 rows at 4-byte units, each array at another one, NaN all around the rows."""
    gen = torch.Generator().manual_seed(T + d)

    def cut(k):
        big = torch.full((T + 2, d + 10), float("nan"), dtype=BF16, device="cuda")
        view = big[1:T + 1, k:k + d]
        view.copy_(draw(gen, T, d, dtype=BF16))
        return view

    check_ln(cut(2), draw(gen, d), draw(gen, d), dy=cut(4), add=cut(6))


@pytest.mark.parametrize("d", [63, 64, 512, 511, 1031])
def test_layernorm_offsets_past_32_bits(d):
    """Rows 2^20 elements apart, 2400 of them: element offsets past 2^31."""
    T, ld = 2400, 1 << 20
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    gen = torch.Generator().manual_seed(d)
    big = torch.empty(T, ld, dtype=BF16, device="cuda")
    x, dy, add = big[:, 16:16 + d], big[:, 4096:4096 + d], big[:, 8192:8192 + d]
    for t in (x, dy, add):
        t.copy_(draw(gen, T, d, dtype=BF16))
    check_ln(x, draw(gen, d), draw(gen, d), dy=dy, add=add)


def test_layernorm_offset_does_not_cancel():
    """A mean a thousand times the deviation: the variance comes from centred values."""
    gen = torch.Generator().manual_seed(3)
    check_ln(draw(gen, 64, 2048, std=1.0, mean=1000.0), draw(gen, 2048), draw(gen, 2048),
             dy=draw(gen, 64, 2048))


def test_layernorm_constant_rows_and_bad_rows():
    """A constant row gives y = bias exactly; a NaN or infinite row stays its own."""
    gen = torch.Generator().manual_seed(4)
    x = draw(gen, 8, 512)
    x[1] = 3.0
    x[3, 7] = float("nan")
    x[5, 9] = float("inf")
    w, b = draw(gen, 512), draw(gen, 512)
    y, mean, rstd = B.moe_layernorm_fwd(x, w, b)
    assert torch.equal(y[1], b)
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    good = [0, 1, 2, 4, 6, 7]
    ref = O.layernorm_fwd(f64(x[good]), f64(w), f64(b), 1e-5)[0]
    np.testing.assert_allclose(f64(y[good]), ref, rtol=1e-4, atol=1e-4)
    dy = draw(gen, 8, 512)
    g = B.moe_layernorm_bwd(dy, x, w, mean, rstd)
    assert torch.isfinite(g["dx"][good]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layernorm_in_place_and_no_rows(dtype):
    gen = torch.Generator().manual_seed(6)
    x, w, b = draw(gen, 77, 640, dtype=dtype), draw(gen, 640), draw(gen, 640)
    want = B.moe_layernorm_fwd(x, w, b)[0]
    z = x.clone()
    assert torch.equal(B.moe_layernorm_fwd(z, w, b, y=z)[0], want)
    e = x[:0]
    y, mean, rstd = B.moe_layernorm_fwd(e, w, b)
    assert y.shape == (0, 640) and mean.shape == (0,)
    g = B.moe_layernorm_bwd(e, e, w, mean, rstd)
    assert g["dx"].shape == (0, 640) and not g["dweight"].any() and not g["dbias"].any()


def test_layernorm_same_result_every_time_and_guarded_outputs():
    """Deterministic column sums; nothing is written outside the outputs."""
    gen = torch.Generator().manual_seed(8)
    for T, d, dtype in ((1000, 1037, F32), (3000, 256, BF16), (200, 2048, BF16), (1000, 700, BF16), (2000, 601, F32),
                        (900, 768, F32), (3000, 2047, BF16), (1300, 7015, BF16), (700, 8192, F32)):
        x, dy, w = draw(gen, T, d, dtype=dtype), draw(gen, T, d, dtype=dtype), draw(gen, d)
        _, mean, rstd = B.moe_layernorm_fwd(x, w)
        first = B.moe_layernorm_bwd(dy, x, w, mean, rstd)
        wsb = B.moe_layernorm_bwd_workspace_size(T, d)
        ws = torch.full((wsb + 512,), 0x7B, device="cuda", dtype=torch.uint8)
        big = torch.full((T * d + 64,), 123.0, device="cuda", dtype=dtype)
        dwb = torch.full((2, d + 16), 55.0, device="cuda")
        out = dict(dx=big[32:32 + T * d].view(T, d), dweight=dwb[0, :d], dbias=dwb[1, :d])
        g = B.moe_layernorm_bwd(dy, x, w, mean, rstd, out=out, ws=ws[:wsb])
        for n in ("dx", "dweight", "dbias"):
            assert torch.equal(g[n], first[n]), n
        assert (big[:32] == 123).all() and (big[32 + T * d:] == 123).all()
        assert (dwb[:, d:] == 55).all() and (ws[wsb:] == 0x7B).all()


# ------------------------------------------------------------------ dropout
def rng_of(seed, offset):
    s = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([s(seed), s(offset)], dtype=torch.int64, device="cuda")


def check_dropout(x, p, seed, offset, res=None, first=0, sample=None):
    rng = rng_of(seed, offset)
    out = B.moe_dropout_fwd(x, p, rng, residual=res)
    dx = B.moe_dropout_bwd(x, p, rng)
    flat, rf = x.reshape(-1), None if res is None else res.reshape(-1)
    for lo, hi in sample or [(0, x.numel())]:
        keep = O.dropout_keep(seed, offset, lo, hi - lo, p)
        X = f64(flat[lo:hi])
        R = None if rf is None else f64(rf[lo:hi])
        fin = np.where(keep & np.isfinite(X), X, 0.0)
        scaled = O.dropout(fin, keep, p)
        mag = np.abs(scaled) + (0 if R is None else np.abs(R))
        ref = scaled if R is None else scaled + R
        h = half_step(x.dtype)
        live = np.isfinite(X) | ~keep          # dropped infinities and NaN count as zero
        got = f64(out.reshape(-1)[lo:hi])
        assert (np.abs(got - ref)[live] <= (4 * U * mag + h * np.abs(ref))[live]).all()
        gdx = f64(dx.reshape(-1)[lo:hi])
        assert (np.abs(gdx - scaled)[live] <= ((4 * U + h) * np.abs(scaled))[live]).all()
        assert (gdx[~keep] == 0).all()
    return out, dx


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 4096, 10007, 20000])
@pytest.mark.parametrize("residual", [True, False])
def test_dropout(dtype, n, residual):
    gen = torch.Generator().manual_seed(n)
    res = draw(gen, n, dtype=dtype) if residual else None
    check_dropout(draw(gen, n, dtype=dtype), 0.1, 1234567890123, 42, res)


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.25, 0.5, 0.999995, 1.0])
def test_dropout_rates(p):
    gen = torch.Generator().manual_seed(1)
    x, res = draw(gen, 3000), draw(gen, 3000)
    out, dx = check_dropout(x, p, (1 << 64) - 5, (1 << 63) + 3, res)
    if p == 0.0:
        assert torch.equal(dx, x) and torch.equal(out, x + res)
    if p == 1.0:
        assert torch.equal(out, res) and not dx.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sx,sr,so", [(1, 0, 0), (0, 1, 0), (3, 3, 3), (0, 0, 5)])
def test_dropout_unaligned(dtype, sx, sr, so):
    gen = torch.Generator().manual_seed(2)
    n = 3001
    x, res = draw(gen, n + 8, dtype=dtype)[sx:sx + n], draw(gen, n + 8, dtype=dtype)[sr:sr + n]
    want, _ = check_dropout(x, 0.3, 5, 6, res)
    buf = torch.full((n + 16,), 9.0, device="cuda", dtype=dtype)
    rng = rng_of(5, 6)
    got = B.moe_dropout_fwd(x, 0.3, rng, residual=res, out=buf[so:so + n])
    assert torch.equal(got, want) and (buf[:so] == 9).all() and (buf[so + n:] == 9).all()


def test_dropout_drops_infinities_and_keeps_shapes():
    gen = torch.Generator().manual_seed(3)
    x = draw(gen, 40, 50)
    x.view(-1)[::3] = float("nan")
    x.view(-1)[1::3] = float("inf")
    out, dx = check_dropout(x, 0.5, 77, 0)
    keep = torch.from_numpy(O.dropout_keep(77, 0, 0, 2000, 0.5)).cuda().view(40, 50)
    assert (out[~keep] == 0).all() and (torch.isnan(out) == (torch.isnan(x) & keep)).all()


def test_dropout_in_place_and_empty():
    gen = torch.Generator().manual_seed(4)
    x, res = draw(gen, 5000, dtype=BF16), draw(gen, 5000, dtype=BF16)
    rng = rng_of(1, 2)
    want = B.moe_dropout_fwd(x, 0.2, rng, residual=res)
    a, b = x.clone(), res.clone()
    assert torch.equal(B.moe_dropout_fwd(a, 0.2, rng, residual=res, out=a), want)
    assert torch.equal(B.moe_dropout_fwd(x, 0.2, rng, residual=b, out=b), want)
    assert B.moe_dropout_fwd(x[:0], 0.2, rng).shape == (0,)


def test_dropout_offsets_past_32_bits():
    """More than 2^32 elements: block numbers and addresses of 64 bits."""
    n = (1 << 32) + 4099
    if torch.cuda.mem_get_info()[0] < 5 * n:
        pytest.skip("needs 20 GB")
    x = torch.ones(n, device="cuda", dtype=BF16)
    rng = rng_of(9, 1)
    B.moe_dropout_bwd(x, 0.5, rng, dx=x)
    for lo, hi in ((0, 2000), ((1 << 31) - 1000, (1 << 31) + 1000), ((1 << 32) - 1000, (1 << 32) + 1000), (n - 2000, n)):
        keep = O.dropout_keep(9, 1, lo, hi - lo, 0.5)
        assert (f64(x[lo:hi]) == keep * 2.0).all()


def test_dropout_replayed_graph_draws_what_the_offset_says():
    gen = torch.Generator().manual_seed(5)
    x, res = draw(gen, 100, 333, dtype=BF16), draw(gen, 100, 333, dtype=BF16)
    rng, out = rng_of(3, 0), torch.empty(100, 333, device="cuda", dtype=BF16)
    B.moe_dropout_fwd(x, 0.4, rng, residual=res, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        B.moe_dropout_fwd(x, 0.4, rng, residual=res, out=out)
    for step in (1, 2, 1 << 40):
        rng[1] = step
        graph.replay()
        assert torch.equal(out, B.moe_dropout_fwd(x, 0.4, rng_of(3, step), residual=res))


def test_calls_on_another_stream():
    gen = torch.Generator().manual_seed(6)
    x, w, dy = draw(gen, 2000, 512, dtype=BF16), draw(gen, 512), draw(gen, 2000, 512, dtype=BF16)
    torch.cuda.synchronize()
    want = B.moe_layernorm_fwd(x, w)
    wb = B.moe_layernorm_bwd(dy, x, w, want[1], want[2])
    wd = B.moe_dropout_fwd(x, 0.1, rng_of(1, 1), residual=dy)
    rng = rng_of(1, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        y, mean, rstd = B.moe_layernorm_fwd(x, w, stream=side)
        g = B.moe_layernorm_bwd(dy, x, w, mean, rstd, stream=side)
        o = B.moe_dropout_fwd(x, 0.1, rng, residual=dy, stream=side)
        # what the current stream allocates meanwhile must not be the side stream's workspace
        junk = [torch.full((1 << 16,), 1.0, device="cuda") for _ in range(8)]
        side.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(o, wd)
        assert all(torch.equal(g[n], wb[n]) for n in g)
        del junk
