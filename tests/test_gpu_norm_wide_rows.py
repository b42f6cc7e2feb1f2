"""Layer norm of rows far wider than a block's registers: widths up to the
largest that the calls accept, against sums in 64 bits."""
import ctypes

import pytest
import torch

from mixture_experts_layer_59_b200 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
STEP = 1 << 27          # columns compared at a time


@pytest.fixture(autouse=True)
def give_memory_back():
    """The large buffers of a test are not kept from those after it."""
    yield
    torch.cuda.empty_cache()


def need(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


@pytest.mark.parametrize("d", [(1 << 31) - 1, (1 << 31) - 1023, (1 << 31) - 1025, (1 << 30) + 1])
def test_widest_rows_by_single_elements(d):
    """Ones of both signs in turn, the last column zero: every sum is a whole
    number below 2^24 in each thread, so the mean is exactly 0 and the sum of
    squares exactly d - 1.  rstd then errs by the rounding of 1 / d, of the
    product and by the root's 2 ulp, fewer than 8 steps of 2^-24; y = +-rstd
    rounds once more, to bf16, which rstd's error may carry over to the next
    value where it lies that near the middle."""
    need(20)
    x = torch.ones(1, d, device="cuda", dtype=BF16)
    x[0, 1::2] = -1
    x[0, -1] = 0
    y = torch.full((1, d), 7.0, device="cuda", dtype=BF16)
    _, mean, rstd = B.moe_layernorm_fwd(x, y=y, mean=torch.full((1,), 7.0, device="cuda"),
                                        rstd=torch.full((1,), 7.0, device="cuda"))
    want = ((d - 1) / d + 1e-5) ** -0.5
    assert float(mean) == 0.0 and abs(float(rstd) - want) <= 8 * 2.0 ** -24
    r = rstd.to(BF16)[0]
    assert abs(float(r) - want) <= 2.0 ** -8
    for i in range(0, d, STEP):
        assert torch.equal(y[0, i:i + STEP], x[0, i:i + STEP] * r), i


def test_widest_row_backward():
    """dx of the widest row (without the column sums, whose workspace would be
    64 partial rows): x and dy alternate in step, so with rstd = 1 the row sums are
    whole numbers: mean(g) = 0, mean(g xh) = (d - 1) / d, 1 in fp32 (its error,
    2^-31, is below half a step), and dx = dy - xh = 0 exactly where x = dy."""
    d = (1 << 31) - 1
    need(20)
    x = torch.ones(1, d, device="cuda", dtype=BF16)
    x[0, 1::2] = -1
    x[0, -1] = 0
    dx = torch.full((1, d), 7.0, device="cuda", dtype=BF16)
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = B.lib().moe_layernorm_bwd(p(x), d, p(x), d, None, p(mean), p(rstd), None, 0, 1, d, B.MOE_BF16, B.MOE_F32,
                                   p(dx), None, None, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    for i in range(0, d, STEP):
        assert not dx[0, i:i + STEP].any(), i


@pytest.mark.parametrize("dtype,d", [(F32, 1 << 28), (F32, (1 << 26) + 1), (BF16, (1 << 28) + 8), (F32, 70000)])
def test_sums_of_very_wide_rows(dtype, d):
    """A constant row: every addition of a long sum rounds the same way.  A
    thread's 64 additions in fp32, the fp64 sums, their rounding, 5 shuffles
    and 32 warps, the division's reciprocal and product are fewer than 128
    roundings: mean and the backward pass's sums are within 128 x 2^-24 of the
    sum of their terms' magnitudes, here all of one sign.  y = (x - mean) rstd
    is then at most |mean's error| / sqrt(eps), and dx likewise."""
    need(8)
    u = 2.0 ** -24
    x = torch.full((1, d), 0.1, device="cuda", dtype=dtype)
    v = float(x[0, 0])
    y, mean, rstd = B.moe_layernorm_fwd(x)
    tol = 128 * u * v
    assert abs(float(mean) - v) <= tol
    assert float(y.abs().max()) <= tol / 1e-5 ** 0.5 * (1 + 2.0 ** -7)
    # g = dy = x, xh = (x - 0) 1: mean(g) = v, mean(g xh) = v^2, dx = v - v - v v^2
    dx = torch.empty_like(x)
    m0, r1 = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = B.lib().moe_layernorm_bwd(p(x), d, p(x), d, None, p(m0), p(r1), None, 0, 1, d,
                                   B.MOE_BF16 if dtype == BF16 else B.MOE_F32, B.MOE_F32, p(dx), None, None, None, 0,
                                   ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    half = torch.finfo(dtype).eps / 2
    err = (dx.double() + v ** 3).abs().max()
    assert float(err) <= tol + 128 * u * v ** 3 + 4 * u * v + 2 * half * v ** 3


def test_column_sums_over_many_wide_rows():
    """dbias and dweight of a constant dy over 400000 rows of 8193 columns: a
    thread's 64 additions, the fp64 sums, their rounding and the partial rows'
    sums (2 in a thread, 32 joined) are fewer than 128 roundings."""
    T, d, u = 400000, 8193, 2.0 ** -24
    need(30)
    dy = torch.full((T, d), 0.1, device="cuda", dtype=F32)
    v = float(dy[0, 0])
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    g = B.moe_layernorm_bwd(dy, dy, None, mean, rstd)
    assert float((g["dbias"].double() - T * v).abs().max()) <= 128 * u * T * v
    assert float((g["dweight"].double() - T * v * v).abs().max()) <= 128 * u * T * v * v
