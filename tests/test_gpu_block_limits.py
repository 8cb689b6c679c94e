"""GPU tests of the block-scaled operators at the ends of their ranges."""
import pytest
import torch

import block_ref as ref
from test_gpu_block import check_gemm, operand
from test_gpu_saved import EPS, near, near_block

pytestmark = pytest.mark.gpu


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


# one width for each form of the forward: a warp per row, a CTA per row with one and with
# two groups of columns per thread, rows read again for each use; aligned and not
LN_WIDTHS = [64, 301, 528, 1001, 4096, 8200, 12288, 16384, 16385, 20000]


@pytest.mark.parametrize("cols", LN_WIDTHS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layernorm_statistics_beyond_fp32(cols, dtype):
    """The formula in fp32 where its sums are infinite.  Row 1: finite values whose squared
    deviations overflow: the variance is inf, rstd 0 and y = beta exactly.  Rows 2 and 3: an
    infinity: the mean is that infinity, rstd and y are NaN (inf - inf).  Row 4: a NaN.  Rows 0
    and 5 are ordinary and are not touched by their neighbours."""
    f = _lib()
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    x = torch.randn(6, cols, generator=g, device="cuda").to(dtype)
    x[1] = 1e30
    x[1, 1::2] *= -1
    x[2, cols // 2] = float("inf")
    x[3, cols - 1] = float("-inf")
    x[4, 0] = float("nan")
    gamma = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    beta = torch.randn(cols, generator=g, device="cuda").to(dtype).float()
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    y, y8 = torch.empty_like(x), f.BlockFp8.empty(6, cols)
    f.fp8_layernorm_fwd(x, gamma, beta, EPS, mean, rstd, y=y, y8=y8)
    torch.cuda.synchronize()
    assert abs(mean[1].double() - x[1].double().mean()) <= 2.0 ** -20 * x[1].double().abs().mean()
    assert rstd[1] == 0
    assert torch.equal(y[1].float(), beta)
    want, _ = ref.quantize(beta[None], y8.fmt)
    assert torch.equal(y8.codes[1, :cols], want[0])
    assert mean[2] == float("inf") and mean[3] == float("-inf")
    assert rstd[2:5].isnan().all() and mean[4].isnan()
    assert y[2:5].isnan().all() and y8.dequantize()[2:5].isnan().all()
    y0, mean0, rstd0 = ref.layernorm(x, gamma, beta, EPS)
    tol = 2.0 ** -18 * (gamma.double().abs() * (1 + (x.double() - mean0[:, None]).abs() * rstd0[:, None]) +
                        beta.double().abs())
    for r in (0, 5):
        near(y[r], y0[r], tol[r] + torch.finfo(dtype).eps / 2 * (y0[r].abs() + tol[r]), ("y", r))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low,high", [(-88.5, -87.5), (-88.5, -80.0), (-20.0, 3.0)])
def test_swiglu_of_gates_that_leave_next_to_nothing(dtype, low, high):
    """Gates down to where exp(-gate) is the largest fp32 number: sigmoid is a subnormal number
    there, its products with the gate and the value are not, and a block's scale reaches down to
    them.  Tolerance: |gate| 2^-22 for the rounding of the X sigmoid's own rounding is 2^-22; no absolute part."""
    f = _lib()
    M, F = 40, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda r, c: torch.rand(r, c, generator=g, device="cuda")
    gate = low + (high - low) * rnd(M, F)
    value = (1 + rnd(M, F)) * torch.where(rnd(M, F) < 0.5, -1000.0, 1000.0)
    h = torch.cat([gate, value], 1).to(dtype)
    a8 = f.BlockFp8.empty(M, F)
    f.fp8_swiglu_fwd(h, a8)
    torch.cuda.synchronize()
    want = ref.swiglu(h)
    rel = 2.0 ** -19 + h[:, :F].double().abs() * 2.0 ** -22
    near_block(a8, want, want.abs() * rel, "a8")
    h8 = f.BlockFp8.empty(M, 2 * F)
    f.fp8_block_quantize(torch.cat([gate, value], 1), h8)
    seen = ref.values(h8)[0]
    assert seen[:, :F].min() > -88.7    # in 8 bits too
    da = ((1 + rnd(M, F)) * 1000).to(dtype)
    dh, a = ref.swiglu_bwd(da, seen), ref.swiglu(seen)
    gs, u = seen.chunk(2, 1)
    s = torch.sigmoid(gs)
    rel = 2.0 ** -19 + gs.abs() * 2.0 ** -22
    size = da.double().abs() * u.abs() * s * (1 + 2 * gs.abs())
    tol = torch.cat([size * rel, da.double().abs() * (gs * s).abs() * rel], 1)
    dh8, dh8t, a8t = f.BlockFp8.empty(M, 2 * F, 1), f.BlockFp8.empty(2 * F, M, 1), f.BlockFp8.empty(F, M)
    f.fp8_swiglu_bwd(da, h8, dh8, dh8t, a8t)
    torch.cuda.synchronize()
    near_block(dh8, dh, tol, "dh8")
    near_block(dh8t, dh.t(), tol.t(), "dh8t")
    near_block(a8t, a.t(), (a.abs() * rel).t(), "a8t")


@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
@pytest.mark.parametrize("M,bb", [(1, 1), (17, 128)])
def test_gemm_of_few_rows_with_more_tiles_than_a_grid_dimension(M, bb, sd):
    """65,537 tiles of 128 rows of B: more than the second and third grid dimensions count."""
    f = _lib()
    edge, K = 65535 * 128, 16
    N = edge + 128 + 5
    A, B = operand(M, K, 0, 1, sd, 1), operand(N, K, 0, bb, sd, 2)
    D = torch.full((M, N + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    f.fp8_block_gemm_tn(A, B, D[:, :N])
    f.fp8_sync_status()
    assert not D[:, :N].isnan().any() and D[:, N:].isnan().all()
    for lo, hi in ((0, 1000), (edge - 256, edge), (edge, N)):
        part = f.BlockFp8(B.codes[lo:hi], B.scales[lo // bb:-(-hi // bb)], K, 0, bb)
        check_gemm(A, part, D[:, lo:hi], (M, lo, sd))


@pytest.mark.parametrize("saved", [False, True])
def test_layernorm_bwd_with_more_slabs_than_a_grid_dimension(saved):
    """65,537 slabs of 4096 columns: more than the second and third grid dimensions count.
    One row with mean 0 and rstd 1, gamma 1 and few nonzero gradients, so that its sums are exact:
    xhat = x, s1 = sum dy, s2 = sum dy x; dgamma = dy x and dbeta = dy without rounding."""
    f = _lib()
    cols = 65536 * 4096 + 24
    x = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    at = torch.tensor([0, 4095, 4096, 32768 * 4096 - 1, 32768 * 4096, 32769 * 4096 + 7, 65535 * 4096 - 1,
                       65535 * 4096, 65536 * 4096 + 3, cols - 1], device="cuda")
    dy[0, at] = torch.tensor([1, 2, -3, 4, 5, -6, 7, 8, -16, 12], device="cuda").bfloat16()
    x[0, at] = torch.tensor([2, -1, 4, 1, 8, -2, 1, 4, 2, -8], device="cuda").bfloat16()
    x[0, 100:200] = 3
    src = x
    if saved:
        src = f.BlockFp8.empty(1, cols)
        f.fp8_block_quantize(x, src)
    one = torch.ones(1, device="cuda")
    gamma = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    dx = torch.full_like(x, float("nan"))
    dgamma, dbeta = torch.full((2, cols), float("nan"), device="cuda")
    f.fp8_layernorm_bwd(dy, src, gamma, 0 * one, one, dx, dgamma, dbeta)
    f.fp8_sync_status()
    assert torch.equal(dbeta, dy[0].float())
    assert torch.equal(dgamma, dy[0].float() * x[0].float())
    xd, dyd = x[0].float(), dy[0].float()
    s1, s2 = float(dyd.double().sum()), float((dyd * xd).double().sum())
    want = dyd - s1 / cols - xd * (s2 / cols)
    # one rounding to BF16 and fp32 ones of each of the terms
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -22 * (dyd.abs() + abs(s1) / cols + xd.abs() * abs(s2) / cols)
    assert ((dx[0].float() - want).abs() <= tol).all()
