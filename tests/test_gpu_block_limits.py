"""GPU tests of the block-scaled operators at the ends of their ranges."""
import pytest
import torch

import block_ref as ref
from test_gpu_saved import EPS, near

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
