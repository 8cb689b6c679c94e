"""GPU tests of the block-scaled operators on matrices of more than 2^31 elements, where an offset
of 32 bits would come back to the start: their first and last rows against 64 bits, with the
checks and tolerances of test_gpu_block.py and test_gpu_saved.py."""
import pytest
import torch

import block_ref as ref
import test_gpu_block as block
from test_gpu_saved import EPS, h, ln_bwd_tolerances, near, near_block

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def rows_of(q, lo, hi):
    return q.__class__(q.codes[lo:hi], q.scales[lo:hi], q.cols, q.fmt, 1)


def pattern(rows, cols, seed=0):
    """Normal values in BF16, a few thousand rows repeated with a sign that changes: cheap to make
    and never the same 2^31 or 2^32 elements later."""
    base = torch.randn(4099, cols, generator=block.gen(seed), device="cuda").to(BF16)
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    for i, lo in enumerate(range(0, rows, 4099)):
        n = min(4099, rows - lo)
        x[lo:lo + n] = base[:n] * (1 + i / 1024)
    return x


def test_quantize_both_ways_and_back():
    f = _lib()
    rows, cols = 66000, 33000
    x = pattern(rows, cols)
    q, qt = f.BlockFp8.empty(rows, cols), f.BlockFp8.empty(cols, rows)
    f.fp8_block_quantize(x, q, qt)
    torch.cuda.synchronize()
    for lo, hi in ((0, 300), (rows // 2, rows // 2 + 300), (rows - 300, rows)):
        block.assert_block(rows_of(q, lo, hi), *ref.quantize(x[lo:hi], 0), ("rows", lo))
    for lo, hi in ((0, 100), (cols // 2, cols // 2 + 100), (cols - 100, cols)):
        block.assert_block(rows_of(qt, lo, hi), *ref.quantize(x[:, lo:hi].t(), 0), ("columns", lo))
    out = torch.empty_like(x)
    f.fp8_block_dequantize(q, out)
    for lo, hi in ((0, 300), (rows - 300, rows)):
        assert torch.equal(out[lo:hi], ref.values(rows_of(q, lo, hi))[0].float().to(BF16))


@pytest.mark.parametrize("kept", [False, True])
def test_layernorm(kept):
    f = _lib()
    rows, cols = 600011, 4001
    x = pattern(rows, cols)
    gamma = 1 + 0.3 * torch.randn(cols, generator=block.gen(1), device="cuda")
    beta = torch.randn(cols, generator=block.gen(2), device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y, x8 = torch.empty_like(x), f.BlockFp8.empty(rows, cols)
    f.fp8_layernorm_fwd(x, gamma, beta, EPS, mean, rstd, y=y, x8=x8)
    for lo, hi in ((0, 200), (rows - 200, rows)):
        want = ref.layernorm(x[lo:hi], gamma, beta, EPS)[0]
        tol = 2.0 ** -18 * (1 + want.abs() + beta.double().abs())
        near(y[lo:hi], want, tol + h(BF16) * (want.abs() + tol), ("y", lo))
        block.assert_block(rows_of(x8, lo, hi), *ref.quantize(x[lo:hi], 0), ("x8", lo))
    dy, dx = y, torch.empty_like(x)
    dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    f.fp8_layernorm_bwd(dy, x8 if kept else x, gamma, mean, rstd, dx, dgamma, dbeta)
    f.fp8_sync_status()
    for lo, hi in ((0, 200), (rows - 200, rows)):
        seen = ref.values(rows_of(x8, lo, hi))[0] if kept else x[lo:hi]
        args = (dy[lo:hi], seen, gamma, mean[lo:hi], rstd[lo:hi])
        want, tol = ref.layernorm_bwd(*args)[0], ln_bwd_tolerances(*args, 0.0)[0]
        near(dx[lo:hi], want, tol + h(BF16) * (want.abs() + tol), ("dx", lo))


def test_layernorm_recompute():
    f = _lib()
    rows, cols = 600011, 4001
    x8, yt = f.BlockFp8.empty(rows, cols), f.BlockFp8.empty(cols, rows)
    f.fp8_block_quantize(pattern(rows, cols), x8)
    gamma = 1 + 0.3 * torch.randn(cols, generator=block.gen(1), device="cuda")
    beta = torch.randn(cols, generator=block.gen(2), device="cuda")
    mean = 0.1 * torch.randn(rows, generator=block.gen(3), device="cuda")
    rstd = 1 + torch.rand(rows, generator=block.gen(4), device="cuda")
    f.fp8_layernorm_recompute(x8, gamma, beta, mean, rstd, yt)
    torch.cuda.synchronize()
    lo = rows - rows % 128 - 256    # the last blocks of all columns
    seen, m, r = ref.values(rows_of(x8, lo, rows))[0], mean[lo:, None].double(), rstd[lo:, None].double()
    want = (seen - m) * r * gamma.double() + beta.double()
    tol = 2.0 ** -22 * ((seen.abs() + m.abs()) * r * gamma.double().abs() + beta.double().abs() + want.abs())
    part = f.BlockFp8(yt.codes[:, lo:], yt.scales[:, lo // 128:], rows - lo)
    near_block(part, want.t(), tol.t(), "yt")


def test_swiglu():
    f = _lib()
    M, F = 100003, 11008
    x = pattern(M, 2 * F)
    a8, h8 = f.BlockFp8.empty(M, F), f.BlockFp8.empty(M, 2 * F)
    f.fp8_swiglu_fwd(x, a8, h8)
    torch.cuda.synchronize()
    for lo, hi in ((0, 200), (M - 200, M)):
        want = ref.swiglu(x[lo:hi])
        tol = want.abs() * (2.0 ** -20 + x[lo:hi, :F].double().abs() * 2.0 ** -22)
        near_block(rows_of(a8, lo, hi), want, tol, ("a8", lo))
        block.assert_block(rows_of(h8, lo, hi), *ref.quantize(x[lo:hi], 0), ("h8", lo))
    da = pattern(M, F, 5)
    dh8, dh8t, a8t = f.BlockFp8.empty(M, 2 * F, 1), f.BlockFp8.empty(2 * F, M, 1), f.BlockFp8.empty(F, M)
    f.fp8_swiglu_bwd(da, h8, dh8, dh8t, a8t)
    torch.cuda.synchronize()
    lo = M - M % 128 - 128
    seen = ref.values(rows_of(h8, lo, M))[0]
    d, (g, u) = da[lo:].double(), seen.chunk(2, 1)
    s, rel = torch.sigmoid(g), 2.0 ** -20 + g.abs() * 2.0 ** -22
    size = d.abs() * u.abs() * s * (1 + g.abs() * (1 - s) + g.abs())
    want, tol = ref.swiglu_bwd(da[lo:], seen), torch.cat([size * rel, d.abs() * (g * s).abs() * rel], 1)
    near_block(rows_of(dh8, lo, M), want, tol, "dh8")
    tail = lambda q: f.BlockFp8(q.codes[:, lo:], q.scales[:, lo // 128:], M - lo, q.fmt)
    near_block(tail(dh8t), want.t(), tol.t(), "dh8t")
    want = ref.swiglu(seen)
    near_block(tail(a8t), want.t(), (want.abs() * rel).t(), "a8t")


@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
@pytest.mark.parametrize("M,N,K", [(70001, 33000, 200), (128, 20000, 130000)])
def test_gemm(M, N, K, sd):
    """A D of more than 2^31 elements, and a B of more than 2^31 codes."""
    f = _lib()
    A, B = block.operand(M, K, 0, 1, sd, 1), block.operand(N, K, 0, 1, sd, 2)
    D = torch.empty(M, N, dtype=BF16, device="cuda")
    f.fp8_block_gemm_tn(A, B, D)
    f.fp8_sync_status()
    for lo in (0, M - 100):
        for c in (0, N - 100):
            block.check_gemm(rows_of(A, lo, lo + 100), rows_of(B, c, c + 100), D[lo:lo + 100, c:c + 100], (lo, c))
