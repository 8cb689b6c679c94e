"""GPU tests of calls whose arguments lie between each other's rows in one buffer, or take an
input's very place: they share nothing, or what they may, and give the same bits as in
buffers of their own."""
import pytest
import torch

from test_gpu_gated import held as filled
from test_gpu_rmsnorm import EPS, _lib, inputs

pytestmark = pytest.mark.gpu


def interleaved(rows, *cols, dtype=torch.bfloat16, gap=0):
    """Matrices side by side in the rows of one buffer."""
    wide = torch.full((rows, sum(cols) + gap * len(cols)), 9, dtype=dtype, device="cuda")
    out, at = [], 0
    for c in cols:
        out.append(wide[:, at:at + c])
        at += c + gap
    return out


def held(rows, cols):
    """An 8-bit matrix whose codes and scales share the rows of one buffer."""
    pitch, words = -(-cols // 16) * 16, -(-cols // 512) * 4
    wide = torch.zeros(rows, -(-(pitch + words) // 16) * 16, dtype=torch.uint8, device="cuda")
    return _lib().BlockFp8(wide[:, :pitch], wide[:, pitch:pitch + words], cols)


def same(p, q):
    nb = -(-p.cols // 128)
    assert torch.equal(p.codes[:, :p.cols], q.codes[:, :q.cols]) and torch.equal(p.scales[:, :nb], q.scales[:, :nb])


@pytest.mark.parametrize("rows,cols", [(1, 64), (37, 301), (300, 4096), (200, 8200), (50, 16400)])
@pytest.mark.parametrize("gap", [0, 3])
def test_rmsnorm_between_each_others_rows(rows, cols, gap):
    f = _lib()
    x0, r0, gamma = inputs(rows, cols, torch.bfloat16, torch.float32, cols)
    x, r, total, y, dsum, dx = interleaved(rows, *[cols] * 6, gap=gap)
    x.copy_(x0), r.copy_(r0), dsum.copy_(r0)
    small = torch.empty(rows + cols + 8, device="cuda")
    rstd, dgamma = small[:rows], small[rows:rows + cols]
    y8, x8 = held(rows, cols), held(rows, cols)
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=r, sum=total, y=y, y8=y8, x8=x8)
    f.fp8_rmsnorm_bwd(y, total, gamma, rstd, dx, dgamma, dsum=dsum)
    yt = f.BlockFp8.empty(cols, rows)
    f.fp8_rmsnorm_recompute(x8, gamma, rstd, yt)
    # each in a buffer of its own, in the same place within it, so that sums have the same order
    places = [interleaved(rows, *[cols] * 6, gap=gap)[k] for k in range(6)]
    x2, r2, total2, y2, dsum2, dx2 = places
    x2.copy_(x0), r2.copy_(r0), dsum2.copy_(r0)
    rstd2, dgamma2 = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")
    y82, x82, yt2 = f.BlockFp8.empty(rows, cols), f.BlockFp8.empty(rows, cols), f.BlockFp8.empty(cols, rows)
    f.fp8_rmsnorm_fwd(x2, gamma, EPS, rstd2, residual=r2, sum=total2, y=y2, y8=y82, x8=x82)
    f.fp8_rmsnorm_bwd(y2, total2, gamma, rstd2, dx2, dgamma2, dsum=dsum2)
    f.fp8_rmsnorm_recompute(x82, gamma, rstd2, yt2)
    f.fp8_sync_status()
    for p, q in ((x, x2), (r, r2), (total, total2), (y, y2), (dsum, dsum2), (dx, dx2), (rstd, rstd2), (dgamma, dgamma2)):
        assert torch.equal(p, q)
    same(y8, y82), same(x8, x82), same(yt, yt2)


@pytest.mark.parametrize("rows,cols", [(1, 8), (1300, 512), (700, 301), (900, 4096), (300, 8200), (300, 12288), (200, 16400)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rmsnorm_in_an_inputs_very_place(rows, cols, dtype):
    """sum and y in x's and in the residual's place, dx in x's and in dy's."""
    f = _lib()
    x, r, gamma = inputs(rows, cols, dtype, torch.float32, cols)
    e = torch.empty_like
    rstd, total, y, dx, dg = torch.empty(rows, device="cuda"), e(x), e(x), e(x), torch.empty(cols, device="cuda")
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=r, sum=total, y=y)
    f.fp8_rmsnorm_bwd(y, total, gamma, rstd, dx, dg, dsum=r)
    for k in range(2):
        a, b = x.clone(), r.clone()
        f.fp8_rmsnorm_fwd(a, gamma, EPS, rstd, residual=b, sum=(a, b)[k], y=(b, a)[k])
        c, d, s = y.clone(), r.clone(), total.clone()
        out, dg2 = (s, c)[k], torch.empty_like(dg)
        f.fp8_rmsnorm_bwd(c, s, gamma, rstd, out, dg2, dsum=d)
        f.fp8_sync_status()
        assert torch.equal((a, b)[k], total) and torch.equal((b, a)[k], y)
        assert torch.equal(out, dx) and torch.equal(dg2, dg)
    # without a residual, and without the sum being kept
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, y=y)
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=r, y=total)
    for res, want in ((None, y), (r, total)):
        a = x.clone()
        f.fp8_rmsnorm_fwd(a, gamma, EPS, rstd, residual=res, y=a)
        f.fp8_sync_status()
        assert torch.equal(a, want)


def test_calls_that_overlap_are_refused():
    f = _lib()
    rows, cols = 6, 64
    wide = torch.ones(rows, 200, dtype=torch.bfloat16, device="cuda")
    gamma, rstd = torch.ones(cols, device="cuda"), torch.empty(rows, device="cuda")
    x, dg = wide[:, :cols], torch.empty(cols, device="cuda")
    for kw in (dict(residual=wide[:, 100:164], sum=wide[:, 8:72]), dict(y=wide[:, 63:127]), dict(y=wide[:, :cols], residual=x, sum=x)):
        with pytest.raises(f.Fp8Error, match="overlap"):
            f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, **kw)
    q = f.BlockFp8.empty(rows, cols)
    with pytest.raises(f.Fp8Error, match="overlap"):
        f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, y8=q, x8=q)
    with pytest.raises(f.Fp8Error, match="overlap"):
        f.fp8_rmsnorm_bwd(x, x, gamma, rstd, wide[:, 1:65], dg)
    f.fp8_sync_status()
    assert (wide == 1).all()


@pytest.mark.parametrize("M,F,K", [(5, 256, 200), (300, 640, 512), (1100, 1408, 256), (2100, 2688, 300)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_gated_product_between_rows_and_in_place(M, F, K, fmt):
    """Outputs whose codes and scales share a buffer's rows; dh8 in h8's place; an infinite value
    among them, which takes a second pass over its rows."""
    f = _lib()
    A, B, W = filled(M, K, 1.0, 0, 1, 1), filled(2 * F, K, 1.5 * K ** -0.5, 0, 128, 2), filled(F, K, K ** -0.5, 0, 128, 4)
    a8, h8, e = held(M, F), held(M, 2 * F), f.BlockFp8.empty
    f.fp8_block_gemm_swiglu_fwd(A, B, a8, h8)
    a82, h82 = e(M, F), e(M, 2 * F)
    f.fp8_block_gemm_swiglu_fwd(A, B, a82, h82)
    same(a8, a82), same(h8, h82)
    h8.fmt = h82.fmt = fmt   # as E5M2 the same bytes are other values, infinities among them
    if fmt:
        h8.codes[0, 3] = h82.codes[0, 3] = 0x7C
    dh8, dh8t, a8t = e(M, 2 * F, fmt), e(2 * F, M, fmt), e(F, M)
    f.fp8_block_gemm_swiglu_bwd(A, W, h82, dh8, dh8t, a8t)
    dh8t2, a8t2 = held(2 * F, M), held(F, M)
    dh8t2.fmt = fmt
    f.fp8_block_gemm_swiglu_bwd(A, W, h8, f.BlockFp8(h8.codes, h8.scales, 2 * F, fmt), dh8t2, a8t2)
    f.fp8_sync_status()
    same(h8, dh8), same(dh8t2, dh8t), same(a8t2, a8t)


def test_norm_beside_the_gradients_it_is_of():
    """The norm, the gradients and the clipped ones one behind the other in one buffer."""
    f = _lib()
    flat = torch.randn(5000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    grads, norm, outs = [flat[:1000], flat[1000:2000]], flat[2000:2001], [flat[2001:3001], flat[3001:4001]]
    want = flat[:2000].double().norm()
    kept = flat.clone()
    f.fp8_grad_norm(grads, norm)
    f.fp8_grad_clip(grads, norm, 1.0, outs)
    f.fp8_sync_status()
    assert abs(norm.item() - want) <= 2.0 ** -20 * want
    c = torch.ones(1, device="cuda") / norm
    assert torch.equal(flat[2001:4001], kept[:2000] * c)
    assert torch.equal(flat[:2000], kept[:2000]) and torch.equal(flat[4001:], kept[4001:])
    f.fp8_grad_clip(outs, norm, 2.0)
    for bad in ([flat[1990:2010]], [flat[2000:2001]]):
        with pytest.raises(f.Fp8Error, match="norm overlap"):
            f.fp8_grad_clip(bad, norm, 1.0)
    ws = flat.view(torch.uint8)[4096:]
    with pytest.raises(f.Fp8Error, match="workspace overlap"):
        f.fp8_grad_norm(grads, norm, ws)
    f.fp8_sync_status()
