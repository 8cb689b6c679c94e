"""GPU tests of LayerNorm forward and backward and of SwiGLU, and of both with their
inputs kept in 8 bits, against plain implementations in 64 bits (block_ref.py).

Tolerances, with h(t) = eps(t) / 2 the half step of a type: an output of type t
may be off by h(t) of its value for its last rounding, and by the fp32
roundings before it: 2^-24 of each intermediate value for each operation; the
sums over a row or down the rows have a bound of 2^-20 of the sum of their
terms' magnitudes (a thread adds at most 64 terms in a row, then a tree).
Values quantized to 8 bits may also sit on the other side of a tie: they are
compared with the unrounded ones, to half a step of the format at that size
under the block's scale, and the scale itself to what the definition gives
for the block's maximum, 2^-16 up or down."""
import pytest
import torch

import block_ref as ref
from test_gpu_block import assert_block, assert_marks, gen, marked

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
EPS = 1e-5


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def h(dtype):
    return torch.finfo(dtype).eps / 2


def near(got, want, tol, what):
    """got is want to tol, or the infinity that want rounds to in got's type."""
    over = want.abs() - tol > torch.finfo(got.dtype).max * (1 + h(got.dtype))
    assert torch.equal(got[over].double(), want[over].sign() * float("inf")), what
    got, want, tol = got[~over], want[~over], tol[~over]
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (what, float((off - tol).max()), torch.nonzero(~(off <= tol))[:4].tolist())


def near_block(q, want, tol, what):
    """q holds want (double, known to tol) quantized with blocks along its columns."""
    got, s = ref.values(q)
    least, bits = (-6, 4) if q.fmt == 0 else (-14, 3)
    half = torch.maximum(want.abs() * 2.0 ** -bits, s * 2.0 ** (least - bits))
    near(got, want, half + 2 * tol, what)
    rows, cols = q.shape
    nb = -(-cols // 128)
    w = torch.zeros(rows, nb * 128, dtype=torch.float64, device=want.device)
    w[:, :cols] = want.abs()
    amax = w.view(rows, nb, 128).amax(2)
    e = q.scales[:rows, :nb].to(torch.int64) - 127
    lo = ref.scale_exponent(amax * (1 - 2.0 ** -16), q.fmt)
    hi = ref.scale_exponent(amax * (1 + 2.0 ** -16), q.fmt)
    assert ((lo <= e) & (e <= hi)).all(), what


def ln_inputs(rows, cols, dtype, wtype, seed):
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * 2 + 0.7
    x[:, ::13] *= 6
    if rows > 2:
        x[1] = 3.25      # a constant row: its variance is 0
    gamma = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(wtype)
    beta = (0.2 * torch.randn(cols, generator=g, device="cuda")).to(wtype)
    return x.to(dtype), gamma, beta


def padded(t, left, right):
    """The same values as a view into a wider matrix."""
    w = torch.full((t.shape[0], t.shape[1] + left + right), 9.0, dtype=t.dtype, device="cuda")
    w[:, left:left + t.shape[1]] = t
    return w[:, left:left + t.shape[1]]


LN_SHAPES = [(1, 1), (1, 8), (2, 3), (5, 127), (3, 128), (4, 1000), (2, 1024), (7, 1025), (300, 264),
             (700, 80), (3, 4096), (5, 4103), (2, 8192), (3, 8200), (2, 16384), (3, 16392),
             (2, 40003)]


@pytest.mark.parametrize("rows,cols", LN_SHAPES)
@pytest.mark.parametrize("dtype,wtype", [(torch.float32, torch.float32),
                                         (torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float32),
                                         (torch.float16, torch.float16)])
def test_layernorm_fwd(rows, cols, dtype, wtype):
    f = _lib()
    x, gamma, beta = ln_inputs(rows, cols, dtype, wtype, rows + cols)
    y0, mean0, rstd0 = ref.layernorm(x, gamma, beta, EPS)
    amean = x.double().abs().mean(1)
    tol_mean = 2.0 ** -20 * amean
    # the mean's error moves every deviation; relative to the row's spread
    spread = (tol_mean + 2.0 ** -23 * x.double().abs().amax(1)) * rstd0
    tol_rstd = rstd0 * (2.0 ** -20 + spread ** 2)
    z = (x.double() - mean0[:, None]).abs() * rstd0[:, None]
    tol_y = (gamma.double().abs() * (spread[:, None] + z * (2.0 ** -19 + spread[:, None] ** 2)) +
             2.0 ** -23 * (beta.double().abs() + y0.abs()))
    for src, out in [(x, torch.empty_like(x)), (padded(x, 8, 8), padded(x, 0, 8)),
                     (padded(x, 1, 2), padded(x, 3, 0))]:
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        f.fp8_layernorm_fwd(src, gamma, beta, EPS, mean, rstd, y=out)
        near(mean, mean0, tol_mean + 2.0 ** -24 * mean0.abs(), "mean")
        near(rstd, rstd0, tol_rstd, "rstd")
        near(out, y0, tol_y + h(dtype) * (y0.abs() + tol_y), ("y", rows, cols))
    for fy, fx, sd in [(0, 0, torch.uint8), (1, 0, torch.float32)]:
        y8, yb = marked(rows, cols, fy, 1, torch.uint8)
        x8, xb = marked(rows, cols, fx, 1, sd)
        f.fp8_layernorm_fwd(padded(x, 1, 2), gamma, beta, EPS, mean, rstd, y8=y8, x8=x8)
        torch.cuda.synchronize()
        near_block(y8, y0, tol_y, ("y8", rows, cols))
        assert_block(x8, *ref.quantize(x, fx), ("x8", rows, cols))
        assert_marks(y8, yb, "y8")
        assert_marks(x8, xb, "x8")


def test_layernorm_special_rows():
    """A NaN or an infinity spoils its own row, and only that one."""
    f = _lib()
    x, gamma, beta = ln_inputs(6, 300, torch.bfloat16, torch.float32, 3)
    x[2, 5] = float("nan")
    x[4, 299] = float("inf")
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    y, y8 = torch.empty_like(x), f.BlockFp8.empty(6, 300)
    f.fp8_layernorm_fwd(x, gamma, beta, EPS, mean, rstd, y=y, y8=y8)
    bad = torch.tensor([0, 0, 1, 0, 1, 0], dtype=torch.bool, device="cuda")
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(y.isnan().any(1), bad)
    assert torch.equal(y8.dequantize().isnan().all(1), bad)


def ln_bwd_tolerances(dy, x, gamma, mean, rstd, err_x):
    """Bounds of the fp32 errors of dx, dgamma and dbeta."""
    dy, x, gamma = dy.double(), x.double(), gamma.double()
    r = rstd.double()[:, None]
    z = (x - mean.double()[:, None]) * r
    ez = 2.0 ** -22 * (x.abs() + mean.double()[:, None].abs()) * r + err_x
    u = (dy * gamma).abs()
    n = x.shape[1]
    e1 = 2.0 ** -20 * u.sum(1, keepdim=True) / n
    e2 = (2.0 ** -20 * (u * z.abs()).sum(1, keepdim=True) + (u * ez).sum(1, keepdim=True)) / n
    m2 = ((dy * gamma) * z).mean(1, keepdim=True).abs()
    m1 = (dy * gamma).mean(1, keepdim=True).abs()
    dx = r * (2.0 ** -22 * (u + m1 + z.abs() * m2) + e1 + z.abs() * e2 + ez * m2)
    return (dx, 2.0 ** -20 * (dy * z).abs().sum(0) + (dy.abs() * ez).sum(0),
            2.0 ** -20 * dy.abs().sum(0))


@pytest.mark.parametrize("rows,cols", LN_SHAPES + [(1001, 72), (2500, 136)])
@pytest.mark.parametrize("dtype,wtype,saved", [(torch.float32, torch.float32, False),
                                               (torch.bfloat16, torch.bfloat16, False),
                                               (torch.float16, torch.float32, False),
                                               (torch.float32, torch.bfloat16, True),
                                               (torch.bfloat16, torch.float32, True),
                                               (torch.float16, torch.float16, True)])
def test_layernorm_bwd(rows, cols, dtype, wtype, saved):
    f = _lib()
    x, gamma, beta = ln_inputs(rows, cols, dtype, wtype, rows + cols)
    _, mean, rstd = ref.layernorm(x, gamma, beta, EPS)
    mean, rstd = mean.float(), rstd.float()
    dy = (torch.randn(rows, cols, generator=gen(rows), device="cuda") * 0.1).to(dtype)
    seen = x
    if saved:
        x8 = f.BlockFp8.empty(rows, cols, rows % 2, 1, torch.float32 if cols % 2 else torch.uint8)
        f.fp8_block_quantize(x, x8)
        seen = ref.values(x8)[0]
    want = ref.layernorm_bwd(dy, seen, gamma, mean, rstd)
    tols = ln_bwd_tolerances(dy, seen, gamma, mean, rstd, 0.0)
    for d, s, out in [(dy, x, torch.empty_like(dy)), (padded(dy, 8, 0), padded(x, 8, 8), padded(dy, 0, 8)),
                      (padded(dy, 1, 0), padded(x, 0, 1), padded(dy, 3, 1))]:
        dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        f.fp8_layernorm_bwd(d, x8 if saved else s, gamma, mean, rstd, out, dgamma, dbeta)
        near(out, want[0], tols[0] + h(dtype) * (want[0].abs() + tols[0]) +
             (2.0 ** -25 if dtype == torch.float16 else 0), ("dx", rows, cols))
        near(dgamma, want[1], tols[1], "dgamma")
        near(dbeta, want[2], tols[2], "dbeta")
    again, dg2, db2 = dy.clone(), torch.empty_like(dgamma), torch.empty_like(dbeta)
    ws = torch.empty(f.fp8_layernorm_bwd_workspace(rows, cols) + 4, dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    f.fp8_layernorm_bwd(again, x8 if saved else x, gamma, mean, rstd, again, dg2, db2,
                        workspace=ws[:-4])     # in place, with a workspace of one's own
    assert (ws[-4:] == 0xFF).all()
    assert torch.equal(again, out) and torch.equal(dg2, dgamma) and torch.equal(db2, dbeta)


def test_layernorm_gradients_against_differences():
    """The kernel's gradients against central differences of the forward in 64 bits.  With
    step t along a direction the difference quotient is off by O(t^2), here 1e-8 relative."""
    f = _lib()
    rows, cols = 9, 200
    x, gamma, beta = ln_inputs(rows, cols, torch.float32, torch.float32, 11)
    x[1] += torch.randn(cols, generator=gen(1), device="cuda")
    dy = torch.randn(rows, cols, generator=gen(2), device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    f.fp8_layernorm_fwd(x, gamma, beta, EPS, mean, rstd)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    f.fp8_layernorm_bwd(dy, x, gamma, mean, rstd, dx, dg, db)
    loss = lambda x, g, b: (dy.double() * ref.layernorm(x, g, b, EPS)[0]).sum().item()
    args = [x.double(), gamma.double(), beta.double()]
    for i, grad in enumerate((dx, dg, db)):
        v = torch.randn(args[i].shape, generator=gen(20 + i), device="cuda", dtype=torch.float64)
        t = 1e-4
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + t * v, args[i] - t * v
        quotient = (loss(*up) - loss(*down)) / (2 * t)
        exact = (grad.double() * v).sum().item()
        size = (grad.double() * v).abs().sum().item()
        assert abs(quotient - exact) <= 1e-5 * size, (i, quotient, exact)


def test_layernorm_bwd_of_no_rows_gives_zero_weight_gradients():
    f = _lib()
    e = lambda *s: torch.full(s, 3.0, device="cuda")
    dg, db = e(5), e(5)
    f.fp8_layernorm_bwd(e(0, 5), e(0, 5), e(5), e(0), e(0), e(0, 5), dg, db)
    f.fp8_layernorm_fwd(e(0, 5), e(5), e(5), EPS, e(0), e(0), y=e(0, 5))
    assert (dg == 0).all() and (db == 0).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (129, 257), (260, 1000), (16, 4096)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_layernorm_recompute(rows, cols, fmt):
    f = _lib()
    x, gamma, beta = ln_inputs(rows, cols, torch.bfloat16, torch.bfloat16, rows + cols)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    x8 = f.BlockFp8.empty(rows, cols)
    f.fp8_layernorm_fwd(x, gamma, beta, EPS, mean, rstd, x8=x8)
    seen = ref.values(x8)[0]
    z = (seen - mean.double()[:, None]) * rstd.double()[:, None]
    want = z * gamma.double() + beta.double()
    tol = 2.0 ** -22 * ((seen.abs() + mean.double().abs()[:, None]) * rstd.double()[:, None] *
                        gamma.double().abs() + beta.double().abs() + want.abs())
    yt, bufs = marked(cols, rows, fmt)
    f.fp8_layernorm_recompute(x8, gamma, beta, mean, rstd, yt)
    torch.cuda.synchronize()
    near_block(yt, want.t(), tol.t(), (rows, cols))
    assert_marks(yt, bufs, (rows, cols))


def swiglu_input(M, F, dtype, seed):
    x = torch.randn(M, 2 * F, generator=gen(seed), device="cuda") * 2
    x[:, ::17] *= 12       # gates far out on both sides
    if M > 1:
        x[1] = 0
    return x.to(dtype)


@pytest.mark.parametrize("M,F", [(1, 128), (3, 256), (130, 384), (257, 128), (64, 1152)])
@pytest.mark.parametrize("dtype", TYPES)
def test_swiglu_fwd(M, F, dtype):
    f = _lib()
    x = swiglu_input(M, F, dtype, M + F)
    want = ref.swiglu(x)
    # exp(-g) is good to a few units and |g| 2^-23; the rest is four roundings
    tol = want.abs() * (2.0 ** -20 + x[:, :F].double().abs() * 2.0 ** -22) + 1e-37
    for fa, fh, src in [(0, 0, x), (1, 0, padded(x, 1, 2)), (0, 1, padded(x, 8, 8))]:
        a8, ab = marked(M, F, fa)
        h8, hb = marked(M, 2 * F, fh)
        f.fp8_swiglu_fwd(src, a8, h8)
        torch.cuda.synchronize()
        near_block(a8, want, tol, (M, F))
        assert_block(h8, *ref.quantize(x, fh), (M, F))
        assert_marks(a8, ab, "a8")
        assert_marks(h8, hb, "h8")
    only = f.BlockFp8.empty(M, F, 0)
    f.fp8_swiglu_fwd(padded(x, 8, 8), only)
    assert torch.equal(only.codes, a8.codes[:, :only.codes.shape[1]])


def swiglu_bwd_case(M, F, dtype, seed):
    f = _lib()
    x = swiglu_input(M, F, torch.float32, seed)
    h8 = f.BlockFp8.empty(M, 2 * F)
    f.fp8_block_quantize(x, h8)
    seen = ref.values(h8)[0]
    da = (torch.randn(M, F, generator=gen(seed + 1), device="cuda") * 0.01).to(dtype)
    return f, h8, seen, da


@pytest.mark.parametrize("M,F", [(1, 128), (3, 256), (130, 384), (257, 128), (300, 1152)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", [0, 1])
def test_swiglu_bwd(M, F, dtype, fmt):
    f, h8, seen, da = swiglu_bwd_case(M, F, dtype, M + F)
    dh, a = ref.swiglu_bwd(da, seen), ref.swiglu(seen)
    g, u = seen.chunk(2, 1)
    rel = 2.0 ** -20 + g.abs() * 2.0 ** -22
    s = torch.sigmoid(g)
    # 1 + g (1 - s) cancels for negative gates: its terms' size counts
    size = da.double().abs() * u.abs() * s * (1 + g.abs() * (1 - s) + g.abs())
    tol = torch.cat([size * rel, da.double().abs() * (g * s).abs() * rel], 1) + 1e-37
    tol_a = a.abs() * rel + 1e-37
    bufs = [marked(M, 2 * F, fmt), marked(2 * F, M, fmt), marked(F, M, 0)]
    dh8, dh8t, a8t = (b[0] for b in bufs)
    for src in (da, padded(da, 1, 2)):
        f.fp8_swiglu_bwd(src, h8, dh8, dh8t, a8t)
        torch.cuda.synchronize()
        near_block(dh8, dh, tol, "dh8")
        near_block(dh8t, dh.t(), tol.t(), "dh8t")
        near_block(a8t, a.t(), tol_a.t(), "a8t")
        for q, b in bufs:
            assert_marks(q, b, (M, F))
    # any of the three alone is the same
    for i in range(3):
        one = [None, None, None]
        q, b = marked(*bufs[i][0].shape, bufs[i][0].fmt)
        one[i] = q
        f.fp8_swiglu_bwd(da, h8, *one)
        torch.cuda.synchronize()
        rows, cols = q.shape
        assert torch.equal(q.codes, bufs[i][0].codes) and torch.equal(q.scales, bufs[i][0].scales)


def test_swiglu_gradient_against_differences():
    """The kernel's dh (in 8 bits, half a step) against central differences of the formula."""
    f, h8, seen, da = swiglu_bwd_case(40, 128, torch.float32, 9)
    dh8 = f.BlockFp8.empty(40, 256)
    f.fp8_swiglu_bwd(da, h8, dh8)
    got, s = ref.values(dh8)
    t = 1e-5
    g, u = seen.chunk(2, 1)
    up = lambda dg, du: (g + dg) * torch.sigmoid(g + dg) * (u + du)
    num = torch.cat([da.double() * (up(t, 0) - up(-t, 0)) / (2 * t),
                     da.double() * (up(0, t) - up(0, -t)) / (2 * t)], 1)
    assert ((got - num).abs() <= num.abs() * 2.0 ** -4 + s * 2.0 ** -10 + 1e-8).all()


def test_backward_in_a_graph_and_on_a_stream():
    f = _lib()
    rows, cols = 300, 520
    x, gamma, beta = ln_inputs(rows, cols, torch.bfloat16, torch.float32, 5)
    dy = torch.randn(rows, cols, device="cuda").to(torch.bfloat16)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    x8 = f.BlockFp8.empty(rows, cols)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)

    def both(stream=None):
        f.fp8_layernorm_fwd(x, gamma, beta, EPS, mean, rstd, x8=x8, stream=stream)
        f.fp8_layernorm_bwd(dy, x8, gamma, mean, rstd, dx, dg, db, stream=stream)

    both()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dx, dg, db)]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for t in (dx, dg, db):
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        both(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (dx, dg, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in (dx, dg, db, mean, rstd):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (dx, dg, db)))
