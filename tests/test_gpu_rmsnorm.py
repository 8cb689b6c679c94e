"""GPU tests of the RMS norm with the residual's addition against plain
implementations in 64 bits.

Tolerances, with h(t) = eps(t) / 2 the half step of a type.  The sum s = x +
residual is one addition in fp32 and one rounding: compared bit for bit.  From
the stored s: the sum of squares (positive terms; a thread adds at most 64 in a
row, then a tree) is known to 2^-20, rstd to half of that and its own
roundings, y to 2^-19 of itself (rstd, two products) and h for its type.  The
backward's sums over a row or down the rows are known to 2^-20 of the sum of
their terms' magnitudes, each product and sum on the way to 2^-24.  Values in 8
bits: as near_block says."""
import pytest
import torch

import block_ref as ref
from test_gpu_block import assert_block, assert_marks, gen, marked
from test_gpu_saved import h, near, near_block, padded

pytestmark = pytest.mark.gpu

EPS = 1e-6
# one width for each form: a warp per row, a CTA per row with one and two groups of columns per
# thread, rows read again for each use; aligned and not
SHAPES = [(1, 1), (1, 8), (2, 3), (5, 127), (3, 128), (9, 512), (4, 1000), (2, 1024), (7, 1025),
          (300, 264), (700, 80), (3, 4096), (5, 4103), (1300, 544), (2, 8192), (3, 8200), (2, 16384),
          (3, 16392), (2, 40003)]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.bfloat16, torch.float32), (torch.float16, torch.float16)]


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def inputs(rows, cols, dtype, wtype, seed):
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    r = torch.randn(rows, cols, generator=g, device="cuda") * 2
    r[:, ::13] *= 6
    if rows > 2:
        x[1] = 0
        r[1] = 0     # a padding token: its norm is 0 / sqrt(eps)
    gamma = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(wtype)
    return x.to(dtype), r.to(dtype), gamma


def plain(s, gamma, eps=EPS):
    s, gamma = s.double(), gamma.double()
    rstd = ((s * s).mean(1) + eps) ** -0.5
    return s * rstd[:, None] * gamma, rstd


def tiny(dtype):
    """Half the smallest step, where values may be below the normal ones."""
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wtype", TYPES)
def test_forward(rows, cols, dtype, wtype):
    f = _lib()
    x, r, gamma = inputs(rows, cols, dtype, wtype, rows + cols)
    for res in (r, None):
        s = x if res is None else (x.float() + res.float()).to(dtype)
        y0, rstd0 = plain(s, gamma)
        tol = 2.0 ** -19 * y0.abs()
        views = [(lambda t: t, lambda t: torch.empty_like(t)),
                 (lambda t: padded(t, 8, 8), lambda t: padded(t, 0, 8)),
                 (lambda t: padded(t, 1, 2), lambda t: padded(t, 3, 0))]
        for src, out in views:
            rstd, y = torch.empty(rows, device="cuda"), out(x)
            total = None if res is None else out(x)
            f.fp8_rmsnorm_fwd(src(x), gamma, EPS, rstd, residual=None if res is None else src(res),
                              sum=total, y=y)
            f.fp8_sync_status()
            near(rstd, rstd0, 2.0 ** -20 * rstd0, "rstd")
            near(y, y0, tol + h(dtype) * (y0.abs() + tol) + tiny(dtype), ("y", rows, cols))
            assert total is None or torch.equal(total, s)
        for fy, fx, sd in [(0, 0, torch.uint8), (1, 0, torch.float32)]:
            y8, yb = marked(rows, cols, fy, 1, torch.uint8)
            x8, xb = marked(rows, cols, fx, 1, sd)
            f.fp8_rmsnorm_fwd(padded(x, 1, 2), gamma, EPS, rstd,
                              residual=None if res is None else padded(res, 8, 0), y8=y8, x8=x8)
            torch.cuda.synchronize()
            near(rstd, rstd0, 2.0 ** -20 * rstd0, "rstd")
            near_block(y8, y0, tol, ("y8", rows, cols))
            assert_block(x8, *ref.quantize(s, fx), ("x8", rows, cols))
            assert_marks(y8, yb, "y8")
            assert_marks(x8, xb, "x8")


@pytest.mark.parametrize("cols", [64, 301, 1001, 4096, 8200, 16384, 16385, 40003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("left", [0, 3, 8])
def test_sum_in_place_of_an_input(cols, dtype, left):
    """sum in x's and in the residual's own memory: the same bits, and nothing beside them."""
    f = _lib()
    rows = 37
    x, r, gamma = inputs(rows, cols, dtype, torch.float32, cols)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    want = torch.empty_like(x)
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=r, sum=want, y=y)
    for which in range(2):
        wide = [torch.full((rows, left + cols + 5), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
        a, b = (w[:, left:left + cols] for w in wide)
        a.copy_(x), b.copy_(r)
        y2, rstd2 = torch.empty_like(x), torch.empty_like(rstd)
        f.fp8_rmsnorm_fwd(a, gamma, EPS, rstd2, residual=b, sum=(a, b)[which], y=y2)
        f.fp8_sync_status()
        assert torch.equal((a, b)[which], want)
        assert torch.equal((b, a)[which], (r, x)[which])
        near(rstd2, plain(want, gamma)[1], 2.0 ** -20 * rstd.double(), "rstd")
        y0 = plain(want, gamma)[0]
        near(y2, y0, (2.0 ** -19 + 2 * h(dtype)) * y0.abs(), "y")
        for w in wide:
            assert (w[:, :left] == 9).all() and (w[:, left + cols:] == 9).all()


@pytest.mark.parametrize("cols", [64, 301, 528, 1001, 4096, 8200, 12288, 16384, 16385, 20000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_beyond_fp32(cols, dtype):
    """Row 1: finite values whose squares overflow: rstd 0 and y 0.  Row 2: an infinity: rstd 0, y
    0 and NaN where it stands.  Row 3: a NaN spoils its row.  Row 4: an infinite sum of finite
    addends.  Rows 0 and 5 are ordinary and are not touched by their neighbours."""
    f = _lib()
    x, r, gamma = inputs(6, cols, dtype, torch.float32, cols)
    r[1], x[1] = 1e30, 1e30
    r[2, cols // 2] = float("inf")
    r[3, 0] = float("nan")
    r[4, cols - 1] = x[4, cols - 1] = torch.finfo(dtype).max
    s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(6, device="cuda")
    y8 = f.BlockFp8.empty(6, cols)
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=r, sum=s, y=y, y8=y8)
    f.fp8_sync_status()
    assert torch.equal(s.isnan(), (x.float() + r.float()).isnan())
    assert rstd[1] == 0 and rstd[2] == 0 and rstd[3].isnan() and rstd[4] == 0
    assert (y[1] == 0).all() and y[3].isnan().all()
    for row, at in ((2, cols // 2), (4, cols - 1)):
        assert s[row, at] == float("inf") and y[row, at].isnan()
        assert int(y[row].isnan().sum()) == 1 and int((y[row] == 0).sum()) == cols - 1
    assert torch.equal(y8.dequantize().isnan(), y.isnan())
    y0, rstd0 = plain(s[[0, 5]], gamma)
    near(rstd[[0, 5]], rstd0, 2.0 ** -20 * rstd0, "rstd")
    near(y[[0, 5]], y0, (2.0 ** -19 + 2 * h(dtype)) * y0.abs(), "y")


def bwd_plain(dy, s, gamma, rstd, dsum):
    dy, s, gamma, r = dy.double(), s.double(), gamma.double(), rstd.double()[:, None]
    z, u = s * r, dy * gamma
    m = (u * z).mean(1, keepdim=True)
    ds = 0 if dsum is None else dsum.double()
    dx = ds + r * (u - z * m)
    size = (0 if dsum is None else ds.abs()) + r * (u.abs() + z.abs() * m.abs())
    tol = 2.0 ** -22 * size + r * z.abs() * 2.0 ** -20 * (u * z).abs().mean(1, keepdim=True)
    return dx, (dy * z).sum(0), tol, 2.0 ** -20 * (dy * z).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SHAPES + [(1001, 72), (2500, 136), (400, 4610)])
@pytest.mark.parametrize("dtype,wtype,saved", [(torch.float32, torch.float32, False),
                                               (torch.bfloat16, torch.bfloat16, False),
                                               (torch.float16, torch.float32, False),
                                               (torch.float32, torch.bfloat16, True),
                                               (torch.bfloat16, torch.float32, True),
                                               (torch.float16, torch.float16, True)])
def test_backward(rows, cols, dtype, wtype, saved):
    f = _lib()
    _, x, gamma = inputs(rows, cols, dtype, wtype, rows + cols)
    rstd = plain(x, gamma)[1].float()
    dy = (torch.randn(rows, cols, generator=gen(rows), device="cuda") * 0.1).to(dtype)
    more = (torch.randn(rows, cols, generator=gen(cols), device="cuda") * 0.1).to(dtype)
    seen = x
    if saved:
        x8 = f.BlockFp8.empty(rows, cols, rows % 2, 1, torch.float32 if cols % 2 else torch.uint8)
        f.fp8_block_quantize(x, x8)
        seen = ref.values(x8)[0]
    for k, (l, q) in enumerate([(0, 0), (8, 8), (1, 2)]):
        dsum = None if k == 1 else padded(more, q, 5)
        want, dg, tol, tol_dg = bwd_plain(dy, seen, gamma, rstd, dsum)
        out = torch.empty_like(dy) if k == 0 else padded(dy, 3 if k == 2 else 0, 8)
        dgamma = torch.empty(cols, device="cuda")
        f.fp8_rmsnorm_bwd(padded(dy, l, 0), x8 if saved else padded(x, 0, q), gamma, rstd, out, dgamma,
                          dsum=dsum)
        f.fp8_sync_status()
        near(out, want, tol + h(dtype) * (want.abs() + tol) + tiny(dtype), ("dx", rows, cols, k))
        near(dgamma, dg, tol_dg, "dgamma")


@pytest.mark.parametrize("rows,cols", [(5000, 256), (5000, 251), (9000, 384), (6001, 511), (20000, 264),
                                       (1000, 8200), (700, 12288), (500, 16384), (160, 16392)])
@pytest.mark.parametrize("dtype,wtype,saved", [(torch.float32, torch.bfloat16, False),
                                               (torch.bfloat16, torch.float32, False),
                                               (torch.bfloat16, torch.bfloat16, True),
                                               (torch.float32, torch.float32, True)])
def test_backward_of_several_rows_each(rows, cols, dtype, wtype, saved):
    """More rows than a CTA or a warp has places for, at the widths where the kernels change."""
    test_backward(rows, cols, dtype, wtype, saved)


@pytest.mark.parametrize("rows,cols", [(50, 77), (300, 1024), (170, 4103), (40, 12288)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_in_place_and_repeated(rows, cols, dtype):
    """dx in dy's and in dsum's own memory, with one workspace: the same bits each time."""
    f = _lib()
    _, x, gamma = inputs(rows, cols, dtype, torch.float32, 3)
    rstd = plain(x, gamma)[1].float()
    dy, ds = ((torch.randn(rows, cols, generator=gen(k), device="cuda") * 0.1).to(dtype) for k in (1, 2))
    dx, dg = torch.empty_like(dy), torch.empty(cols, device="cuda")
    ws = torch.empty(f.fp8_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    f.fp8_rmsnorm_bwd(dy, x, gamma, rstd, dx, dg, dsum=ds, workspace=ws)
    for which in range(2):
        a, b, dg2 = dy.clone(), ds.clone(), torch.empty_like(dg)
        f.fp8_rmsnorm_bwd(a, x, gamma, rstd, (a, b)[which], dg2, dsum=b, workspace=ws.fill_(255))
        f.fp8_sync_status()
        assert torch.equal((a, b)[which], dx) and torch.equal(dg2, dg)


def test_gradients_against_differences():
    """dx and dgamma against central differences of the forward in 64 bits: with a step of
    2^-12 they are off by the third derivative's 2^-24 / 6 and the rounding's 2^-52 / 2^-12."""
    f = _lib()
    rows, cols = 4, 96
    _, x, gamma = inputs(rows, cols, torch.float32, torch.float32, 9)
    x[1] += 0.5    # not at the norm's pole
    dy, ds = (torch.randn(rows, cols, generator=gen(k), device="cuda") for k in (1, 2))
    rstd = plain(x, gamma)[1].float()
    dx, dg = torch.empty_like(x), torch.empty(cols, device="cuda")
    f.fp8_rmsnorm_bwd(dy, x, gamma, rstd, dx, dg, dsum=ds)

    def loss(x, gamma):
        return (plain(x, gamma)[0] * dy.double()).sum() + (x.double() * ds.double()).sum()

    step, x, gamma = 2.0 ** -12, x.double(), gamma.double()
    for r, c in [(0, 0), (1, 13), (2, 95), (3, 40)]:
        e = torch.zeros_like(x)
        e[r, c] = step
        want = (loss(x + e, gamma) - loss(x - e, gamma)) / (2 * step)
        assert abs(dx[r, c].double() - want) <= 1e-5 * (1 + abs(want)), (r, c)
        e = torch.zeros_like(gamma)
        e[c] = step
        want = (loss(x, gamma + e) - loss(x, gamma - e)) / (2 * step)
        assert abs(dg[c].double() - want) <= 1e-5 * (1 + abs(want)), c


@pytest.mark.parametrize("rows,cols", [(1, 1), (130, 257), (300, 1000), (64, 4096)])
@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [0, 1])
def test_recompute(rows, cols, wtype, fmt):
    f = _lib()
    _, x, gamma = inputs(rows, cols, torch.bfloat16, wtype, rows + cols)
    x8 = f.BlockFp8.empty(rows, cols)
    f.fp8_block_quantize(x, x8)
    rstd = plain(x, gamma)[1].float()
    yt, bufs = marked(cols, rows, fmt)
    f.fp8_rmsnorm_recompute(x8, gamma, rstd, yt)
    f.fp8_sync_status()
    want = (ref.values(x8)[0] * rstd.double()[:, None] * gamma.double()).t()
    near_block(yt, want, 2.0 ** -22 * want.abs(), "yt")
    assert_marks(yt, bufs, "yt")


def test_empty_and_streams_and_graph():
    """No rows; a stream of its own; two captured passes that share a workspace, replayed on
    new data."""
    f = _lib()
    e = lambda *s: torch.empty(*s, device="cuda")
    gamma, dg = e(7), torch.full((7,), 5.0, device="cuda")
    f.fp8_rmsnorm_fwd(e(0, 7), gamma, EPS, e(0), residual=e(0, 7), sum=e(0, 7), y=e(0, 7))
    f.fp8_rmsnorm_bwd(e(0, 7), e(0, 7), gamma, e(0), e(0, 7), dg)
    torch.cuda.synchronize()
    assert (dg == 0).all()
    rows, cols = 65, 640
    x, r, gamma = inputs(rows, cols, torch.bfloat16, torch.float32, 4)
    s, y, rstd = torch.empty_like(x), torch.empty_like(x), e(rows)
    dx, dgamma = torch.empty_like(x), e(cols)
    ws = torch.empty(f.fp8_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")

    def step(stream=None, workspace=ws):
        f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=r, sum=s, y=y, stream=stream)
        f.fp8_rmsnorm_bwd(y, s, gamma, rstd, dx, dgamma, dsum=r, workspace=workspace, stream=stream)

    def check(what):
        y0 = plain(s, gamma)[0]
        near(y, y0, (2.0 ** -19 + 2 * h(x.dtype)) * y0.abs(), what)
        want, dg0, tol, tol_dg = bwd_plain(y, s, gamma, rstd, r)
        near(dx, want, tol + h(x.dtype) * (want.abs() + tol), what)
        near(dgamma, dg0, tol_dg, what)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side, None)
    torch.cuda.current_stream().wait_stream(side)
    check("side")
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for k in range(4):
        x.copy_(torch.randn(rows, cols, generator=gen(k), device="cuda"))
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        check(("replay", k))


def test_more_than_2_31_elements():
    """Offsets past 32 bits: the last rows of 140000 x 16384 (2.3 G elements)."""
    f = _lib()
    rows, cols = 140000, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = slice(rows - 3, rows)
    g = gen(1)
    x[tail] = torch.randn(3, cols, generator=g, device="cuda").to(torch.bfloat16)
    x[0] = x[rows - 1]
    gamma = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    rstd, dg = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")
    y8 = f.BlockFp8.empty(rows, cols)
    f.fp8_rmsnorm_fwd(x, gamma, EPS, rstd, residual=x, sum=x, y8=y8)   # s = 2 x, exactly
    f.fp8_sync_status()
    y0, rstd0 = plain(x[tail], gamma)
    near(rstd[tail], rstd0, 2.0 ** -20 * rstd0, "rstd")
    part = f.BlockFp8(y8.codes[tail], y8.scales[tail], cols)
    near_block(part, y0, 2.0 ** -19 * y0.abs(), "y8")
    assert torch.equal(y8.codes[0], y8.codes[rows - 1])
    assert (y8.codes[1:rows - 3] & 0x7F == 0).all()   # -0 where gamma is negative
    dx = torch.empty_like(x)
    f.fp8_rmsnorm_bwd(x, x, gamma, rstd, dx, dg, dsum=x)
    f.fp8_sync_status()
    want, _, tol, _ = bwd_plain(x[tail], x[tail], gamma, rstd[tail], x[tail])
    near(dx[tail], want, tol + h(x.dtype) * (want.abs() + tol), "dx")
    assert torch.equal(dx[0], dx[rows - 1]) and (dx[1:rows - 3] == 0).all()
