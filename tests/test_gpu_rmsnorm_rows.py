"""GPU tests of the RMS norm where a CTA has many rows: places of the backward's ring used again
and again at every width, rows summed one after the other into dgamma, in place, and the
forward's loops.

Tolerances, first order in 2^-24, the half step of fp32.  dgamma: a thread adds its CTA's
rows one after the other: ceil(rows / (SMs teams)) of them, or up to 8 where there are so few that
not all CTAs start.  A team is a CTA, one an SM past 4608 columns, two down to 2049, up to 16 below
that; up to 256 columns it is one of a CTA's 8 warps, whose sums are added in turn.  Then a
thread of the join adds at most 2432 / 32 = 76 CTAs' sums and 5 levels follow; xhat is rounded once.
So dgamma is known to (rows of a team + 8 + 76 + 5 + 1) 2^-24 of the sum of its terms' magnitudes,
and no better where they have one sign and round the same way.  dx: u and xhat are rounded once each, the sum over a row takes at most 20
additions of a thread and 10 behind them (2^-19 with u's and xhat's), its mean two more
roundings, and two fused operations end it: 5 roundings of the largest of its terms, 2^-21."""
import pytest
import torch

from test_gpu_block import gen
from test_gpu_rmsnorm import EPS, _lib, inputs, plain, tiny
from test_gpu_rmsnorm import test_forward as check_forward
from test_gpu_saved import h, near
import block_ref as ref

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


def dgamma_tol(rows, cols, size):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    threads = -(-cols // 512) * 32
    teams = 16 if cols <= 512 else 1 if cols > 4608 else 512 // threads if threads <= 128 else 2
    # fewer than 8 rows each only where an SM has one CTA
    each = -(-rows // (sms * teams))
    return ((each if teams == 1 else max(each, 8)) + 90) * UNIT * size


def reference(dy, x, gamma, rstd, dsum, part=1 << 26):
    """dx with its tolerance and dgamma with the sum of its terms' magnitudes, in 64 bits, some
    rows at a time."""
    rows, cols = dy.shape
    some = max(1, part // cols)
    g = gamma.double()
    dg, size = torch.zeros(2, cols, dtype=torch.float64, device="cuda")
    for at in range(0, rows, some):
        cut = slice(at, at + some)
        d, r = dy[cut].double(), rstd[cut].double()[:, None]
        z, u = x[cut].double() * r, d * g
        t = d * z
        dg += t.sum(0)
        size += t.abs().sum(0)
        ds = 0 if dsum is None else dsum[cut].double()
        m = (u * z).mean(1, keepdim=True)
        dx = ds + r * (u - z * m)
        big = r * (u.abs() + z.abs() * m.abs()) + (0 if dsum is None else ds.abs())
        tol = 2.0 ** -21 * big + r * z.abs() * 2.0 ** -19 * (u * z).abs().mean(1, keepdim=True)
        yield cut, dx, tol
    yield dg, size


def check(got, dgamma, dy, x, gamma, rstd, dsum, what):
    for item in reference(dy, x, gamma, rstd, dsum):
        if len(item) == 3:
            cut, dx, tol = item
            near(got[cut], dx, tol + h(dy.dtype) * (dx.abs() + tol) + tiny(dy.dtype), ("dx", *what))
        else:
            near(dgamma, item[0], dgamma_tol(*dy.shape, item[1]), ("dgamma", *what))


def noise(rows, cols, dtype, seed, std=0.1):
    return (torch.randn(rows, cols, generator=gen(seed), device="cuda") * std).to(dtype)


# widths of one, two (512, 288 and 256 threads) and many CTAs an SM, aligned and not, and of the
# kernels of longer rows; the rings hold 1 to 8 rows
WIDTHS = [(3000, 8192), (2500, 4610), (3000, 8191), (3000, 4608), (3000, 4103), (4000, 4096),
          (4000, 2049), (9000, 1032), (1500, 12288), (1000, 8201), (1000, 16392)]


@pytest.mark.parametrize("rows,cols", WIDTHS)
@pytest.mark.parametrize("dtype,wtype,saved", [(torch.float32, torch.bfloat16, False),
                                               (torch.bfloat16, torch.float32, False),
                                               (torch.float16, torch.float16, False),
                                               (torch.bfloat16, torch.bfloat16, True),
                                               (torch.float32, torch.float32, True)])
def test_backward_where_the_ring_goes_round(rows, cols, dtype, wtype, saved):
    f = _lib()
    _, x, gamma = inputs(rows, cols, dtype, wtype, cols)
    rstd = plain(x, gamma)[1].float()
    dy, ds = noise(rows, cols, dtype, 1), noise(rows, cols, dtype, 2)
    seen, kept = x, x
    if saved:
        kept = f.BlockFp8.empty(rows, cols, cols % 2, 1, torch.float32 if rows % 1000 else torch.uint8)
        f.fp8_block_quantize(x, kept)
        seen = ref.values(kept)[0]
    for dsum in (ds, None):
        dx, dgamma = torch.empty_like(dy), torch.empty(cols, device="cuda")
        f.fp8_rmsnorm_bwd(dy, kept, gamma, rstd, dx, dgamma, dsum=dsum)
        f.fp8_sync_status()
        check(dx, dgamma, dy, seen, gamma, rstd, dsum, (rows, cols, dsum is None))


@pytest.mark.parametrize("rows,cols", [(3000, 4103), (2500, 8192), (300, 8201), (900, 12288), (300, 16392),
                                       (300, 16385)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_in_place_of_many_rows(rows, cols, dtype):
    """dx in dy's, in dsum's and in both's own memory: the same bits, and the formula's."""
    f = _lib()
    _, x, gamma = inputs(rows, cols, dtype, torch.float32, 3)
    rstd = plain(x, gamma)[1].float()
    dy, ds = noise(rows, cols, dtype, 1), noise(rows, cols, dtype, 2)
    dx, dg = torch.empty_like(dy), torch.empty(cols, device="cuda")
    f.fp8_rmsnorm_bwd(dy, x, gamma, rstd, dx, dg, dsum=ds)
    f.fp8_sync_status()
    check(dx, dg, dy, x, gamma, rstd, ds, (rows, cols))
    for which in range(2):
        pair, dg2 = (dy.clone(), ds.clone()), torch.empty_like(dg)
        f.fp8_rmsnorm_bwd(pair[0], x, gamma, rstd, pair[which], dg2, dsum=pair[1])
        f.fp8_sync_status()
        assert torch.equal(pair[which], dx) and torch.equal(dg2, dg)
        assert torch.equal(pair[1 - which], (ds, dy)[which])
    both, dg2 = dy.clone(), torch.empty_like(dg)
    f.fp8_rmsnorm_bwd(dy, x, gamma, rstd, dx, dg, dsum=dy)
    f.fp8_rmsnorm_bwd(both, x, gamma, rstd, both, dg2, dsum=both)
    f.fp8_sync_status()
    assert torch.equal(both, dx) and torch.equal(dg2, dg)


@pytest.mark.parametrize("rows,cols", [(1000003, 64), (300000, 260), (60000, 8192), (100000, 4099), (30000, 16384),
                                       (20000, 16391)])
@pytest.mark.parametrize("same", [False, True])
def test_dgamma_of_one_sign_over_many_rows(rows, cols, same):
    """Terms of one sign, random ones and (same) all equal, hundreds of them to a CTA: nothing
    cancels, and equal terms round the same way again and again."""
    f = _lib()
    g = gen(rows)
    if same:
        x = torch.full((1, cols), 1.0 / 3, dtype=torch.bfloat16, device="cuda").expand(rows, cols).contiguous()
        dy = torch.full((1, cols), 0.7, dtype=torch.bfloat16, device="cuda").expand(rows, cols).contiguous()
    else:
        x = torch.rand(rows, cols, generator=g, device="cuda").bfloat16()
        dy = torch.rand(rows, cols, generator=g, device="cuda").bfloat16()
    rstd = 1.2 + torch.rand(rows, generator=g, device="cuda") * (0 if same else 1)
    gamma, dgamma = torch.ones(cols, device="cuda"), torch.empty(cols, device="cuda")
    f.fp8_rmsnorm_bwd(dy, x, gamma, rstd, torch.empty_like(x), dgamma)
    f.fp8_sync_status()
    *_, (want, size) = reference(dy, x, gamma, rstd, None)
    assert torch.equal(want, size)
    near(dgamma, want, dgamma_tol(rows, cols, size), "dgamma")


def test_dgamma_past_2_31_elements():
    """140000 x 16384, all zeros but the first, the last three and one in between: zeros add
    nothing, so that dgamma is the sum of five rows, known to 8 + 5 + 5 + 1 roundings."""
    f = _lib()
    rows, cols = 140000, 16384
    at = [0, 77777, rows - 3, rows - 2, rows - 1]
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    for k, r in enumerate(at):
        x[r] = noise(1, cols, torch.bfloat16, k, 1)[0]
        dy[r] = noise(1, cols, torch.bfloat16, k + 9)[0]
    gamma = 1 + 0.3 * torch.randn(cols, generator=gen(1), device="cuda")
    rstd = torch.full((rows,), EPS ** -0.5, device="cuda")
    rstd[at] = plain(x[at], gamma)[1].float()
    dgamma = torch.empty(cols, device="cuda")
    f.fp8_rmsnorm_bwd(dy, x, gamma, rstd, dy, dgamma)   # in place: dy is kept in five rows alone
    f.fp8_sync_status()
    d = torch.stack([noise(1, cols, torch.bfloat16, k + 9)[0] for k in range(5)]).double()
    t = d * x[at].double() * rstd[at].double()[:, None]
    near(dgamma, t.sum(0), 19 * UNIT * t.abs().sum(0), "dgamma")


@pytest.mark.parametrize("rows,cols", [(9001, 40), (5001, 512), (2500, 520), (1301, 4096), (1300, 4099), (701, 5120),
                                       (650, 5121), (500, 8192), (500, 8191), (321, 12288), (321, 8200), (1300, 16392)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward_of_several_rows_each(rows, cols, dtype):
    """More rows than are in work at once, at the widths where the kernels change."""
    check_forward(rows, cols, dtype, torch.float32)
