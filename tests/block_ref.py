"""Plain implementations in 64 bits of the block-scaled operators, for their tests.

A block-scaled value is code * scale.  The scale of a block is the smallest
power of two 2^e, e >= -127, with amax <= fmax 2^e over the block's finite
values, found here by trying every e; a code is the nearest value of the format, found by
searching the table of all of them, ties to the even code."""
import torch

E4M3, E5M2 = 0, 1
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
FMAX = {E4M3: 448.0, E5M2: 57344.0}


def _table(fmt):
    """Non-negative finite values in the order of their codes."""
    v = torch.arange(128, dtype=torch.uint8).view(F8[fmt]).double()
    return v[torch.isfinite(v)]


def scale_exponent(amax, fmt):
    """e of the definition for every entry of amax (double)."""
    es = torch.arange(-127, 128, dtype=torch.float64, device=amax.device)
    fits = amax.unsqueeze(-1) <= torch.ldexp(torch.full_like(es, FMAX[fmt]).cpu(),
                                             es.cpu().to(torch.int32)).to(amax.device)
    return es[fits.to(torch.int8).argmax(-1)].to(torch.int64)


def pow2(e):
    """2^e, exactly (from its bits)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def nearest_code(q, fmt):
    """Code (uint8) of the nearest value; ties to even; NaN gives 0x7F."""
    t = _table(fmt).to(q.device)
    a = q.abs().clamp(max=FMAX[fmt])
    hi = torch.searchsorted(t, torch.nan_to_num(a)).clamp(max=len(t) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - t[lo], t[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = pick.to(torch.int64) + 128 * torch.signbit(q)
    return torch.where(q.isnan(), 0x7F, code).to(torch.uint8)


def quantize(x, fmt, block_rows=1):
    """x [rows, cols] (any type) -> codes uint8 [rows, cols], scale bytes uint8."""
    x = x.double()
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    v = torch.zeros(br * block_rows, bc * 128, dtype=torch.float64, device=x.device)
    v[:rows, :cols] = x
    v = v.view(br, block_rows, bc, 128)
    amax = torch.where(v.isfinite(), v.abs(), torch.zeros_like(v)).amax((1, 3))
    e = scale_exponent(amax, fmt)
    codes = nearest_code(v / pow2(e)[:, None, :, None], fmt)
    return codes.view(br * block_rows, bc * 128)[:rows, :cols], (e + 127).to(torch.uint8)


def scale_values(scales):
    if scales.dtype == torch.uint8:
        return torch.where(scales == 255, float("nan"), pow2(scales.to(torch.int64) - 127))
    return scales.double()


def values(q):
    """What a BlockFp8 stands for, in double, and its scales spread over the elements."""
    rows, cols = q.shape
    s = scale_values(q.scales)[: -(-rows // q.block_rows), : -(-cols // 128)]
    s = s.repeat_interleave(q.block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q.codes[:, :cols].contiguous().view(F8[q.fmt]).double() * s, s


def layernorm(x, gamma, beta, eps):
    x, gamma, beta = x.double(), gamma.double(), beta.double()
    mean = x.mean(1)
    rstd = (((x - mean[:, None]) ** 2).mean(1) + eps) ** -0.5
    return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def layernorm_bwd(dy, x, gamma, mean, rstd):
    dy, x, gamma, r = dy.double(), x.double(), gamma.double(), rstd.double()[:, None]
    xhat = (x - mean.double()[:, None]) * r
    u = dy * gamma
    dx = r * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def swiglu(h):
    g, u = h.double().chunk(2, 1)
    return g * torch.sigmoid(g) * u


def swiglu_bwd(da, h):
    g, u = h.double().chunk(2, 1)
    da, s = da.double(), torch.sigmoid(g)
    return torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
