"""GPU tests of the block-scaled quantizer and matrix product against plain
implementations in 64 bits (block_ref.py).

Tolerances.  The quantizer is exact: a division by a power of two and one
rounding, so codes and scales are compared bit for bit (NaN codes as a class).
The product: half a step of BF16 of the result, 2^-8 |D|, for the final
rounding, and for the sums, with P = sum of |a b| sA sB: at most 2^-23 P for
each of the ~ 128 + K / 128 additions a term passes through."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def spread(rows, cols, dtype, seed):
    """Values over many orders of magnitude from block to block, with zero blocks, NaN,
    infinities, subnormals and amaxes at the border between two scales."""
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float64)
    top = 12 if dtype == torch.float16 else 100
    e = torch.randint(-2 * top // 3, top, (rows, -(-cols // 128)), generator=g, device="cuda")
    x = x * ref.pow2(e.clamp(-140, 120)).repeat_interleave(128, 1)[:, :cols]
    x = x.to(dtype)
    tiny = torch.finfo(dtype).smallest_normal
    flat = x.view(-1)
    n = flat.numel()

    def put(k, value):
        at = torch.randint(0, n, (max(1, n // k),), generator=g, device="cuda")
        flat[at] = value

    put(97, float("inf")), put(101, float("-inf")), put(89, float("nan")), put(31, 0.0)
    put(37, -0.0), put(53, tiny / 4)
    if rows > 3:
        x[1] = 0
        x[2] = float("nan")
        x[3] = tiny / 8
    if rows > 6:   # amax exactly at, and just above, 1.75 times a power of two
        x[4] = x[4].clamp(-1, 1).nan_to_num(0.5)
        x[4, ::128] = 1.75
        x[5] = x[4]
        x[5, ::128] = torch.nextafter(torch.tensor(1.75, dtype=torch.float32),
                                      torch.tensor(2.0)).item() if dtype == torch.float32 \
            else 1.75 * (1 + torch.finfo(dtype).eps)
        x[6] = torch.finfo(dtype).max
    return x


def nan_code(c, fmt):
    m = c & 0x7F
    return (m == 0x7F) if fmt == ref.E4M3 else (m > 0x7C)


def assert_block(q, codes, scales, what):
    rows, cols = q.shape
    got = q.codes[:, :cols]
    bad = (got != codes) & ~(nan_code(got, q.fmt) & nan_code(codes, q.fmt))
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist())
    s = q.scales[: scales.shape[0], : scales.shape[1]]
    if s.dtype == torch.float32:
        assert torch.equal(s.double(), ref.scale_values(scales)), what
    else:
        assert torch.equal(s, scales), (what, torch.nonzero(s != scales)[:4].tolist())


def marked(rows, cols, fmt=0, block_rows=1, scale_dtype=torch.uint8, pitch=None):
    """Buffers filled with a mark, wider than they need be."""
    f = _lib()
    pitch = -(-cols // 16) * 16 + 32 if pitch is None else pitch
    codes = torch.full((rows + 1, pitch), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-rows // block_rows) + 1, -(-cols // 512) * 4 + 4), 0x5A,
                   dtype=torch.uint8, device="cuda")
    if scale_dtype == torch.float32:
        s = torch.full(s.shape, -77.0, device="cuda")
    return f.BlockFp8(codes[:rows], s[:-1], cols, fmt, block_rows), (codes, s)


def assert_marks(q, bufs, what):
    codes, s = bufs
    rows, cols = q.shape
    assert (codes[rows:] == 0xA5).all() and (codes[:, cols:] == 0xA5).all(), what
    mark = 0x5A if s.dtype == torch.uint8 else -77.0
    nb = -(-cols // 128)
    assert (s[-1] == mark).all() and (s[:, nb:] == mark).all(), what


SHAPES = [(1, 1), (1, 128), (3, 5), (7, 129), (127, 128), (128, 127), (129, 257), (130, 16),
          (300, 1000), (16, 4097)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize(rows, cols, dtype, fmt):
    f = _lib()
    x = spread(rows, cols, dtype, rows * 7 + cols + fmt)
    wide = torch.zeros(rows, cols + 24, dtype=dtype, device="cuda")
    wide[:, 8:8 + cols] = x      # 16-byte aligned for 16-bit types at an even pitch
    odd = torch.zeros(rows, cols + 3, dtype=dtype, device="cuda")
    odd[:, 1:1 + cols] = x
    for br in (1, 128):
        want, want_t = ref.quantize(x, fmt, br), ref.quantize(x.t(), fmt, br)
        for src, sd, ways in [(x, torch.uint8, "both"), (wide[:, 8:8 + cols], torch.float32, "rows"),
                              (odd[:, 1:1 + cols], torch.uint8, "cols"),
                              (wide[:, 8:8 + cols], torch.uint8, "cols"),
                              (odd[:, 1:1 + cols], torch.uint8, "rows")]:
            what = (rows, cols, dtype, fmt, br, ways)
            q, qb = marked(rows, cols, fmt, br, sd)
            qt, qtb = marked(cols, rows, fmt, br, sd)
            f.fp8_block_quantize(src, q if ways != "cols" else None, qt if ways != "rows" else None)
            torch.cuda.synchronize()
            if ways != "cols":
                assert_block(q, *want, what)
                assert_marks(q, qb, what)
            if ways != "rows":
                assert_block(qt, *want_t, what)
                assert_marks(qt, qtb, what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt,br,sd", [(0, 1, torch.uint8), (1, 1, torch.float32),
                                       (0, 128, torch.float32), (1, 128, torch.uint8)])
def test_dequantize(dtype, fmt, br, sd):
    f = _lib()
    for rows, cols in [(1, 1), (5, 130), (129, 1031), (3, 4096)]:
        q, _ = marked(rows, cols, fmt, br, sd)
        q.codes.copy_(torch.randint(0, 256, q.codes.shape, generator=gen(3), device="cuda"))
        e = torch.randint(110, 140, q.scales.shape, generator=gen(4), device="cuda").to(torch.uint8)
        q.scales.copy_(e if sd == torch.uint8 else ref.scale_values(e) * 1.37)
        if sd == torch.uint8:
            q.scales[0, 0] = 255     # a NaN scale
        want = ref.values(q)[0]
        out = torch.full((rows, cols + 1), 9.0, dtype=dtype, device="cuda")
        f.fp8_block_dequantize(q, out[:, :cols])
        # one rounding to fp32 (the product) and one to the type
        exp = want.float().to(dtype)
        assert torch.equal(out[:, :cols].isnan(), exp.isnan())
        assert torch.equal(out[:, :cols].nan_to_num(1), exp.nan_to_num(1)), (rows, cols)
        assert (out[:, cols] == 9).all()
    assert q.dequantize(dtype).shape == (3, 4096)


def operand(rows, K, fmt, br, sd, seed):
    """Random codes of every finite size, scales that vary by block, NaN codes beyond the columns."""
    f = _lib()
    g = gen(seed)
    pitch = -(-K // 16) * 16
    codes = torch.full((rows, pitch), 0x7F, dtype=torch.uint8, device="cuda")
    v = torch.randn(rows, K, generator=g, device="cuda") * (100 if fmt == 0 else 3000)
    codes[:, :K] = v.clamp(-448, 448).to(ref.F8[fmt]).view(torch.uint8) if fmt == 0 else \
        v.to(ref.F8[fmt]).view(torch.uint8)
    shape = (-(-rows // br), -(-K // 512) * 4)
    if sd == torch.uint8:
        s = torch.randint(115, 125, shape, generator=g, device="cuda", dtype=torch.uint8)
        s[:, -(-K // 128):] = 255    # scales of blocks that do not exist
    else:
        s = torch.exp2(torch.randn(shape, generator=g, device="cuda") * 3 - 6)
        s[:, -(-K // 128):] = float("nan")
    return f.BlockFp8(codes, s, K, fmt, br)


def check_gemm(A, B, D, what, spare=None):
    a, _ = ref.values(A)
    b, _ = ref.values(B)
    want = a @ b.t()
    P = a.abs() @ b.abs().t()
    K = A.cols
    tol = 2.0 ** -8 * want.abs() + (128 + K / 128) * 2.0 ** -23 * P
    off = (D.double() - want).abs()
    assert (off <= tol).all(), (what, float((off - tol).max()), torch.nonzero(~(off <= tol))[:4].tolist())


GEMM_SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 512), (2, 130, 4096), (5, 77, 200), (16, 256, 640),
               (17, 1000, 1000), (33, 384, 2048), (64, 129, 129), (65, 128, 384), (100, 500, 300),
               (128, 256, 1024), (129, 257, 127), (200, 64, 1536), (256, 256, 256), (300, 700, 900),
               (513, 1031, 640), (1000, 24, 1111)]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
def test_gemm(M, N, K, sd):
    f = _lib()
    for i, (fa, fb, ba, bb) in enumerate([(0, 0, 1, 128), (1, 0, 1, 1), (0, 1, 128, 1),
                                          (1, 1, 128, 128)]):
        A, B = operand(M, K, fa, ba, sd, M + i), operand(N, K, fb, bb, sd, N + 7 * i)
        for pad in (0, 8 - N % 8):     # rows of D contiguous, and aligned
            D = torch.full((M + 1, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            f.fp8_block_gemm_tn(A, B, D[:M, :N])
            f.fp8_sync_status()
            check_gemm(A, B, D[:M, :N], (M, N, K, sd, fa, fb, ba, bb, pad))
            assert (D[M] == 7).all() and (D[:, N:] == 7).all()


@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
@pytest.mark.parametrize("M,N,K", [(2048, 4096, 1024), (3, 11008, 4096), (48, 4096, 11008),
                                   (1500, 2600, 3500)])
def test_gemm_larger(M, N, K, sd):
    f = _lib()
    A, B = operand(M, K, 0, 1, sd, 1), operand(N, K, 0, 128, sd, 2)
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    f.fp8_block_gemm_tn(A, B, D)
    again = torch.empty_like(D)
    f.fp8_block_gemm_tn(A, B, again)
    f.fp8_sync_status()
    check_gemm(A, B, D, (M, N, K, sd))
    assert torch.equal(D, again)


@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
@pytest.mark.parametrize("bb", [1, 128])
@pytest.mark.parametrize("M,N,K", [(2200, 2250, 300), (2304, 2305, 1100), (2500, 2503, 640),
                                   (2560, 2560, 130), (4900, 4801, 40)])
def test_gemm_last_wave_in_pieces(M, N, K, sd, bb):
    """A few more 256 x 256 tiles than CTA pairs: the last ones are cut by columns."""
    f = _lib()
    A, B = operand(M, K, 1, 1, sd, M), operand(N, K, 0, bb, sd, N)
    for pad in (0, 8 - N % 8):
        D = torch.full((M + 1, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        f.fp8_block_gemm_tn(A, B, D[:M, :N])
        f.fp8_sync_status()
        check_gemm(A, B, D[:M, :N], (M, N, K, sd, bb, pad))
        assert (D[M] == 7).all() and (D[:, N:] == 7).all()


@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
@pytest.mark.parametrize("M,N,K", [(4, 256, 512), (300, 256, 512)])
def test_gemm_special_values(M, N, K, sd):
    """NaN codes, NaN scales, infinities (E5M2) and a block of zeros under the smallest scale."""
    f = _lib()
    A, B = operand(M, K, 1, 1, sd, 5), operand(N, K, 0, 128, sd, 6)
    A.codes[0, 3] = 0x7C            # +inf
    A.codes[1, 130] = 0x7E          # NaN
    B.codes[9, 400] = 0x7F          # NaN
    A.codes[2, 128:256] = 0
    if sd == torch.uint8:
        A.scales[2, 1] = 0
        A.scales[3, 2] = 255
    else:
        A.scales[2, 1] = 2.0 ** -127
        A.scales[3, 2] = float("nan")
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    f.fp8_block_gemm_tn(A, B, D)
    f.fp8_sync_status()
    assert D[1].isnan().all() and D[3].isnan().all() and D[:, 9].isnan().all()
    b0 = ref.values(B)[0][:, 3]
    ok = torch.ones(N, dtype=torch.bool, device="cuda")
    ok[9] = False
    assert torch.equal(D[0][ok & (b0 != 0)].float(),
                       torch.where(b0 > 0, float("inf"), float("-inf"))[ok & (b0 != 0)].float())
    a, b = ref.values(A)[0], ref.values(B)[0]
    want, P = a[2] @ b[ok].t(), a[2].abs() @ b[ok].abs().t()
    assert ((D[2][ok].double() - want).abs() <= 2.0 ** -8 * want.abs() + 132 * 2.0 ** -23 * P).all()


def test_gemm_without_columns_is_zero():
    f = _lib()
    q = lambda n: f.BlockFp8(torch.empty(n, 0, dtype=torch.uint8, device="cuda"),
                             torch.empty(n, 0, dtype=torch.uint8, device="cuda"), 0)
    D = torch.full((6, 12), 5.0, dtype=torch.bfloat16, device="cuda")
    f.fp8_block_gemm_tn(q(6), q(9), D[:, :9])
    torch.cuda.synchronize()
    assert (D[:, :9] == 0).all() and (D[:, 9:] == 5).all()


def test_empty_calls_do_nothing():
    f = _lib()
    e = f.BlockFp8.empty
    f.fp8_block_quantize(torch.empty(0, 7, device="cuda"), e(0, 7), e(7, 0))
    f.fp8_block_quantize(torch.empty(7, 0, device="cuda"), e(7, 0), e(0, 7))
    f.fp8_block_dequantize(e(0, 7), torch.empty(0, 7, device="cuda"))
    f.fp8_block_gemm_tn(e(0, 64), e(5, 64), torch.empty(0, 5, dtype=torch.bfloat16, device="cuda"))
    f.fp8_block_gemm_tn(e(5, 64), e(0, 64), torch.empty(5, 0, dtype=torch.bfloat16, device="cuda"))
    f.fp8_sync_status()


def test_other_streams_and_graphs():
    """On a stream of its own, and captured into a graph that is replayed on new data."""
    f = _lib()
    M, N, K = 70, 384, 512
    x = torch.randn(M, K, device="cuda")
    B = operand(N, K, 0, 128, torch.uint8, 3)
    q, qt = f.BlockFp8.empty(M, K), f.BlockFp8.empty(K, M)
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f.fp8_block_quantize(x, q, qt, stream=side)
    f.fp8_block_gemm_tn(q, B, D, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    check_gemm(q, B, D, "side stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.fp8_block_quantize(x, q, qt)
        f.fp8_block_gemm_tn(q, B, D)
    for seed in range(2):
        x.copy_(torch.randn(M, K, generator=gen(seed), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert_block(q, *ref.quantize(x, 0), "replay")
        assert_block(qt, *ref.quantize(x.t(), 0), "replay")
        check_gemm(q, B, D, "replay")
