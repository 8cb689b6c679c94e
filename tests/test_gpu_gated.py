"""GPU tests of the gated feed-forward product, forward and backward, against plain
implementations in 64 bits (block_ref.py).

Tolerances.  The product's sums, with P = sum of |a b| sA sB: at most 2^-23 P for each of
the 128 + K / 128 additions a term passes through; nothing is rounded behind them.  An
error e of g, u or da moves the results by the formulas' slopes, of which that of g * s(g)
is at most 1.1.  The elementwise arithmetic: 2^-20 and |g| 2^-22 of a result's terms, as
for fp8_swiglu_fwd and fp8_swiglu_bwd.  Values in 8 bits: half a step of the format at that
size under the block's scale, and the scale what the definition gives for a maximum within the
tolerance."""
import pytest
import torch

import block_ref as ref
from test_gpu_block import assert_marks, gen, marked, nan_code
from test_gpu_saved import near

pytestmark = pytest.mark.gpu


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def held(rows, cols, std, fmt, block, seed, spread=True):
    """Normal values in 8 bits, their size differing from block to block; codes beyond the
    columns are NaN, scales of blocks that do not exist too."""
    f = _lib()
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    if spread:
        x *= torch.exp2(torch.randint(-3, 2, (rows, -(-cols // 128)), generator=g,
                                      device="cuda").float()).repeat_interleave(128, 1)[:, :cols]
    q = f.BlockFp8.empty(rows, cols, fmt, block)
    q.codes.fill_(0x7F), q.scales.fill_(255)
    f.fp8_block_quantize(x, q)
    return q


def near_q(q, want, tol, what):
    """q holds want, known to tol, quantized with blocks along its columns."""
    got, s = ref.values(q)
    least, bits = (-6, 4) if q.fmt == 0 else (-14, 3)
    half = torch.maximum(want.abs() * 2.0 ** -bits, s * 2.0 ** (least - bits))
    near(got, want, half + 2 * tol, what)
    rows, cols = q.shape
    nb = -(-cols // 128)

    def exponent(v):
        w = torch.zeros(rows, nb * 128, dtype=torch.float64, device=v.device)
        w[:, :cols] = v
        return ref.scale_exponent(w.view(rows, nb, 128).amax(2), q.fmt)

    e = scale_bytes(q)[:rows, :nb].to(torch.int64) - 127
    assert ((exponent((want.abs() - tol).clamp(min=0)) <= e) & (e <= exponent(want.abs() + tol))).all(), what


def scale_bytes(q):
    if q.scales.dtype == torch.uint8:
        return q.scales
    return (torch.frexp(q.scales.double()).exponent + 126).to(torch.uint8)


def product(A, B):
    a, b = ref.values(A)[0], ref.values(B)[0]
    return a @ b.t(), (128 + A.cols / 128) * 2.0 ** -23 * (a.abs() @ b.abs().t())


def fwd_plain(A, B):
    """h, a and their tolerances."""
    h, eh = product(A, B)
    (g, u), (eg, eu) = h.chunk(2, 1), eh.chunk(2, 1)
    s = torch.sigmoid(g)
    a = g * s * u
    ta = 1.1 * u.abs() * eg + (g * s).abs() * eu + 1.1 * eg * eu + a.abs() * (2.0 ** -20 + g.abs() * 2.0 ** -22)
    return h, a, eh, ta


def check_fwd(A, B, fmt_a, fmt_h, sd, what):
    f = _lib()
    M, F = A.rows, B.rows // 2
    a8, ab = marked(M, F, fmt_a, 1, sd)
    h8, hb = marked(M, 2 * F, fmt_h, 1, sd)
    f.fp8_block_gemm_swiglu_fwd(A, B, a8, h8)
    f.fp8_sync_status()
    h, a, eh, ta = fwd_plain(A, B)
    near_q(h8, h, eh, ("h8", what))
    near_q(a8, a, ta, ("a8", what))
    assert_marks(a8, ab, what)
    assert_marks(h8, hb, what)
    alone, bufs = marked(M, F, fmt_a, 1, sd)
    f.fp8_block_gemm_swiglu_fwd(A, B, alone)
    f.fp8_sync_status()
    assert torch.equal(alone.codes, a8.codes) and torch.equal(alone.scales, a8.scales), what
    assert_marks(alone, bufs, what)


SHAPES = [(1, 128, 1), (1, 256, 128), (1, 2688, 4096), (3, 384, 127), (7, 128, 200), (16, 640, 1000),
          (17, 512, 640), (32, 1152, 512), (48, 2688, 1031), (65, 128, 513), (128, 384, 384),
          (129, 256, 257), (256, 128, 1024), (300, 640, 1000), (513, 1152, 130), (777, 2688, 1000)]


@pytest.mark.parametrize("M,F,K", SHAPES)
@pytest.mark.parametrize("fa,fb,block_b", [(0, 0, 128), (1, 0, 1), (0, 1, 128)])
def test_forward(M, F, K, fa, fb, block_b):
    A = held(M, K, 1.0, fa, 1, M + K)
    B = held(2 * F, K, 1.5 * K ** -0.5, fb, block_b, F)
    check_fwd(A, B, fa, fb, torch.float32 if fa else torch.uint8, (M, F, K))


@pytest.mark.parametrize("M,F,K", [(2100, 2688, 300), (4100, 4096, 130), (8, 11008, 1000), (200, 11008, 640),
                                   (1100, 5504, 1500), (2048, 1024, 4096)])
def test_forward_where_its_loops_go_round_several_times(M, F, K):
    A, B = held(M, K, 1.0, 0, 1, 1), held(2 * F, K, 1.5 * K ** -0.5, 0, 128, 2)
    check_fwd(A, B, 0, 0, torch.uint8, (M, F, K))


@pytest.mark.parametrize("M", [2, 20, 60, 100, 300])
def test_forward_with_block_of_a_and_odd_pitches(M):
    """A with a scale per tile, views into wider buffers."""
    f = _lib()
    F, K = 384, 700
    A, B = held(M, K, 1.0, 0, 128, 3), held(2 * F, K, 0.05, 1, 128, 4)

    def wider(q):
        codes = torch.full((q.rows + 2, q.codes.shape[1] + 48), 0x7F, dtype=torch.uint8, device="cuda")
        scales = torch.full((q.scales.shape[0] + 2, q.scales.shape[1] + 8), 255, dtype=torch.uint8, device="cuda")
        codes[1:-1, 16:16 + q.codes.shape[1]] = q.codes
        scales[1:-1, 4:4 + q.scales.shape[1]] = q.scales
        return f.BlockFp8(codes[1:-1, 16:16 + q.codes.shape[1]], scales[1:-1, 4:4 + q.scales.shape[1]], q.cols,
                          q.fmt, q.block_rows)

    check_fwd(wider(A), wider(B), 0, 1, torch.uint8, M)


@pytest.mark.parametrize("M", [4, 40, 300])
def test_forward_special_values(M):
    """NaN and infinite operands spoil their own rows or columns, and blocks take their scale from
    what is finite; a row of zeros; gates far below 0 and far above it."""
    f = _lib()
    F, K = 256, 256
    A, B = held(M, K, 1.0, 1, 1, 5, False), held(2 * F, K, 0.1, 0, 128, 6, False)
    A.codes[0, 130] = 0x7E              # NaN
    A.codes[1, 3] = 0x7C                # +inf
    A.codes[2] = 0
    A.scales[3] = 127 + 30              # products around 2^32: SiLU 0 or the gate itself
    B.codes[5, 7] = 0x7F                # NaN in one gate row
    a8, h8 = f.BlockFp8.empty(M, F), f.BlockFp8.empty(M, 2 * F)
    f.fp8_block_gemm_swiglu_fwd(A, B, a8, h8)
    f.fp8_sync_status()
    av, hv = ref.values(a8)[0], ref.values(h8)[0]
    assert av[0].isnan().all() and hv[0].isnan().all()
    assert nan_code(a8.codes[:, 5], 0).all() and nan_code(h8.codes[:, 5], 0).all()
    ok = torch.ones(2 * F, dtype=torch.bool, device="cuda")
    ok[5] = False
    okf = ok[:F]
    # an infinity saturates the codes and is not in the scale: its block has nothing finite but 0
    b3 = ref.values(B)[0][:, 3]
    assert torch.equal(hv[1][ok & (b3 != 0)].sign(), b3[ok & (b3 != 0)].sign())
    assert (scale_bytes(h8)[1] == 0).all()
    assert (av[2][okf] == 0).all() and (hv[2][ok] == 0).all()
    rows = [r for r in range(M) if r > 2]
    Ar = f.BlockFp8(A.codes[rows], A.scales[rows], K, 1)
    B.codes[5, 7] = 0
    h, a, eh, ta = fwd_plain(Ar, B)
    pick = lambda q, r: f.BlockFp8(q.codes[r], q.scales[r], q.cols, q.fmt)
    sub = pick(h8, rows)
    got = ref.values(sub)[0]
    half = torch.maximum(h.abs() * 2.0 ** -4, ref.values(sub)[1] * 2.0 ** -10)
    assert ((got - h).abs() <= half + 2 * eh)[:, ok].all()
    sub = pick(a8, rows)
    got = ref.values(sub)[0]
    half = torch.maximum(a.abs() * 2.0 ** -4, ref.values(sub)[1] * 2.0 ** -10)
    assert ((got - a).abs() <= half + 2 * ta)[:, okf].all()


def bwd_plain(A, B, h8):
    da, ed = product(A, B)
    h = ref.values(h8)[0]
    g, u = h.chunk(2, 1)
    dh, a, s = ref.swiglu_bwd(da, h), ref.swiglu(h), torch.sigmoid(g)
    rel = 2.0 ** -20 + g.abs() * 2.0 ** -22
    # 1 + g (1 - s) cancels for negative gates: its terms' size counts
    slope = u.abs() * s * (1 + g.abs() * (1 - s) + g.abs())
    tol = torch.cat([da.abs() * slope * rel + ed * slope * (1 + rel),
                     da.abs() * (g * s).abs() * rel + ed * (g * s).abs() * (1 + rel)], 1) + 1e-37
    return dh, a, tol, a.abs() * rel + 1e-37


def check_bwd(A, B, h8, fmt, fmt_a, sd, what, parts=True):
    f = _lib()
    M, F = A.rows, B.rows
    outs = [((M, 2 * F), fmt), ((2 * F, M), fmt), ((F, M), fmt_a)]
    bufs = [marked(*shape, k, 1, sd) for shape, k in outs]
    f.fp8_block_gemm_swiglu_bwd(A, B, h8, *(b[0] for b in bufs))
    f.fp8_sync_status()
    dh, a, tol, tol_a = bwd_plain(A, B, h8)
    near_q(bufs[0][0], dh, tol, ("dh8", what))
    near_q(bufs[1][0], dh.t(), tol.t(), ("dh8t", what))
    near_q(bufs[2][0], a.t(), tol_a.t(), ("a8t", what))
    for q, b in bufs:
        assert_marks(q, b, what)
    for i in range(3 if parts else 0):   # any of the three alone is the same
        one = [None, None, None]
        q, b = marked(*outs[i][0], outs[i][1], 1, sd)
        one[i] = q
        f.fp8_block_gemm_swiglu_bwd(A, B, h8, *one)
        f.fp8_sync_status()
        assert torch.equal(q.codes, bufs[i][0].codes) and torch.equal(q.scales, bufs[i][0].scales), (what, i)
        assert_marks(q, b, what)


@pytest.mark.parametrize("M,F,K", SHAPES)
@pytest.mark.parametrize("fmt,fmt_a,fmt_h", [(1, 0, 0), (0, 1, 1)])
def test_backward(M, F, K, fmt, fmt_a, fmt_h):
    A = held(M, K, 1e-3, fmt, 1, M + K)
    B = held(F, K, K ** -0.5, fmt_a, 128 if fmt else 1, F)
    h8 = held(M, 2 * F, 1.5, fmt_h, 1, 3)
    check_bwd(A, B, h8, fmt, fmt_a, torch.float32 if fmt else torch.uint8, (M, F, K))


@pytest.mark.parametrize("M,F,K", [(2100, 5504, 300), (4100, 4096, 130), (300, 11008, 640), (2048, 1024, 4096)])
def test_backward_where_its_loops_go_round_several_times(M, F, K):
    A, B, h8 = held(M, K, 1e-3, 1, 1, 1), held(F, K, K ** -0.5, 0, 128, 2), held(M, 2 * F, 1.5, 0, 1, 3)
    check_bwd(A, B, h8, 1, 0, torch.uint8, (M, F, K), parts=False)


def test_backward_special_values():
    """A NaN of dy, of h8 and of B stay where they belong; infinities are not in the scales."""
    f = _lib()
    M, F, K = 200, 256, 256
    A, B, h8 = held(M, K, 1e-3, 1, 1, 1), held(F, K, K ** -0.5, 0, 128, 2), held(M, 2 * F, 1.5, 1, 1, 3)
    A.codes[3, 5] = 0x7E
    h8.codes[7, 9] = 0x7F               # one gate
    h8.codes[8, F + 10] = 0x7C          # one value: +inf
    B.codes[20, 30] = 0x7F
    dh8, dh8t, a8t = f.BlockFp8.empty(M, 2 * F, 1), f.BlockFp8.empty(2 * F, M, 1), f.BlockFp8.empty(F, M)
    f.fp8_block_gemm_swiglu_bwd(A, B, h8, dh8, dh8t, a8t)
    f.fp8_sync_status()
    bad = torch.zeros(M, 2 * F, dtype=torch.bool, device="cuda")
    bad[3] = bad[:, 20] = bad[:, F + 20] = bad[7, 9] = bad[7, F + 9] = True
    v, vt, at = ref.values(dh8)[0], ref.values(dh8t)[0].t(), ref.values(a8t)[0].t()
    assert torch.equal(v.isnan(), bad) and torch.equal(vt.isnan(), bad)
    bad_a = torch.zeros(M, F, dtype=torch.bool, device="cuda")
    bad_a[7, 9] = True
    assert torch.equal(at.isnan(), bad_a)
    dh, a, tol, tol_a = bwd_plain(A, B, h8)
    odd = bad.clone()
    odd[8, 10] = odd[8, F + 10] = True
    for got, q, want, t, skip in [(v, ref.values(dh8)[1], dh, tol, odd), (vt, ref.values(dh8t)[1].t(), dh, tol, odd),
                                  (at, ref.values(a8t)[1].t(), a, tol_a, odd[:, :F] & odd[:, F:])]:
        bits, least = (3, -14) if got is not at else (4, -6)
        half = torch.maximum(want.abs() * 2.0 ** -bits, q * 2.0 ** (least - bits))
        off = (got - want).abs() <= half + 2 * t
        assert off[~skip].all()


def test_gradients_against_differences():
    """dh against central differences of the forward's formula in 64 bits, to half a step of E4M3
    and the step's error."""
    f = _lib()
    M, F, K = 40, 128, 256
    A, B, h8 = held(M, K, 1.0, 0, 1, 1), held(F, K, K ** -0.5, 0, 128, 2), held(M, 2 * F, 1.5, 0, 1, 3)
    dh8 = f.BlockFp8.empty(M, 2 * F)
    f.fp8_block_gemm_swiglu_bwd(A, B, h8, dh8)
    f.fp8_sync_status()
    da, ed = product(A, B)
    h, t = ref.values(h8)[0], 1e-5
    g, u = h.chunk(2, 1)
    up = lambda dg, du: (g + dg) * torch.sigmoid(g + dg) * (u + du)
    num = torch.cat([da * (up(t, 0) - up(-t, 0)) / (2 * t), da * (up(0, t) - up(0, -t)) / (2 * t)], 1)
    got, s = ref.values(dh8)
    slope = torch.cat([1.1 * u.abs(), (g * torch.sigmoid(g)).abs()], 1)
    tol = num.abs() * 2.0 ** -4 + s * 2.0 ** -10 + 2 * torch.cat([ed, ed], 1) * slope + 1e-8 * (1 + da.abs().max())
    assert ((got - num).abs() <= tol).all()


def test_equal_calls_give_equal_bits_on_any_stream_and_in_graphs():
    f = _lib()
    M, F, K = 300, 640, 512
    A, B, W = held(M, K, 1.0, 0, 1, 1), held(2 * F, K, 0.07, 0, 128, 2), held(F, K, 0.05, 0, 128, 4)
    few = f.BlockFp8(A.codes[:5], A.scales[:5], K)

    def outs():
        e = f.BlockFp8.empty
        return (e(M, F), e(M, 2 * F), e(M, 2 * F, 1), e(2 * F, M, 1), e(F, M), e(5, F))

    def step(o, stream=None):
        f.fp8_block_gemm_swiglu_fwd(A, B, o[0], o[1], stream)
        f.fp8_block_gemm_swiglu_bwd(A, W, o[1], o[2], o[3], o[4], stream)
        f.fp8_block_gemm_swiglu_fwd(few, B, o[5], None, stream)

    def same(x, y):
        for p, q in zip(x, y):
            assert torch.equal(p.codes[:, :p.cols], q.codes[:, :p.cols])
            nb = -(-p.cols // 128)
            assert torch.equal(p.scales[:, :nb], q.scales[:, :nb])

    first, second = outs(), outs()
    step(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(second, side)
    torch.cuda.current_stream().wait_stream(side)
    f.fp8_sync_status()
    same(first, second)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(second)
    A.codes.copy_(A.codes.flip(0))
    A.scales.copy_(A.scales.flip(0))
    g.replay()
    step(first)
    f.fp8_sync_status()
    same(first, second)


def test_empty_calls_do_nothing():
    f = _lib()
    e = f.BlockFp8.empty
    f.fp8_block_gemm_swiglu_fwd(e(0, 64), e(256, 64), e(0, 128), e(0, 256))
    f.fp8_block_gemm_swiglu_fwd(e(4, 64), e(0, 64), e(4, 0))
    f.fp8_block_gemm_swiglu_bwd(e(0, 64), e(128, 64), e(0, 256), e(0, 256), e(256, 0), e(128, 0))
    f.fp8_sync_status()


def test_more_than_2_31_elements():
    """Offsets past 32 bits: 98400 tokens of [gate | value] 2 x 11008 wide (2.2 G codes); the last
    block of 128 tokens, partly filled, against the formulas, and the first rows the same bits."""
    f = _lib()
    M, F, K = 98400, 11008, 128
    e = f.BlockFp8.empty
    rows = slice(98304, M)
    first = held(96, K, 1.0, 0, 1, 1)

    def repeated(q, into):
        """The same 96 rows at the beginning, in the last block and, over and over, between."""
        at = torch.arange(M, device="cuda") % 96
        at[rows] = torch.arange(96, device="cuda")
        into.codes.copy_(q.codes[at]), into.scales.copy_(q.scales[at])
        return into

    A, B = repeated(first, e(M, K)), held(2 * F, K, 1.5 * K ** -0.5, 0, 128, 2)
    a8, h8 = e(M, F), e(M, 2 * F)
    f.fp8_block_gemm_swiglu_fwd(A, B, a8, h8)
    f.fp8_sync_status()
    part = lambda q, r: f.BlockFp8(q.codes[r], q.scales[r], q.cols, q.fmt)
    h, a, eh, ta = fwd_plain(first, B)
    near_q(part(h8, rows), h, eh, "h8")
    near_q(part(a8, rows), a, ta, "a8")

    def ends_equal(q):
        nb = q.cols // 128
        return torch.equal(q.codes[:96], q.codes[rows]) and torch.equal(q.scales[:96, :nb], q.scales[rows, :nb])

    assert ends_equal(a8) and ends_equal(h8)
    del a8
    W = held(F, K, K ** -0.5, 0, 128, 4)
    dh8, dh8t, a8t = e(M, 2 * F, 1), e(2 * F, M, 1), e(F, M)
    f.fp8_block_gemm_swiglu_bwd(A, W, h8, dh8, dh8t, a8t)
    f.fp8_sync_status()
    dh, a, tol, tol_a = bwd_plain(first, W, part(h8, rows))
    near_q(part(dh8, rows), dh, tol, "dh8")
    assert ends_equal(dh8)
    tail = lambda q: f.BlockFp8(q.codes[:, rows.start:], q.scales[:, rows.start // 128:], 96, q.fmt)
    near_q(tail(dh8t), dh.t(), tol.t(), "dh8t")
    near_q(tail(a8t), a.t(), tol_a.t(), "a8t")


def test_two_calls_at_once():
    """On two streams, each with data of its own: the same bits as one after the other."""
    f = _lib()
    cases = [(300, 640, 512), (16, 1152, 700), (1100, 1024, 256)]
    data, alone = [], []
    for k, (M, F, K) in enumerate(cases):
        A, B, W = held(M, K, 1.0, 0, 1, k), held(2 * F, K, 0.07, 0, 128, k + 9), held(F, K, 0.05, 0, 128, k + 7)
        data.append((A, B, W))

    def run(k, stream=None):
        (M, F, K), (A, B, W), e = cases[k], data[k], f.BlockFp8.empty
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            o = (e(M, F), e(M, 2 * F), e(M, 2 * F, 1), e(2 * F, M, 1), e(F, M))
        for q in o:
            q.codes.zero_(), q.scales.zero_()
        torch.cuda.synchronize()
        return o, lambda: (f.fp8_block_gemm_swiglu_fwd(A, B, o[0], o[1], stream),
                           f.fp8_block_gemm_swiglu_bwd(A, W, o[1], o[2], o[3], o[4], stream))

    for k in range(3):
        o, go = run(k)
        go()
        alone.append(o)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [run(k, s) for k, s in enumerate(streams)]
    torch.cuda.synchronize()
    for _ in range(5):
        for _, go in outs:
            go()
    f.fp8_sync_status()
    torch.cuda.synchronize()
    for (o, _), want in zip(outs, alone):
        for p, q in zip(o, want):
            nb = -(-p.cols // 128)
            assert torch.equal(p.codes[:, :p.cols], q.codes[:, :p.cols])
            assert torch.equal(p.scales[:, :nb], q.scales[:, :nb])
