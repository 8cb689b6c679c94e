"""GPU tests of the norm of many gradients together and of clipping by it, against
64-bit sums.

Tolerances.  The norm: squares of 32 values are summed in fp32 (at most 2^-20
of the sum: some 14 roundings), everything behind that is exact to more bits, and
the root halves it: 2^-20 with the last rounding; a norm below 2^-126 is held in
steps of 2^-149, half of which, 2^-150, its rounding may be off, and one above
fp32's largest number, 2^128 (1 - 2^-24), by more than half a step rounds to infinity.  Clipping is one division, one
product and one rounding, each correctly rounded: compared bit for bit with the
same three of torch's."""
import pytest
import torch

from test_gpu_block import gen

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def norm_of(tensors):
    return sum(float(t.double().square().sum()) for t in tensors) ** 0.5


def run_norm(tensors, **kw):
    f = _lib()
    norm = torch.full((1,), -5.0, device="cuda")
    f.fp8_grad_norm(tensors, norm, **kw)
    f.fp8_sync_status()
    return norm


def near_norm(norm, want):
    if want > 2.0 ** 128:
        assert norm.item() == float("inf")
        return
    assert abs(norm.double().item() - want) <= 2.0 ** -20 * want + 2.0 ** -150, (norm.item(), want)


def clipped(g, norm, max_norm, dtype):
    n = norm.item()
    c = torch.ones_like(norm) if not (max_norm < n < float("inf")) \
        else torch.tensor([max_norm], device="cuda", dtype=torch.float32) / norm
    return (g.float() * c).to(dtype)


LENGTHS = [0, 1, 2, 3, 7, 8, 9, 31, 511, 4096, 16383, 16384, 16385, 100003]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", LENGTHS)
def test_one_tensor(dtype, n):
    g = torch.randn(n, generator=gen(n), device="cuda").to(dtype)
    norm = run_norm([g])
    if n == 0:
        assert norm.item() == 0
    near_norm(norm, norm_of([g]))
    for out in TYPES:
        o = torch.full((n + 2,), 9.0, dtype=out, device="cuda")
        _lib().fp8_grad_clip([g], norm, 0.5, [o[1:1 + n]])
        torch.cuda.synchronize()
        assert torch.equal(o[1:1 + n], clipped(g, norm, 0.5, out))
        assert o[0] == 9 and o[-1] == 9


def flat_list(seed, shift, dtypes=TYPES, count=40):
    """Views of every alignment into flat buffers, with empty ones among them."""
    g, out = gen(seed), []
    r = torch.Generator().manual_seed(seed)
    for k in range(count):
        n = int(torch.randint(0, 40000, (1,), generator=r)) if k % 5 else k % 3
        d = dtypes[k % len(dtypes)]
        flat = torch.randn(n + 16, generator=g, device="cuda").to(d)
        out.append(flat[(k + shift) % 9:][:n])
    return out


@pytest.mark.parametrize("shift", range(3))
def test_many_tensors_of_all_types_and_alignments(shift):
    f = _lib()
    grads = flat_list(7, shift)
    norm = run_norm(grads)
    near_norm(norm, norm_of(grads))
    assert torch.equal(norm, run_norm(grads))
    big = [torch.full((t.numel() + 16,), 9.0, dtype=TYPES[(k + shift) % 3], device="cuda")
           for k, t in enumerate(grads)]
    outs = [b[(5 * k) % 8:][: t.numel()] for k, (b, t) in enumerate(zip(big, grads))]
    want = [clipped(g, norm, 1.5, o.dtype) for g, o in zip(grads, outs)]
    f.fp8_grad_clip(grads, norm, 1.5, outs)
    torch.cuda.synchronize()
    for k, (o, w, b) in enumerate(zip(outs, want, big)):
        assert torch.equal(o, w), k
        at = (5 * k) % 8
        assert (b[:at] == 9).all() and (b[at + o.numel():] == 9).all()
    # in place
    want = [clipped(g, norm, 1.5, g.dtype) for g in grads]
    f.fp8_grad_clip(grads, norm, 1.5)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(grads, want))


def test_views_that_share_a_flat_buffer():
    """Neighbours in one buffer, in place: a 16-byte block belongs to two tensors."""
    f = _lib()
    for dtype in TYPES:
        flat = torch.randn(60000, generator=gen(3), device="cuda").to(dtype)
        cuts = [0, 1, 4, 17, 18, 1000, 1003, 20001, 40000, 60000]
        grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
        norm = run_norm(grads)
        near_norm(norm, norm_of([flat]))
        want = clipped(flat, norm, 2.0, dtype)
        f.fp8_grad_clip(grads, norm, 2.0)
        torch.cuda.synchronize()
        assert torch.equal(flat, want)


@pytest.mark.parametrize("count", [1, 64, 65, 1000, 1001, 2500])
def test_long_lists(count):
    f = _lib()
    flat = torch.randn(count * 37, generator=gen(count), device="cuda")
    grads = [flat[37 * k: 37 * k + 1 + k % 37] for k in range(count)]
    norm = run_norm(grads)
    near_norm(norm, norm_of(grads))
    outs = [torch.empty_like(g, dtype=torch.bfloat16) for g in grads]
    f.fp8_grad_clip(grads, norm, 1.0, outs)
    torch.cuda.synchronize()
    assert all(torch.equal(o, clipped(g, norm, 1.0, o.dtype)) for g, o in zip(grads, outs))


def test_values_outside_fp32s_squares():
    """Squares that overflow or vanish in fp32, alone and beside ordinary ones."""
    for scale in (1e-30, 1e-44, 1e-20, 1e15, 1e25, 3e37):
        g = (torch.rand(50001, generator=gen(1), device="cuda") * scale).float()
        near_norm(run_norm([g]), norm_of([g]))
        near_norm(run_norm([g, g[:77]]), norm_of([g, g[:77]]))
    mixed = torch.randn(40000, generator=gen(2), device="cuda")
    mixed[::1000] *= 1e20
    mixed[1::3] *= 1e-20
    near_norm(run_norm([mixed]), norm_of([mixed]))
    big = torch.full((40000,), 3e38, device="cuda")
    assert run_norm([big]).item() == float("inf")
    small = torch.full((5,), torch.finfo(torch.float16).tiny / 1024, dtype=torch.float16, device="cuda")
    near_norm(run_norm([small]), norm_of([small]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan"])
def test_a_norm_that_is_not_finite_changes_nothing(dtype, bad):
    f = _lib()
    g = torch.randn(70001, generator=gen(5), device="cuda").to(dtype)
    other = torch.randn(30, generator=gen(6), device="cuda")
    g[41234] = float(bad)
    norm = run_norm([other, g])
    assert norm.isnan().item() if bad == "nan" else norm.item() == float("inf")
    outs = [torch.empty_like(other), torch.empty_like(g)]
    before = g.clone()
    f.fp8_grad_clip([other, g], norm, 1.0, outs)
    f.fp8_grad_clip([other, g], norm, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], other)
    assert torch.equal(outs[1].nan_to_num(7.0), before.nan_to_num(7.0))
    assert torch.equal(g.nan_to_num(7.0), before.nan_to_num(7.0))


def test_limits_of_max_norm():
    """Clipping begins above max_norm, not at it; max_norm 0 and infinity; a list without tensors."""
    f = _lib()
    g = torch.tensor([3.0, 4.0], device="cuda")
    norm = run_norm([g])
    assert norm.item() == 5.0
    for limit, want in [(5.0, [3.0, 4.0]), (10.0, [3.0, 4.0]), (float("inf"), [3.0, 4.0]),
                        (2.5, [1.5, 2.0]), (0.0, [0.0, 0.0])]:
        o = torch.full_like(g, 9.0)
        f.fp8_grad_clip([g], norm, limit, [o])
        torch.cuda.synchronize()
        assert o.tolist() == want, limit
    assert run_norm([]).item() == 0
    f.fp8_grad_clip([], norm, 1.0)
    f.fp8_grad_clip([], norm, 1.0, [])
    f.fp8_sync_status()


def test_refusals():
    f = _lib()
    g, norm = torch.zeros(8, device="cuda"), torch.zeros(1, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        f.fp8_grad_norm([g[::2]], norm)
    with pytest.raises(ValueError, match="float32"):
        f.fp8_grad_norm([g.double()], norm)
    with pytest.raises(ValueError, match="outs"):
        f.fp8_grad_clip([g], norm, 1.0, [])
    with pytest.raises(ValueError, match="twice"):
        f.fp8_grad_clip([g, g], norm, 1.0)
    with pytest.raises(f.Fp8Error, match="elements"):
        f.fp8_grad_clip([g], norm, 1.0, [torch.zeros(7, device="cuda")])
    with pytest.raises(f.Fp8Error, match="max_norm"):
        f.fp8_grad_clip([g], norm, -1.0)
    with pytest.raises(f.Fp8Error, match="bytes"):
        f.fp8_grad_norm([g], norm, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_streams_and_graphs():
    """On a stream of its own; two captured passes that share a workspace, replayed on new data."""
    f = _lib()
    grads = [torch.empty(n, device="cuda", dtype=d) for n, d in [(5000, torch.float32), (70001, torch.bfloat16)]]
    outs = [torch.empty_like(g, dtype=torch.bfloat16) for g in grads]
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(f.fp8_grad_norm_workspace(2), dtype=torch.uint8, device="cuda")

    def fill(seed):
        for g in grads:
            g.copy_(torch.randn(g.numel(), generator=gen(seed), device="cuda"))

    def step(stream=None, workspace=ws):
        f.fp8_grad_norm(grads, norm, workspace, stream)
        f.fp8_grad_clip(grads, norm, 1.0, outs, stream)

    def check():
        torch.cuda.synchronize()
        near_norm(norm, norm_of(grads))
        assert all(torch.equal(o, clipped(g, norm, 1.0, o.dtype)) for g, o in zip(grads, outs))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side, None)
    check()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for k in range(4):
        fill(k)
        graphs[k % 2].replay()
        check()


def test_more_than_2_31_elements():
    f = _lib()
    n = (1 << 31) + 20011
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-50000:] = torch.randn(50000, generator=gen(2), device="cuda").to(torch.bfloat16)
    g[:100] = 1
    norm = run_norm([g])
    near_norm(norm, (norm_of([g[-50000:]]) ** 2 + 100) ** 0.5)
    want = clipped(g[-50000:], norm, 1.0, g.dtype), clipped(g[:100], norm, 1.0, g.dtype)
    f.fp8_grad_clip([g], norm, 1.0)
    f.fp8_sync_status()
    assert torch.equal(g[-50000:], want[0]) and torch.equal(g[:100], want[1])
    assert (g[100:-50000] == 0).all()
