"""GPU tests of memory that the block-scaled calls allocate for work on another stream than the
current one: it must not be memory that the current stream's pending work still writes."""
import pytest
import torch

from test_gpu_block import gen

pytestmark = pytest.mark.gpu

MB = 1 << 20


def pending_writes(nbytes, count):
    """Freed blocks of the current stream, which it will overwrite some 0.2 s from now."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(count)]
    torch.cuda._sleep(400_000_000)
    for b in blocks:
        b.fill_(9)


@pytest.mark.parametrize("raw", [False, True])
def test_dequantize_on_another_stream(raw):
    import fp8_mixed_precision_amax_gb300 as f
    x = torch.randn(1024, 1024, generator=gen(1), device="cuda")
    q = f.BlockFp8.empty(1024, 1024)
    f.fp8_block_quantize(x, q)
    want = q.dequantize()
    side = torch.cuda.Stream()
    q.dequantize(stream=side)       # the library is set up
    pending_writes(2 * MB, 4)
    out = q.dequantize(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_mlp_made_on_another_stream():
    import fp8_mixed_precision_amax_gb300 as f
    K = F = 1024
    n = lambda *s: torch.randn(*s, generator=gen(2), device="cuda").bfloat16()
    args = (n(K), n(K), n(2 * F, K), n(K, F), 16)
    want = f.Fp8BlockMlp(*args)
    side = torch.cuda.Stream()
    f.Fp8BlockMlp(*args, stream=side)
    pending_writes(2 * MB, 8)
    pending_writes(MB, 8)
    mlp = f.Fp8BlockMlp(*args, stream=side)
    torch.cuda.synchronize()
    for name in ("W1q", "W1t", "W2q", "W2t"):
        assert torch.equal(getattr(mlp, name).codes, getattr(want, name).codes), name
        assert torch.equal(getattr(mlp, name).scales[:, :8], getattr(want, name).scales[:, :8]), name


@pytest.mark.parametrize("private", [True, False])
def test_calls_go_to_the_current_stream(monkeypatch, private):
    from fp8_mixed_precision_amax_gb300 import api
    if not private:
        monkeypatch.setattr(api, "_raw_stream", None)
    handle = lambda s: getattr(s, "value", s) or 0
    assert handle(api._stream(None)) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert handle(api._stream(None)) == side.cuda_stream
    assert handle(api._stream(side)) == handle(api._stream(side.cuda_stream)) == side.cuda_stream
