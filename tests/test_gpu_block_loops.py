"""GPU tests of the block-scaled operators at sizes where their persistent loops go round: more
rows or tiles than a grid holds several times over, so that prefetches, alternating buffers,
rings and barriers' phases come to their second and third use.  The checks and tolerances are
those of test_gpu_block.py and test_gpu_saved.py, against 64 bits."""
import pytest
import torch

import block_ref as ref
import test_gpu_block as block
import test_gpu_saved as saved

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
RAGGED = (9 * 128 + 37, 92 * 128 + 5)   # 10 x 93 tiles: over 3 for each of 2 CTAs on 152 SMs
TALL = (950 * 128 + 3, 100)             # 951 x 1


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# (columns, rows per SM): a warp per row takes 16 rows per SM at a time, a CTA per row up to 10,
# and aligned rows go in pairs; one row more makes the last pair half empty
LN_FWD = [(64, 80), (301, 48), (528, 50), (1000, 30), (4096, 10), (4103, 6), (16384, 3), (16392, 9)]


@pytest.mark.parametrize("cols,per_sm", LN_FWD)
@pytest.mark.parametrize("dtype,wtype", [(F32, F32), (BF16, BF16)])
def test_layernorm_fwd(cols, per_sm, dtype, wtype):
    saved.test_layernorm_fwd(per_sm * sms() + 1, cols, dtype, wtype)


# 8 CTAs per SM at up to 1024 columns, 2 at 2049 to 4608, 1 up to 8192: over 18 rows for each CTA,
# where a ring holds 8 at most
LN_BWD = [(136, 80), (505, 48), (1000, 152), (1024, 152), (4096, 38), (4103, 38), (8192, 19), (7001, 19),
          (8200, 9), (16392, 9)]


@pytest.mark.parametrize("cols,per_sm", LN_BWD)
@pytest.mark.parametrize("dtype,wtype,kept", [(BF16, BF16, False), (BF16, F32, True), (F32, F32, True)])
def test_layernorm_bwd(cols, per_sm, dtype, wtype, kept):
    saved.test_layernorm_bwd(per_sm * sms() + 1, cols, dtype, wtype, kept)


@pytest.mark.parametrize("rows,cols", [RAGGED, TALL])
@pytest.mark.parametrize("dtype,fmt", [(F32, 0), (BF16, 1), (F16, 0)])
def test_quantize(rows, cols, dtype, fmt):
    block.test_quantize(rows, cols, dtype, fmt)


@pytest.mark.parametrize("rows,cols", [RAGGED, TALL])
@pytest.mark.parametrize("fmt", [0, 1])
def test_layernorm_recompute(rows, cols, fmt):
    saved.test_layernorm_recompute(rows, cols, fmt)


@pytest.mark.parametrize("M,F", [(RAGGED[0], 47 * 128), (500 * 128 + 3, 128)])
@pytest.mark.parametrize("dtype,fmt", [(F32, 0), (BF16, 1), (F16, 1)])
def test_swiglu_bwd(M, F, dtype, fmt):
    saved.test_swiglu_bwd(M, F, dtype, fmt)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu_fwd(dtype):
    F = 130 * 128   # 32 blocks per CTA and 64 CTAs per SM: more blocks than that
    saved.test_swiglu_fwd(64 * 32 * sms() // 130 + 100, F, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dequantize(dtype):
    f = block._lib()
    rows, cols = 64 * 8 * sms() // 2 + 100, 1030   # two segments of 1024 per row, 512 warps per SM
    q, _ = block.marked(rows, cols, 0, 1)
    q.codes.copy_(torch.randint(0, 256, q.codes.shape, generator=block.gen(3), device="cuda"))
    q.scales.copy_(torch.randint(110, 140, q.scales.shape, generator=block.gen(4), device="cuda"))
    out = torch.full((rows, cols), 9.0, dtype=dtype, device="cuda")
    f.fp8_block_dequantize(q, out)
    want = ref.values(q)[0].float().to(dtype)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(1), want.nan_to_num(1))


@pytest.mark.parametrize("sd", [torch.uint8, torch.float32])
@pytest.mark.parametrize("bb", [1, 128])
def test_gemm(sd, bb):
    """17 x 19 tiles for 76 pairs of CTAs, 11 k-blocks each."""
    f = block._lib()
    M, N, K = 4100, 4700, 1290
    A, B = block.operand(M, K, 1, 1, sd, 1), block.operand(N, K, 0, bb, sd, 2)
    D = torch.full((M + 1, N + 4), 7.0, dtype=BF16, device="cuda")
    f.fp8_block_gemm_tn(A, B, D[:M, :N])
    f.fp8_sync_status()
    block.check_gemm(A, B, D[:M, :N], (M, N, K, sd, bb))
    assert (D[M] == 7).all() and (D[:, N:] == 7).all()
