"""Refusals of the gated product's calls: every bad argument is found on the host, before any
CUDA call, with the documented status and a message naming the call (CPU only)."""
import pytest

import fp8_mixed_precision_amax_gb300 as f
from test_block_abi import BAD_BLOCK, ERR_ALIGN, ERR_ARG, blk, refused

FWD, BWD = "fp8_block_gemm_swiglu_fwd", "fp8_block_gemm_swiglu_bwd"


@pytest.mark.parametrize("status,words,bad", BAD_BLOCK)
def test_bad_block_tensors(status, words, bad):
    b = blk(50, 100, **bad)
    refused(status, words, FWD, b, blk(256, 100), blk(50, 128), None)
    refused(status, words, FWD, blk(50, 100), blk(256, 100, **bad), blk(50, 128), None)
    refused(status, words, FWD, blk(50, 64), blk(256, 64), b, None)
    refused(status, words, FWD, blk(50, 64), blk(256, 64), blk(50, 128), b)
    args = [blk(50, 100), blk(128, 100), blk(50, 256), blk(50, 256), blk(256, 50), blk(128, 50)]
    for i in range(6):
        refused(status, words, BWD, *args[:i], blk(128, 100, **bad) if i == 1 else b, *args[i + 1:])


def test_shapes_and_combinations():
    ok = dict(A=blk(4, 64), B=blk(256, 64), a8=blk(4, 128), h8=blk(4, 256))
    for status, words, k in [(ERR_ARG, "A is NULL", dict(A=None)), (ERR_ARG, "B is NULL", dict(B=None)),
                             (ERR_ARG, "a8 is NULL", dict(a8=None)),
                             (ERR_ARG, "A has 64 columns, B 65", dict(B=blk(256, 65))),
                             (ERR_ARG, "no columns", dict(A=blk(4, 0), B=blk(256, 0))),
                             (ERR_ARG, "E8M0", dict(A=blk(4, 64, st=1))), (ERR_ARG, "E8M0", dict(B=blk(256, 64, st=1))),
                             (ERR_ALIGN, "multiple of 128", dict(B=blk(128, 64), a8=blk(4, 64))),
                             (ERR_ALIGN, "multiple of 128", dict(B=blk(300, 64))),
                             (ERR_ARG, "expected 4 x 128", dict(a8=blk(4, 256))),
                             (ERR_ARG, "expected 4 x 256", dict(h8=blk(4, 128))),
                             (ERR_ARG, "block_rows must be 1", dict(a8=blk(4, 128, br=128))),
                             (ERR_ARG, "block_rows must be 1", dict(h8=blk(4, 256, br=128)))]:
        refused(status, words, FWD, *{**ok, **k}.values())
    ok = dict(A=blk(4, 64), B=blk(128, 64), h8=blk(4, 256), dh8=blk(4, 256), dh8t=blk(256, 4), a8t=blk(128, 4))
    for status, words, k in [(ERR_ARG, "A is NULL", dict(A=None)), (ERR_ARG, "B is NULL", dict(B=None)),
                             (ERR_ARG, "h8 is NULL", dict(h8=None)),
                             (ERR_ARG, "all NULL", dict(dh8=None, dh8t=None, a8t=None)),
                             (ERR_ARG, "A has 64 columns, B 65", dict(B=blk(128, 65))),
                             (ERR_ARG, "no columns", dict(A=blk(4, 0), B=blk(128, 0))),
                             (ERR_ARG, "E8M0", dict(A=blk(4, 64, st=1))), (ERR_ARG, "E8M0", dict(B=blk(128, 64, st=1))),
                             (ERR_ALIGN, "multiple of 128", dict(B=blk(64, 64))),
                             (ERR_ARG, "expected 4 x 256", dict(h8=blk(4, 128))),
                             (ERR_ARG, "expected 4 x 256", dict(dh8=blk(256, 4))),
                             (ERR_ARG, "expected 256 x 4", dict(dh8t=blk(4, 256))),
                             (ERR_ARG, "expected 128 x 4", dict(a8t=blk(256, 4))),
                             (ERR_ARG, "block_rows must be 1", dict(h8=blk(4, 256, br=128))),
                             (ERR_ARG, "differ in format", dict(dh8t=blk(256, 4, fmt=1)))]:
        refused(status, words, BWD, *{**ok, **k}.values())
    refused(ERR_ARG, "tiles", FWD, blk(1 << 30, 64), blk(1 << 30, 64), blk(1 << 30, 1 << 29), None)


def test_binding_refuses_what_it_cannot_pass():
    q = f.BlockFp8.empty(16, 32, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_block_gemm_swiglu_fwd(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_block_gemm_swiglu_bwd(q, q, q, q)
