"""The block-scaled operators' refusals: every bad argument is found on the host,
before any CUDA call, with the documented status and a message naming the call
(CPU only); and the binding's structs and constants are the header's."""
import ctypes
import re

import pytest
import torch

import fp8_mixed_precision_amax_gb300 as f
from fp8_mixed_precision_amax_gb300 import api

OK, ERR_ARG, ERR_ALIGN, ERR_UNSUPPORTED = 0, 1, 2, 5
P = 0x1000   # never read: a refused call, or one on a machine without a GPU, enqueues nothing


def mat(rows, cols, ld=None, dtype=1, data=P):
    return api.fp8_matrix(data, rows, cols, cols if ld is None else ld, dtype)


def blk(rows, cols, ld=None, lds=None, fmt=0, br=1, st=0, codes=P, scales=P):
    return api.fp8_block_tensor(codes, rows, cols, -(-cols // 16) * 16 if ld is None else ld,
                                scales, -(-cols // 512) * 4 if lds is None else lds, fmt, br, st)


def err(name, *args):
    lib = f.library()
    status = getattr(lib, name)(*args, None)
    return status, lib.fp8_last_error().decode()


def refused(status, words, name, *args):
    s, msg = err(name, *args)
    assert s == status, (name, s, msg)
    assert name in msg and words in msg, msg


BAD_MATRIX = [
    (ERR_ARG, "bad type", dict(dtype=3)),
    (ERR_ARG, "bad type", dict(dtype=-1)),
    (ERR_ARG, "row stride", dict(ld=99)),
    (ERR_ARG, "no data", dict(data=None)),
    (ERR_ALIGN, "aligned to its elements", dict(data=0x1001)),
    (ERR_ALIGN, "aligned to its elements", dict(data=0x1002, dtype=0)),
]
BAD_BLOCK = [
    (ERR_ARG, "bad format", dict(fmt=2)),
    (ERR_ARG, "block_rows", dict(br=64)),
    (ERR_ARG, "bad scale type", dict(st=2)),
    (ERR_ARG, "row stride", dict(ld=96)),
    (ERR_ARG, "scales per row", dict(lds=0)),
    (ERR_ARG, "no codes", dict(codes=None)),
    (ERR_ARG, "no codes", dict(scales=None)),
    (ERR_ALIGN, "16-byte aligned", dict(ld=104)),
    (ERR_ALIGN, "16-byte aligned", dict(codes=0x1008)),
    (ERR_ALIGN, "4-byte aligned", dict(scales=0x1002)),
    (ERR_ALIGN, "4-byte aligned", dict(lds=5)),
]


@pytest.mark.parametrize("status,words,bad", BAD_MATRIX)
def test_bad_matrices(status, words, bad):
    q, qt = blk(50, 100), blk(100, 50)
    refused(status, words, "fp8_block_quantize", mat(50, 100, **bad), q, qt)
    refused(status, words, "fp8_block_dequantize", q, mat(50, 100, **bad))
    refused(status, words, "fp8_block_gemm_tn", blk(50, 64), blk(100, 64), mat(50, 100, **bad))
    refused(status, words, "fp8_layernorm_fwd", mat(50, 100, **bad), P, P, 0, 1e-5, None, q, None,
            P, P)
    refused(status, words, "fp8_layernorm_bwd", mat(50, 100, **bad), None, q, P, 0, P, P,
            mat(50, 100), P, P, P, 1 << 30)
    refused(status, words, "fp8_layernorm_bwd", mat(50, 100), None, q, P, 0, P, P,
            mat(50, 100, **bad), P, P, P, 1 << 30)


@pytest.mark.parametrize("status,words,bad", BAD_BLOCK)
def test_bad_block_tensors(status, words, bad):
    b = blk(50, 100, **bad)
    refused(status, words, "fp8_block_quantize", mat(50, 100), b, None)
    refused(status, words, "fp8_block_quantize", mat(100, 50), None, b)
    refused(status, words, "fp8_block_dequantize", b, mat(50, 100))
    refused(status, words, "fp8_block_gemm_tn", b, blk(64, 100), mat(50, 64))
    refused(status, words, "fp8_block_gemm_tn", blk(64, 100), b, mat(64, 50))
    refused(status, words, "fp8_layernorm_fwd", mat(50, 100), P, P, 0, 1e-5, None, b, None, P, P)
    refused(status, words, "fp8_layernorm_bwd", mat(50, 100), None, b, P, 0, P, P, mat(50, 100), P,
            P, P, 1 << 30)
    refused(status, words, "fp8_layernorm_recompute", b, P, P, 0, P, P, blk(100, 50))
    refused(status, words, "fp8_layernorm_recompute", blk(100, 50), P, P, 0, P, P, b)


def test_shapes_and_combinations():
    refused(ERR_ARG, "both NULL", "fp8_block_quantize", mat(4, 4), None, None)
    refused(ERR_ARG, "x is NULL", "fp8_block_quantize", None, blk(4, 4), None)
    refused(ERR_ARG, "expected 4 x 5", "fp8_block_quantize", mat(4, 5), blk(5, 4), None)
    refused(ERR_ARG, "expected 5 x 4", "fp8_block_quantize", mat(4, 5), None, blk(4, 5))
    for other in (dict(fmt=1), dict(br=128), dict(st=1)):
        refused(ERR_ARG, "differ", "fp8_block_quantize", mat(4, 5), blk(4, 5), blk(5, 4, **other))
    refused(ERR_ARG, "bad size", "fp8_block_quantize", mat(-1, 5), blk(4, 5), None)
    refused(ERR_ARG, "bad size", "fp8_block_quantize", mat(4, 1 << 31), blk(4, 5), None)
    refused(ERR_ARG, "tiles", "fp8_block_quantize", mat(1 << 30, 1 << 30),
            blk(1 << 30, 1 << 30), None)

    refused(ERR_ARG, "columns", "fp8_block_gemm_tn", blk(4, 64), blk(4, 65), mat(4, 4))
    refused(ERR_ARG, "different types", "fp8_block_gemm_tn", blk(4, 64), blk(4, 64, st=1),
            mat(4, 4))
    refused(ERR_ARG, "expected 4 x 6", "fp8_block_gemm_tn", blk(4, 64), blk(6, 64), mat(6, 4))
    refused(ERR_ARG, "BF16", "fp8_block_gemm_tn", blk(4, 64), blk(6, 64), mat(4, 6, dtype=0))

    fwd = lambda **k: (k.get("x", mat(4, 5)), k.get("gamma", P), k.get("beta", P), k.get("wt", 0),
                       k.get("eps", 1e-5), k.get("y"), k.get("y8"), k.get("x8"),
                       k.get("mean", P), k.get("rstd", P))
    for words, k in [("no columns", dict(x=mat(4, 0))), ("eps", dict(eps=-1.0)),
                     ("eps", dict(eps=float("nan"))), ("bad type", dict(wt=9)),
                     ("gamma", dict(gamma=None)), ("beta", dict(beta=None)),
                     ("mean", dict(mean=None)), ("rstd", dict(rstd=None)),
                     ("expected 4 x 5", dict(y=mat(5, 4))), ("x's type", dict(y=mat(4, 5, dtype=0))),
                     ("expected 4 x 5", dict(y8=blk(4, 6))),
                     ("block_rows must be 1", dict(x8=blk(4, 5, br=128)))]:
        refused(ERR_ARG, words, "fp8_layernorm_fwd", *fwd(**k))
    refused(ERR_ALIGN, "gamma", "fp8_layernorm_fwd", *fwd(gamma=0x1002))

    bwd = lambda **k: (k.get("dy", mat(4, 5)), k.get("x", mat(4, 5)), k.get("x8"),
                       k.get("gamma", P), k.get("wt", 0), k.get("mean", P), k.get("rstd", P),
                       k.get("dx", mat(4, 5)), k.get("dg", P), k.get("db", P), k.get("ws", P),
                       k.get("n", 1 << 20))
    need = f.fp8_layernorm_bwd_workspace(4, 5)
    assert need > 0 and f.fp8_layernorm_bwd_workspace(0, 5) == 0
    for words, k in [("exactly one", dict(x8=blk(4, 5))), ("exactly one", dict(x=None)),
                     ("no columns", dict(dy=mat(4, 0))), ("expected 4 x 5", dict(x=mat(4, 6))),
                     ("dy's type", dict(x=mat(4, 5, dtype=0))),
                     ("dy's type", dict(dx=mat(4, 5, dtype=0))),
                     ("expected 4 x 5", dict(dx=mat(3, 5))), ("dgamma", dict(dg=None)),
                     ("dbeta", dict(db=None)), ("workspace", dict(ws=None)),
                     ("bytes", dict(n=need - 1))]:
        refused(ERR_ARG, words, "fp8_layernorm_bwd", *bwd(**k))
    refused(ERR_ALIGN, "workspace", "fp8_layernorm_bwd", *bwd(ws=0x1008))

    refused(ERR_ARG, "expected 5 x 4", "fp8_layernorm_recompute", blk(4, 5), P, P, 0, P, P,
            blk(4, 5))
    refused(ERR_ALIGN, "multiple of 128", "fp8_swiglu_fwd", mat(4, 384), blk(4, 192), None)
    refused(ERR_ARG, "expected 4 x 128", "fp8_swiglu_fwd", mat(4, 256), blk(4, 256), None)
    refused(ERR_ARG, "expected 4 x 256", "fp8_swiglu_fwd", mat(4, 256), blk(4, 128), blk(4, 128))
    refused(ERR_ALIGN, "multiple of 128", "fp8_swiglu_bwd", mat(4, 64), blk(4, 128), blk(4, 128),
            None, None)
    refused(ERR_ARG, "all NULL", "fp8_swiglu_bwd", mat(4, 128), blk(4, 256), None, None, None)
    refused(ERR_ARG, "expected 256 x 4", "fp8_swiglu_bwd", mat(4, 128), blk(4, 256), None,
            blk(4, 256), None)
    refused(ERR_ARG, "expected 128 x 4", "fp8_swiglu_bwd", mat(4, 128), blk(4, 256), None, None,
            blk(256, 4))
    refused(ERR_ARG, "differ in format", "fp8_swiglu_bwd", mat(4, 128), blk(4, 256), blk(4, 256),
            blk(256, 4, fmt=1), None)


def test_binding_refuses_what_it_cannot_pass():
    x = torch.zeros(16, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_block_quantize(x, None, None)
    q = f.BlockFp8.empty(16, 32, device="cpu")
    assert q.shape == (16, 32) and q.nbytes == 16 * 32 + 16 * 4
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_block_dequantize(q, x)
    t = f.BlockFp8.empty(130, 700, f.E5M2, 128, torch.float32, device="cpu")
    assert t.codes.shape == (130, 704) and t.scales.shape == (2, 8)


def test_structs_and_constants_match_the_header():
    src = open(api.HEADER_PATH).read()
    for name in ("fp8_matrix", "fp8_block_tensor"):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, src).group(1)
        fields = [w for line in re.findall(r"([^;]*);", body)
                  for w in re.findall(r"(\w+)\s*(?:,|$)", line)]
        assert fields == [n for n, _ in getattr(api, name)._fields_]
    enum = dict((k, int(v)) for k, v in re.findall(r"\b(FP8_[A-Z0-9_]+)\s*=\s*(\d+)", src))
    assert [enum["FP8_DTYPE_F32"], enum["FP8_DTYPE_BF16"], enum["FP8_DTYPE_F16"]] == \
        [api._DTYPES[t] for t in (torch.float32, torch.bfloat16, torch.float16)]
    assert (enum["FP8_SCALE_E8M0"], enum["FP8_SCALE_F32"]) == (api.SCALE_E8M0, api.SCALE_F32)
