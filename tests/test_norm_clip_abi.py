"""Refusals of the RMS norm's calls and of those on lists of gradients: every bad argument is
found on the host, before any CUDA call, with the documented status and a message naming
the call (CPU only)."""
import re

import pytest
import torch

import fp8_mixed_precision_amax_gb300 as f
from fp8_mixed_precision_amax_gb300 import api
from test_block_abi import BAD_BLOCK, BAD_MATRIX, ERR_ALIGN, ERR_ARG, P, blk, mat, refused


def fwd(**k):
    return (k.get("x", mat(4, 5)), k.get("res"), k.get("gamma", P), k.get("wt", 0), k.get("eps", 1e-5),
            k.get("sum"), k.get("y"), k.get("y8"), k.get("x8"), k.get("rstd", P))


def bwd(**k):
    return (k.get("dy", mat(4, 5)), k.get("x", mat(4, 5)), k.get("x8"), k.get("gamma", P),
            k.get("wt", 0), k.get("rstd", P), k.get("ds"), k.get("dx", mat(4, 5)), k.get("dg", P),
            k.get("ws", P), k.get("n", 1 << 20))


@pytest.mark.parametrize("status,words,bad", BAD_MATRIX)
def test_bad_matrices(status, words, bad):
    m, ok = mat(50, 100, **bad), mat(50, 100)
    for k in (dict(x=m), dict(x=ok, res=m), dict(x=ok, res=ok, sum=m), dict(x=ok, y=m)):
        refused(status, words, "fp8_rmsnorm_fwd", *fwd(**k))
    for k in (dict(dy=m), dict(x=m), dict(ds=m), dict(dx=m)):
        refused(status, words, "fp8_rmsnorm_bwd", *bwd(**{"dy": ok, "x": ok, "dx": ok, **k}))


@pytest.mark.parametrize("status,words,bad", BAD_BLOCK)
def test_bad_block_tensors(status, words, bad):
    b, ok = blk(50, 100, **bad), mat(50, 100)
    refused(status, words, "fp8_rmsnorm_fwd", *fwd(x=ok, y8=b))
    refused(status, words, "fp8_rmsnorm_fwd", *fwd(x=ok, x8=b))
    refused(status, words, "fp8_rmsnorm_bwd", *bwd(dy=ok, x=None, x8=b, dx=ok))
    refused(status, words, "fp8_rmsnorm_recompute", b, P, 0, P, blk(100, 50))
    refused(status, words, "fp8_rmsnorm_recompute", blk(100, 50), P, 0, P, b)


def test_shapes_and_combinations():
    for words, k in [("no columns", dict(x=mat(4, 0))), ("eps", dict(eps=-1.0)),
                     ("eps", dict(eps=float("nan"))), ("bad type", dict(wt=9)),
                     ("gamma", dict(gamma=None)), ("rstd", dict(rstd=None)),
                     ("x is NULL", dict(x=None)), ("without a residual", dict(sum=mat(4, 5))),
                     ("expected 4 x 5", dict(res=mat(5, 4))),
                     ("x's type", dict(res=mat(4, 5, dtype=0))),
                     ("expected 4 x 5", dict(res=mat(4, 5), sum=mat(4, 6))),
                     ("x's type", dict(res=mat(4, 5), sum=mat(4, 5, dtype=2))),
                     ("expected 4 x 5", dict(y=mat(5, 4))), ("x's type", dict(y=mat(4, 5, dtype=0))),
                     ("expected 4 x 5", dict(y8=blk(4, 6))),
                     ("block_rows must be 1", dict(x8=blk(4, 5, br=128)))]:
        refused(ERR_ARG, words, "fp8_rmsnorm_fwd", *fwd(**k))
    refused(ERR_ALIGN, "gamma", "fp8_rmsnorm_fwd", *fwd(gamma=0x1002))
    refused(ERR_ALIGN, "rstd", "fp8_rmsnorm_fwd", *fwd(rstd=0x1002))
    need = f.fp8_rmsnorm_bwd_workspace(4, 5)
    assert need > 0 and f.fp8_rmsnorm_bwd_workspace(0, 5) == 0
    for words, k in [("exactly one", dict(x8=blk(4, 5))), ("exactly one", dict(x=None)),
                     ("no columns", dict(dy=mat(4, 0))), ("expected 4 x 5", dict(x=mat(4, 6))),
                     ("dy's type", dict(x=mat(4, 5, dtype=0))), ("dy's type", dict(ds=mat(4, 5, dtype=0))),
                     ("dy's type", dict(dx=mat(4, 5, dtype=0))), ("expected 4 x 5", dict(ds=mat(4, 4))),
                     ("expected 4 x 5", dict(dx=mat(3, 5))), ("dgamma", dict(dg=None)),
                     ("dx is NULL", dict(dx=None)), ("rstd", dict(rstd=None)),
                     ("workspace", dict(ws=None)), ("bytes", dict(n=need - 1))]:
        refused(ERR_ARG, words, "fp8_rmsnorm_bwd", *bwd(**k))
    refused(ERR_ALIGN, "workspace", "fp8_rmsnorm_bwd", *bwd(ws=0x1008))
    refused(ERR_ARG, "expected 5 x 4", "fp8_rmsnorm_recompute", blk(4, 5), P, 0, P, blk(4, 5))
    refused(ERR_ARG, "rstd", "fp8_rmsnorm_recompute", blk(4, 5), P, 0, None, blk(5, 4))


def vec(n=8, data=P, dtype=0):
    return api.fp8_vector(data, n, dtype)


def test_lists_of_gradients():
    def norm(*v, count=None, out=P, ws=P, room=1 << 20):
        return (api.fp8_vector * len(v))(*v) if v else None, len(v) if count is None else count, out, ws, room

    def clip(v, o=None, out=P, limit=1.0):
        a = lambda x: None if x is None else (api.fp8_vector * len(x))(*x)
        return a(v), a(o), len(v), out, limit

    assert f.fp8_grad_norm_workspace(0) == f.fp8_grad_norm_workspace(1000) > 0
    assert f.fp8_grad_norm_workspace(1001) == 2 * f.fp8_grad_norm_workspace(1)
    for status, words, bad in [(ERR_ARG, "bad type", vec(dtype=3)), (ERR_ARG, "bad length", vec(n=-1)),
                               (ERR_ARG, "bad length", vec(n=1 << 41)), (ERR_ARG, "no data", vec(data=None)),
                               (ERR_ALIGN, "aligned", vec(data=0x1002)),
                               (ERR_ALIGN, "aligned", vec(data=0x1001, dtype=1))]:
        refused(status, words, "fp8_grad_norm", *norm(vec(), bad))
        refused(status, words, "fp8_grad_clip", *clip([vec(), bad]))
        refused(status, words, "fp8_grad_clip", *clip([vec(), vec()], [vec(), bad]))
    refused(ERR_ARG, "count", "fp8_grad_norm", *norm(vec(), count=-1))
    refused(ERR_ARG, "grads is NULL", "fp8_grad_norm", *norm(count=2))
    refused(ERR_ARG, "norm is NULL", "fp8_grad_norm", *norm(vec(), out=None))
    refused(ERR_ALIGN, "norm", "fp8_grad_norm", *norm(vec(), out=0x1002))
    refused(ERR_ARG, "workspace is NULL", "fp8_grad_norm", *norm(vec(), ws=None))
    refused(ERR_ALIGN, "workspace", "fp8_grad_norm", *norm(vec(), ws=0x1004))
    refused(ERR_ARG, "are needed", "fp8_grad_norm",
            *norm(vec(), room=f.fp8_grad_norm_workspace(1) - 1))
    refused(ERR_ARG, "outs[1] has 9", "fp8_grad_clip", *clip([vec(), vec()], [vec(), vec(n=9)]))
    refused(ERR_ARG, "norm is NULL", "fp8_grad_clip", *clip([vec()], out=None))
    for limit in (-1.0, float("nan")):
        refused(ERR_ARG, "max_norm", "fp8_grad_clip", *clip([vec()], limit=limit))


def test_binding_refuses_what_it_cannot_pass():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_rmsnorm_fwd(x, x[0], 1e-5, x[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_rmsnorm_bwd(x, x, x[0], x[:, 0], x, x[0])
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_grad_norm([x], torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_grad_clip([x], torch.zeros(1), 1.0)


def test_vector_struct_matches_the_header():
    src = open(api.HEADER_PATH).read()
    body = re.search(r"typedef struct \{([^}]*)\} fp8_vector;", src).group(1)
    assert re.findall(r"(\w+);", body) == [n for n, _ in api.fp8_vector._fields_]


def test_what_is_written_overlaps_nothing():
    def clip(grads, outs=None):
        a = lambda x: None if x is None else (api.fp8_vector * len(x))(*x)
        return a(grads), a(outs), len(grads), P, 1.0

    at = lambda place, n=8, dtype=0: vec(n, P + place, dtype)
    refused(ERR_ARG, "outs[0] and outs[1] overlap", "fp8_grad_clip", *clip([at(0), at(0)]))
    refused(ERR_ARG, "outs[1] and outs[0] overlap", "fp8_grad_clip", *clip([at(64), at(36)]))
    refused(ERR_ARG, "outs[0] and outs[2] overlap", "fp8_grad_clip",
            *clip([at(0), at(64), at(128)], [at(256), at(512), at(284)]))
    # of another type, of another start, and another one's
    refused(ERR_ARG, "outs[0] and grads[0] overlap", "fp8_grad_clip", *clip([at(0)], [at(0, dtype=1)]))
    refused(ERR_ARG, "outs[0] and grads[0] overlap", "fp8_grad_clip", *clip([at(0)], [at(28)]))
    refused(ERR_ARG, "outs[1] and grads[0] overlap", "fp8_grad_clip",
            *clip([at(0), at(64)], [at(128), at(0)]))
    # a long list, where one of 300 covers many
    apart = [at(64 * i) for i in range(300)]
    refused(ERR_ARG, "outs[7] and outs[8] overlap", "fp8_grad_clip",
            *clip(apart[:7] + [at(64 * 7, 2000)] + apart[8:]))
    outs = [at(64 * i + 32) for i in range(300)]
    refused(ERR_ARG, "outs[7] and grads[8] overlap", "fp8_grad_clip",
            *clip(apart, outs[:7] + [at(64 * 7 + 40)] + outs[8:]))


def test_long_lists_have_a_limit():
    many = (api.fp8_vector * 17)(*[vec(1 << 40)] * 17)
    refused(ERR_ARG, "too many elements", "fp8_grad_norm", many, 17, P, P, 1 << 20)
