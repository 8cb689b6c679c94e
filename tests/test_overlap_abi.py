"""Refusals of calls whose outputs share memory with each other, or with an input in any other
way than in its very place: found on the host, before any CUDA call (CPU only).  Calls that
share nothing are tested where a GPU runs them."""
import pytest

import fp8_mixed_precision_amax_gb300 as f
from test_block_abi import ERR_ARG, refused
from test_host_setup import run_check
from fp8_mixed_precision_amax_gb300 import api

BASE = 1 << 32


def test_areas_against_a_table_of_bytes(tmp_path):
    run_check("overlap_check", tmp_path)


class Memory:
    """Places far apart from each other, for arguments that share nothing."""

    def __init__(self):
        self.next = BASE

    def place(self):
        self.next += 1 << 24
        return self.next

    def mat(self, rows, cols, ld=None, at=None, dtype=1):
        return api.fp8_matrix(self.place() if at is None else at, rows, cols, ld or cols, dtype)

    def blk(self, rows, cols, codes=None, scales=None, br=1):
        return api.fp8_block_tensor(codes or self.place(), rows, cols, -(-cols // 16) * 16,
                                    scales or self.place(), -(-cols // 512) * 4, 0, br, 0)


def rms_fwd(m, rows=50, cols=100, **k):
    a = dict(x=m.mat(rows, cols), residual=m.mat(rows, cols), gamma=m.place(), wtype=0, eps=1e-5, sum=m.mat(rows, cols),
             y=m.mat(rows, cols), y8=m.blk(rows, cols), x8=m.blk(rows, cols), rstd=m.place())
    a.update(k)
    return list(a.values())


def rms_bwd(m, rows=50, cols=100, **k):
    a = dict(dy=m.mat(rows, cols), x=m.mat(rows, cols), x8=None, gamma=m.place(), wtype=0, rstd=m.place(),
             dsum=m.mat(rows, cols), dx=m.mat(rows, cols), dgamma=m.place(), workspace=m.place(),
             room=f.fp8_rmsnorm_bwd_workspace(rows, cols))
    a.update(k)
    return list(a.values())


def test_rmsnorm_forward():
    m = Memory()
    at, other = m.place(), m.place()
    for words, k in [
            ("sum and x overlap", dict(x=m.mat(50, 100, at=at), sum=m.mat(50, 100, at=at + 2))),
            ("sum and x overlap", dict(x=m.mat(50, 100, at=at), sum=m.mat(50, 100, ld=104, at=at))),
            ("sum and residual overlap", dict(residual=m.mat(50, 100, 120, at=at), sum=m.mat(50, 100, 120, at=at - 198))),
            ("sum and residual overlap", dict(residual=m.mat(50, 100, 120, at=at), sum=m.mat(50, 100, 120, at=at + 42))),
            ("y and x overlap", dict(x=m.mat(50, 100, at=at), y=m.mat(50, 100, at=at + 9998))),
            ("sum and y overlap", dict(sum=m.mat(50, 100, at=at), y=m.mat(50, 100, at=at))),
            ("y8's codes and x8's codes overlap", dict(y8=m.blk(50, 100, codes=at), x8=m.blk(50, 100, codes=at))),
            ("y8's scales and x8's scales overlap", dict(y8=m.blk(50, 100, scales=at), x8=m.blk(50, 100, scales=at))),
            ("y8's codes and y8's scales overlap", dict(y8=m.blk(50, 100, codes=at, scales=at + 16))),
            ("x8's codes and x overlap", dict(x=m.mat(50, 100, at=at), x8=m.blk(50, 100, codes=at))),
            ("rstd and gamma overlap", dict(gamma=at, rstd=at + 4 * 99)),
            ("x8's scales and rstd overlap", dict(x8=m.blk(50, 100, scales=at), rstd=at + 4 * 49))]:
        refused(ERR_ARG, words, "fp8_rmsnorm_fwd", *rms_fwd(m, **k))
    # one row's stride says nothing, and a shifted row is no place of its own
    refused(ERR_ARG, "sum and x overlap", "fp8_rmsnorm_fwd",
            *rms_fwd(m, 1, 8, x=m.mat(1, 8, 50, at=other), sum=m.mat(1, 8, 8, at=other + 4)))


def test_rmsnorm_backward_and_recompute():
    m = Memory()
    at = m.place()
    need = f.fp8_rmsnorm_bwd_workspace(50, 100)
    for words, k in [
            ("dx and dy overlap", dict(dy=m.mat(50, 100, at=at), dx=m.mat(50, 100, at=at + 200))),
            ("dx and dsum overlap", dict(dsum=m.mat(50, 100, 128, at=at), dx=m.mat(50, 100, 136, at=at))),
            ("dx and x overlap", dict(x=m.mat(50, 100, at=at), dx=m.mat(50, 100, at=at + 2))),
            ("dx and x8's codes overlap", dict(x=None, x8=m.blk(50, 100, codes=at), dx=m.mat(50, 100, at=at))),
            ("dgamma and gamma overlap", dict(gamma=at, dgamma=at)),
            ("dgamma and workspace overlap", dict(dgamma=at + need - 4, workspace=at)),
            ("dx and workspace overlap", dict(dx=m.mat(50, 100, at=at), workspace=at + 9984)),
            ("workspace and rstd overlap", dict(rstd=at + 16, workspace=at))]:
        refused(ERR_ARG, words, "fp8_rmsnorm_bwd", *rms_bwd(m, **k))
    for words, x8, yt in [("yt's codes and x8's codes", m.blk(64, 64, codes=at), m.blk(64, 64, codes=at)),
                          ("yt's scales and x8's scales", m.blk(64, 64, scales=at), m.blk(64, 64, scales=at)),
                          ("yt's codes and yt's scales", m.blk(64, 64), m.blk(64, 64, codes=at, scales=at + 4092))]:
        refused(ERR_ARG, words, "fp8_rmsnorm_recompute", x8, m.place(), 0, m.place(), yt)


def gated(m, backward, **k):
    a = dict(A=m.blk(60, 200), B=m.blk(128 if backward else 256, 200, br=128))
    a |= dict(h8=m.blk(60, 256), dh8=m.blk(60, 256), dh8t=m.blk(256, 60), a8t=m.blk(128, 60)) if backward else \
        dict(a8=m.blk(60, 128), h8=m.blk(60, 256))
    a.update(k)
    return list(a.values())


def test_gated_product():
    m = Memory()
    at = m.place()
    for words, k in [
            ("a8's codes and h8's codes overlap", dict(a8=m.blk(60, 128, at), h8=m.blk(60, 256, at + 128))),
            ("a8's codes and a8's scales overlap", dict(a8=m.blk(60, 128, at, at + 16))),
            ("a8's scales and h8's scales overlap", dict(a8=m.blk(60, 128, scales=at), h8=m.blk(60, 256, scales=at))),
            ("a8's codes and A's codes overlap", dict(A=m.blk(60, 128, at), B=m.blk(256, 128), a8=m.blk(60, 128, at))),
            ("h8's codes and A's scales overlap", dict(A=m.blk(60, 200, scales=at + 64), h8=m.blk(60, 256, at))),
            ("h8's codes and B's codes overlap", dict(B=m.blk(256, 200, at, br=128), h8=m.blk(60, 256, at + 256 * 208 - 16)))]:
        refused(ERR_ARG, words, "fp8_block_gemm_swiglu_fwd", *gated(m, False, **k))
    for words, k in [
            ("dh8's codes and dh8t's codes overlap", dict(dh8=m.blk(60, 256, at), dh8t=m.blk(256, 60, at))),
            ("dh8t's scales and a8t's scales overlap", dict(dh8t=m.blk(256, 60, scales=at), a8t=m.blk(128, 60, scales=at))),
            ("dh8's codes and h8's codes overlap", dict(h8=m.blk(60, 256, at), dh8=m.blk(60, 256, at + 256))),
            ("dh8's scales and h8's scales overlap", dict(h8=m.blk(60, 256, scales=at), dh8=m.blk(60, 256, scales=at + 4))),
            ("a8t's codes and A's codes overlap", dict(A=m.blk(60, 200, at), a8t=m.blk(128, 60, at))),
            ("dh8t's codes and B's codes overlap", dict(B=m.blk(128, 200, at, br=128), dh8t=m.blk(256, 60, at))),
            ("a8t's codes and h8's codes overlap", dict(h8=m.blk(60, 256, at), a8t=m.blk(128, 60, at)))]:
        refused(ERR_ARG, words, "fp8_block_gemm_swiglu_bwd", *gated(m, True, **k))


def test_norm_and_clipping():
    m = Memory()
    at, elsewhere = m.place(), m.place()
    v = lambda *places: (api.fp8_vector * len(places))(*[api.fp8_vector(p, 8, 0) for p in places])
    for norm in (elsewhere, elsewhere + 28):   # its first and its last element
        refused(ERR_ARG, "outs[1] and norm overlap", "fp8_grad_clip", v(at, elsewhere), None, 2, norm, 1.0)
        refused(ERR_ARG, "outs[1] and norm overlap", "fp8_grad_clip", v(at, at + 32), v(at, elsewhere), 2, norm, 1.0)
    room = f.fp8_grad_norm_workspace(2)
    for ws in (elsewhere - room + 8, elsewhere + 24):
        refused(ERR_ARG, "grads[1] and workspace overlap", "fp8_grad_norm", v(at, elsewhere), 2, m.place(), ws, room)
    refused(ERR_ARG, "norm and workspace overlap", "fp8_grad_norm", v(at), 1, elsewhere + 8, elsewhere, room)
