"""The pre-norm gated MLP layer step by step: each tensor of a pass, kept, shared or returned,
against 64 bits from the operands that the step before it left.

Tolerances are the operators' own (test_gpu_rmsnorm, test_gpu_rmsnorm_rows, test_gpu_gated):
a product is known to (128 + K / 128) 2^-23 of the sum of its terms' magnitudes and half a step of
BF16, 2^-8; quantized inputs bit for bit."""
import pytest
import torch

import block_ref as ref
from test_gpu_block import assert_block
from test_gpu_gated import bwd_plain as product_bwd
from test_gpu_gated import fwd_plain as product_fwd
from test_gpu_gated import near_q, product
from test_gpu_gated_mlp import inputs, lib, weights
from test_gpu_rmsnorm import plain
from test_gpu_rmsnorm_rows import check
from test_gpu_saved import h, near, near_block

pytestmark = pytest.mark.gpu


def near_product(got, A, B, what):
    want, tol = product(A, B)
    near(got, want, tol + h(got.dtype) * (want.abs() + tol), what)


@pytest.mark.parametrize("M,K,F", [(1, 128, 128), (100, 200, 384), (777, 1000, 896), (1300, 512, 1024)])
@pytest.mark.parametrize("grad_fmt", [0, 1])
@pytest.mark.parametrize("with_residual", [True, False])
def test_each_step(M, K, F, grad_fmt, with_residual):
    f = lib()
    gamma, W1, W2 = weights(K, F, M)
    x, residual, dy, ds = inputs(M, K, K)
    residual, ds = (residual, ds) if with_residual else (None, None)
    mlp = f.Fp8GatedMlp(gamma, W1, W2, M, grad_fmt=grad_fmt)
    c = mlp.scratch
    y, s = mlp.forward(x, residual)
    f.fp8_sync_status()
    for q, w in ((mlp.W1q, W1), (mlp.W1t, W1.t()), (mlp.W2q, W2), (mlp.W2t, W2.t())):
        assert_block(q, *ref.quantize(w, 0, 128), "weights")
    assert torch.equal(s, x if residual is None else (x.float() + residual.float()).bfloat16())
    n, rstd = plain(s, gamma, mlp.eps)
    near(mlp.rstd, rstd, 2.0 ** -20 * rstd, "rstd")
    assert_block(mlp.x8, *ref.quantize(s, 0), "x8")
    near_block(c.n8, n, 2.0 ** -19 * n.abs(), "n8")
    hh, a, eh, ta = product_fwd(c.n8, mlp.W1q)
    near_q(mlp.h8, hh, eh, "h8")
    near_q(c.a8, a, ta, "a8")
    near_product(y, c.a8, mlp.W2q, "y")

    dx, dW1, dW2, dgamma = mlp.backward(dy, ds)
    f.fp8_sync_status()
    assert_block(c.dy8, *ref.quantize(dy, grad_fmt), "dy8")
    assert_block(c.dy8t, *ref.quantize(dy.t(), grad_fmt), "dy8t")
    dh, a, tol, tol_a = product_bwd(c.dy8, mlp.W2t, mlp.h8)
    near_q(c.dh8, dh, tol, "dh8")
    near_q(c.dh8t, dh.t(), tol.t(), "dh8t")
    near_q(c.a8t, a.t(), tol_a.t(), "a8t")
    near_product(dW2, c.dy8t, c.a8t, "dW2")
    near_product(c.dn, c.dh8, mlp.W1t, "dn")
    seen = ref.values(mlp.x8)[0]
    nt = (seen * mlp.rstd.double()[:, None] * gamma.double()).t()
    near_block(c.n8t, nt, 2.0 ** -22 * nt.abs(), "n8t")
    near_product(dW1, c.dh8t, c.n8t, "dW1")
    check(dx, dgamma, c.dn, seen, gamma, mlp.rstd, ds, (M, K))
