"""GPU test of the whole backward of LayerNorm + linear: the layer's own, which ends at the
gradient of LayerNorm's output, and fp8_layernorm_bwd from there with what the layer keeps."""
import pytest
import torch

import block_ref as ref
from test_gpu_block import gen
from test_gpu_saved import h, ln_bwd_tolerances, near

pytestmark = pytest.mark.gpu


def test_layernorm_linear_backward_to_its_input():
    import fp8_mixed_precision_amax_gb300 as f
    M, K, N = 256, 512, 384
    n = lambda *s: torch.randn(*s, generator=gen(M + len(s)), device="cuda")
    W, X, dY = (n(N, K) * K ** -0.5).bfloat16(), (2 * n(M, K) + 0.5).bfloat16(), (n(M, N) * 0.1).bfloat16()
    gamma, beta = (1 + 0.2 * n(K)).bfloat16(), (0.1 * n(K)).bfloat16()
    layer = f.Fp8LayerNormLinear(W, M, gamma, beta, 1e-5, f.Recipe())
    layer.forward(X)
    dX, dW = layer.backward(dY)
    of_output = dX.clone()
    dgamma, dbeta = torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    f.fp8_layernorm_bwd(dX, X, gamma, layer.mean, layer.rstd, dX, dgamma, dbeta)
    f.fp8_sync_status()
    # what the layer keeps is LayerNorm's statistics, and the rest is test_layernorm_bwd's check
    _, mean, rstd = ref.layernorm(X, gamma, beta, 1e-5)
    near(layer.mean, mean, 2.0 ** -20 * X.double().abs().mean(1), "mean")
    near(layer.rstd, rstd, 2.0 ** -19 * rstd, "rstd")
    want = ref.layernorm_bwd(of_output, X, gamma, layer.mean, layer.rstd)
    tol = ln_bwd_tolerances(of_output, X, gamma, layer.mean, layer.rstd, 0.0)
    near(dX, want[0], tol[0] + h(torch.bfloat16) * (want[0].abs() + tol[0]), "dx")
    near(dgamma, want[1], tol[1], "dgamma")
    near(dbeta, want[2], tol[2], "dbeta")
