"""The block-scaled LayerNorm + SwiGLU MLP: its step against the formulas in 64 bits, its
determinism, and its capture into a CUDA graph.

Tolerance against the unquantized formulas (relative Frobenius error).  A rounding to
E4M3 is off by at most 2^-4 of the value, as a uniform error 2^-4 / sqrt(3) = 0.036
rms; E5M2 twice that, 0.072.  Errors of a product's operands add in squares:
  h: two operands                                   0.051
  a: both halves of h, the gate's slope up to 1.5,  0.10
     and h's own 8 bits in the backward pass
  y: a, its rounding and W2's                       0.12
  da: dy in E5M2 and W2                             0.08
  dh: da, both halves of h, its rounding            0.16
  dn, dW1, dW2: dh (or dy and a), an operand        0.20
doubled to leave room for values below the formats' normal range: 0.25 for y, 0.4 for
the gradients; a wrong operand or a wrong transpose is off by 1 or more."""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu


def build(M, K, F, seed=0, **kw):
    import fp8_mixed_precision_amax_gb300 as f
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    gamma, beta = (1 + 0.1 * n(K)).bfloat16(), (0.1 * n(K)).bfloat16()
    W1, W2 = (n(2 * F, K) * K ** -0.5).bfloat16(), (n(K, F) * F ** -0.5).bfloat16()
    x, dy = n(M, K).bfloat16() * 2, (n(M, K) * 1e-3).bfloat16()
    return f, f.Fp8BlockMlp(gamma, beta, W1, W2, M, **kw), (gamma, beta, W1, W2, x, dy)


def fro(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("M,K,F", [(300, 264, 384), (1, 128, 128), (777, 1000, 896)])
@pytest.mark.parametrize("grad_fmt", [0, 1])
def test_step_against_the_formulas(M, K, F, grad_fmt):
    f, mlp, (gamma, beta, W1, W2, x, dy) = build(M, K, F, grad_fmt=grad_fmt)
    y = mlp.forward(x)
    dx, dW1, dW2, dgamma, dbeta = mlp.backward(dy)
    f.fp8_sync_status()
    n, mean, rstd = ref.layernorm(x, gamma, beta, 1e-5)
    h = n @ W1.double().t()
    a = ref.swiglu(h)
    assert fro(y, a @ W2.double().t()) < 0.25
    dyd = dy.double()
    da = dyd @ W2.double()
    dh = ref.swiglu_bwd(da, h)
    dn = dh @ W1.double()
    want = ref.layernorm_bwd(dn, x, gamma, mean, rstd)
    for name, got, exact in [("dW2", dW2, dyd.t() @ a), ("dW1", dW1, dh.t() @ n), ("dx", dx, want[0]),
                             ("dgamma", dgamma, want[1]), ("dbeta", dbeta, want[2])]:
        assert fro(got, exact) < 0.4, (name, fro(got, exact))
    # what is kept is 8 bits and a byte per 128, and two statistics per token
    nb = lambda c: -(-c // 16) * 16 + -(-c // 512) * 4
    assert mlp.saved_bytes == M * (nb(K) + nb(2 * F) + 8)


def test_step_is_deterministic_and_its_graph_replays_it():
    f, mlp, (gamma, beta, W1, W2, x, dy) = build(520, 512, 640)
    first = [t.clone() for t in (mlp.forward(x), *mlp.backward(dy))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [mlp.forward(x, side), *mlp.backward(dy, side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp.forward(x)
        mlp.backward(dy)
    keep = x.clone()
    x.zero_()
    graph.replay()
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    now = [mlp.y, mlp.dx, mlp.dW1, mlp.dW2, mlp.dgamma, mlp.dbeta]
    assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_gradient_descent_lowers_the_loss():
    """Twenty steps on |y - target|^2 with the MLP's own gradients."""
    f, mlp, (gamma, beta, W1, W2, x, dy) = build(256, 256, 256, seed=3)
    target = torch.tanh(x.float() @ torch.randn(256, 256, device="cuda") / 16)
    W1, W2 = W1.float(), W2.float()
    losses = []
    for _ in range(20):
        y = mlp.forward(x).float()
        losses.append(float(((y - target) ** 2).mean()))
        _, dW1, dW2, _, _ = mlp.backward((2 * (y - target) / y.numel()).bfloat16())
        W1 -= 30.0 * dW1.float()
        W2 -= 30.0 * dW2.float()
        mlp.load_weights(W1.bfloat16(), W2.bfloat16())
    assert np.isfinite(losses).all() and losses[-1] < 0.7 * losses[0], losses


def test_refusals():
    import fp8_mixed_precision_amax_gb300 as f
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="W1"):
        f.Fp8BlockMlp(z(64), z(64), z(128, 64), z(64, 128), 16)
    with pytest.raises(ValueError, match="128"):
        f.Fp8BlockMlp(z(64), z(64), z(128, 64), z(64, 64), 16)
    mlp = f.Fp8BlockMlp(z(64), z(64), z(256, 64), z(64, 128), 16)
    with pytest.raises(ValueError, match="x must be"):
        mlp.forward(z(15, 64))
    with pytest.raises(ValueError, match="dy must be"):
        mlp.backward(z(16, 32))
