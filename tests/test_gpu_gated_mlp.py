"""The pre-norm gated MLP layer (RMS norm with the residual's addition, gated product): its step
against the formulas in 64 bits, two layers with clipping and the Adam step behind them,
determinism, capture into a CUDA graph.

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
the gradients; a wrong operand or a wrong transpose is off by 1 or more.  A second layer has the
first one's errors in its input, beside the residual that carries none: half as much again."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu


def weights(K, F, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return ((1 + 0.1 * n(K)).bfloat16(), (n(2 * F, K) * K ** -0.5).bfloat16(), (n(K, F) * F ** -0.5).bfloat16())


def inputs(M, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda s: (torch.randn(M, K, generator=g, device="cuda") * s).bfloat16()
    return n(0.5), n(2.0), n(1e-3), n(1e-3)


def lib():
    import fp8_mixed_precision_amax_gb300 as f
    return f


def fro(got, want):
    return float((got.double() - want).norm() / want.norm())


def plain(x, residual, gamma, W1, W2, eps=1e-6):
    s = x if residual is None else x + residual
    n = s * (s.square().mean(1, keepdim=True) + eps) ** -0.5 * gamma
    return ref.swiglu(n @ W1.t()) @ W2.t(), s


@pytest.mark.parametrize("M,K,F", [(300, 264, 384), (1, 128, 128), (777, 1000, 896)])
@pytest.mark.parametrize("grad_fmt", [0, 1])
@pytest.mark.parametrize("with_residual", [True, False])
def test_step_against_the_formulas(M, K, F, grad_fmt, with_residual):
    f = lib()
    params = weights(K, F, M)
    x, residual, dy, ds = inputs(M, K, K)
    residual, ds = (residual, ds) if with_residual else (None, None)
    mlp = f.Fp8GatedMlp(*params, M, grad_fmt=grad_fmt)
    y, s = mlp.forward(x, residual)
    got = mlp.backward(dy, ds)
    f.fp8_sync_status()
    leaves = [t.double().requires_grad_() for t in (x, *params)]
    r = None if residual is None else residual.double()
    y0, s0 = plain(leaves[0], r, *leaves[1:])
    loss = (y0 * dy.double()).sum() + (0 if ds is None else (s0 * ds.double()).sum())
    dx, dgamma, dW1, dW2 = torch.autograd.grad(loss, leaves)
    assert fro(y, y0.detach()) < 0.25
    assert fro(s, s0.detach()) < 2.0 ** -8
    for name, g, want in zip(("dx", "dW1", "dW2", "dgamma"), got, (dx, dW1, dW2, dgamma)):
        assert fro(g, want) < 0.4, (name, fro(g, want))
    nb = lambda c: -(-c // 16) * 16 + -(-c // 512) * 4
    assert mlp.saved_bytes == M * (nb(K) + nb(2 * F) + 4)


def two_layers(f, M, K, F, scratch=True):
    params = [weights(K, F, k) for k in range(2)]
    first = f.Fp8GatedMlp(*params[0], M)
    second = f.Fp8GatedMlp(*params[1], M, scratch=first.scratch if scratch else None)
    return params, first, second


def pass_of(layers, x, r, dy, ds):
    """Both layers forward and backward: the second's residual is the first's s."""
    first, second = layers
    y, s = first.forward(x, r)
    y2, s2 = second.forward(y, s)
    dx, *g2 = second.backward(dy, ds)     # of y and of s: the residual has the same gradient
    dx1, *g1 = first.backward(dx, dx)
    return y2, s2, dx1, [*g1, *g2]


def test_two_layers_then_clipping_and_adam():
    f = lib()
    M, K, F = 260, 256, 384
    params, first, second = two_layers(f, M, K, F)
    x, r, dy, ds = inputs(M, K, 9)
    y, s, dx, grads = pass_of((first, second), x, r, dy * 1000, ds)
    leaves = [t.double().requires_grad_() for t in (x, *params[0], *params[1])]
    ya, sa = plain(leaves[0], r.double(), *leaves[1:4])
    yb, sb = plain(ya, sa, *leaves[4:])
    want = torch.autograd.grad((yb * dy.double() * 1000).sum() + (sb * ds.double()).sum(), leaves)
    y = y.clone()   # the layer's own buffer
    assert fro(y, yb.detach()) < 0.375 and fro(s, sb.detach()) < 0.25
    exact = [want[0], want[2], want[3], want[1], want[5], want[6], want[4]]
    for k, (g, w) in enumerate(zip([dx, *grads], exact)):
        assert fro(g, w) < 0.6, (k, fro(g, w))
    # the gradients' norm, and the clipped ones for the Adam step, which takes 16 bits
    norm = torch.empty(1, device="cuda")
    f.fp8_grad_norm(grads, norm)
    outs = [torch.empty_like(g, dtype=torch.bfloat16) for g in grads]
    f.fp8_grad_clip(grads, norm, 1.0, outs)
    total = sum(float(g.double().square().sum()) for g in grads) ** 0.5
    assert total > 1 and abs(norm.item() - total) <= 2.0 ** -20 * total
    clipped = sum(float(g.double().square().sum()) for g in outs) ** 0.5
    assert abs(clipped - 1) <= 2.0 ** -8
    before = [p.clone() for layer in params for p in layer[1:]]
    matrices = [p for layer in params for p in layer[1:]]
    states = [f.Fp8AdamState(p) for p in matrices]
    steps = [outs[0], outs[1], outs[3], outs[4]]
    for state, g, p in zip(states, steps, matrices):
        state.step(g, p, f.AdamHyper(lr=1e-3))
    first.load_weights(*params[0][1:]), second.load_weights(*params[1][1:])
    f.fp8_sync_status()
    # Adam's first step moves each weight by lr g / (|g| + eps), for gradients far above eps = 1e-8
    # by lr, to the roundings of FP16 states and BF16 weights: against the gradient's sign
    for p, b, g in zip(matrices, before, steps):
        moved, big = (p.double() - b.double()), g.abs() > 1e-5
        half = 2.0 ** -8 * b.double().abs() + 2.0 ** -11 * b.abs().max().double()
        assert ((moved + 1e-3 * g.double().sign()).abs() <= 2e-5 + 2 * half)[big].all()
    y2, *_ = pass_of((first, second), x, r, dy, ds)
    assert torch.isfinite(y2).all() and not torch.equal(y2, y)


def test_sharing_scratch_changes_nothing_and_graphs_replay():
    f = lib()
    M, K, F = 520, 512, 640
    x, r, dy, ds = inputs(M, K, 1)
    flat = lambda p: [t.clone() for t in (p[0], p[1], p[2], *p[3])]
    _, a, b = two_layers(f, M, K, F, scratch=False)
    alone = flat(pass_of((a, b), x, r, dy, ds))
    _, a, b = two_layers(f, M, K, F)
    assert a.scratch is b.scratch
    shared = flat(pass_of((a, b), x, r, dy, ds))
    assert all(torch.equal(p, q) for p, q in zip(alone, shared))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = flat(pass_of((a, b), x, r, dy, ds))
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(alone, again))
    # two graphs over the same layers and scratch, replayed in turn on new data
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pass_of((a, b), x, r, dy, ds))
        graphs.append(g)
    keep = x.clone()
    x.zero_()
    graphs[0].replay()
    x.copy_(keep)
    for g, o in zip(graphs, outs):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(alone, flat(o)))


def test_refusals():
    f = lib()
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="W1"):
        f.Fp8GatedMlp(z(64), z(128, 64), z(64, 128), 16)
    with pytest.raises(ValueError, match="128"):
        f.Fp8GatedMlp(z(64), z(128, 64), z(64, 64), 16)
    with pytest.raises(ValueError, match="scratch"):
        f.Fp8GatedMlp(z(64), z(256, 64), z(64, 128), 16, scratch=f.GatedMlpScratch(17, 64, 128))
    mlp = f.Fp8GatedMlp(z(64), z(256, 64), z(64, 128), 16)
    with pytest.raises(RuntimeError, match="forward"):
        mlp.backward(z(16, 64))
    for bad in (z(15, 64), z(16, 64).float()):
        with pytest.raises(ValueError, match="x must be"):
            mlp.forward(bad)
        with pytest.raises(ValueError, match="residual must be"):
            mlp.forward(z(16, 64), bad)
    mlp.forward(z(16, 64))
    with pytest.raises(ValueError, match="dy must be"):
        mlp.backward(z(16, 32))
    with pytest.raises(ValueError, match="ds must be"):
        mlp.backward(z(16, 64), z(16, 32))
