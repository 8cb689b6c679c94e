"""What an Fp8BlockMlp holds: its memory, and layers that share the scratch of their passes."""
import pytest
import torch

from test_gpu_block_mlp import build

pytestmark = pytest.mark.gpu


def held():
    """Bytes that live tensors asked for (the allocator's own rounding is not theirs)."""
    return torch.cuda.memory_stats()["requested_bytes.all.current"]


def test_a_layer_that_shares_scratch_holds_what_it_says():
    """Beyond the first, a layer adds its weights (two FP8 copies), what it keeps and its results:
    no h in 16 bits, no transposes."""
    M, K, F = 2048, 512, 1408
    f, first, (gamma, beta, W1, W2, x, dy) = build(M, K, F)
    before = held()
    second = f.Fp8BlockMlp(gamma, beta, W1, W2, M, scratch=first.scratch)
    added = held() - before
    nb = lambda r, c, br=1: r * (-(-c // 16) * 16) + -(-r // br) * (-(-c // 512) * 4)
    kept = nb(M, K) + nb(M, 2 * F) + 8 * M
    weights = nb(2 * F, K, 128) + nb(K, 2 * F, 128) + nb(K, F, 128) + nb(F, K, 128)
    results = 2 * (2 * M * K + 2 * F * K + K * F) + 8 * K
    assert second.saved_bytes == kept
    assert added == kept + weights + results
    scratch = [(M, K), (M, F), (M, K), (K, M), (M, 2 * F), (2 * F, M), (F, M), (K, M)]
    assert first.scratch.nbytes == sum(nb(*s) for s in scratch) + 2 * M * (2 * F + F + K) + \
        f.fp8_layernorm_bwd_workspace(M, K)
    before = held()
    alone = f.Fp8BlockMlp(gamma, beta, W1, W2, M)
    assert held() - before == added + alone.scratch.nbytes


def test_layers_that_share_scratch_do_not_mix():
    """Forward of both, then backward of both: bit for bit what each gives by itself."""
    M, K, F = 300, 264, 384
    f, a, (gamma, beta, W1, W2, x, dy) = build(M, K, F)
    _, b, (gamma2, beta2, V1, V2, _, _) = build(M, K, F, seed=7)
    ya = a.forward(x).clone()
    yb = b.forward(ya).clone()
    db = [t.clone() for t in b.backward(dy)]
    da = [t.clone() for t in a.backward(db[0])]
    first = f.Fp8BlockMlp(gamma, beta, W1, W2, M)
    second = f.Fp8BlockMlp(gamma2, beta2, V1, V2, M, scratch=first.scratch)
    y = second.forward(first.forward(x))
    assert torch.equal(first.y, ya) and torch.equal(y, yb)
    for got, want in zip(second.backward(dy), db):
        assert torch.equal(got, want)
    for got, want in zip(first.backward(second.dx), da):
        assert torch.equal(got, want)


def test_scratch_of_other_sizes_is_refused():
    import fp8_mixed_precision_amax_gb300 as f
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    scratch = f.BlockMlpScratch(16, 64, 128)
    args = (z(64), z(64), z(256, 64), z(64, 128))
    f.Fp8BlockMlp(*args, 16, scratch=scratch)
    with pytest.raises(ValueError, match="scratch"):
        f.Fp8BlockMlp(*args, 17, scratch=scratch)
    with pytest.raises(ValueError, match="scratch"):
        f.Fp8BlockMlp(*args, 16, grad_fmt=f.E4M3, scratch=scratch)
    with pytest.raises(ValueError, match="scratch"):
        f.Fp8BlockMlp(z(64), z(64), z(512, 64), z(64, 256), 16, scratch=scratch)


def test_backward_before_any_forward_is_refused():
    """There is nothing kept to go back from, only what the memory held before."""
    f, mlp, (_, _, _, _, x, dy) = build(16, 64, 128)
    with pytest.raises(RuntimeError, match="forward"):
        mlp.backward(dy)
    mlp.forward(x)
    first = [t.clone() for t in mlp.backward(dy)]
    for a, b in zip(first, mlp.backward(dy)):    # what is kept stays for a second one
        assert torch.equal(a, b)
