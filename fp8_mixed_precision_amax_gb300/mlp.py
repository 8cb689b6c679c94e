"""LayerNorm + SwiGLU MLP in block-scaled FP8, from the block-scaled operators of api.

    n = LayerNorm(x);  h = n W1^T = [gate | value];  y = SwiGLU(h) W2^T

All four products (and the two of the weight gradients) run on FP8 operands with
a power-of-two scale for each block of 128.  From forward to backward a layer keeps
x and h alone, both in 8 bits, with LayerNorm's two statistics per token; the
backward pass computes LayerNorm's and SwiGLU's outputs again from them, straight
into the transposed operands that the weight gradients need.  What a pass needs
while it runs is not kept: layers of the same sizes share one set of it
(``BlockMlpScratch``).
"""
from __future__ import annotations

import logging

import torch

from .api import (E4M3, E5M2, BlockFp8, fp8_block_gemm_tn, fp8_block_quantize, fp8_layernorm_bwd,
                  fp8_layernorm_bwd_workspace, fp8_layernorm_fwd, fp8_layernorm_recompute,
                  fp8_swiglu_bwd, fp8_swiglu_fwd, _on_stream)

_log = logging.getLogger(__name__)


class BlockMlpScratch:
    """What the passes of an Fp8BlockMlp of ``M`` tokens, [K -> F -> K], need while they
    run.  Any number of layers of these sizes may share one, if their passes do not
    overlap on the GPU (one stream, or streams that wait for one another)."""

    def __init__(self, M: int, K: int, F: int, grad_fmt: int = E5M2, device="cuda"):
        self.key = (M, K, F, grad_fmt)
        e = lambda r, c, fmt=E4M3: BlockFp8.empty(r, c, fmt, device=device)
        b = lambda r, c: torch.empty((r, c), dtype=torch.bfloat16, device=device)
        # forward: LayerNorm's output, h, SwiGLU's output
        self.n8, self.h, self.a8 = e(M, K), b(M, 2 * F), e(M, F)
        # backward: the gradients and their transposes, both outputs again
        self.dy8, self.dy8t, self.da = e(M, K, grad_fmt), e(K, M, grad_fmt), b(M, F)
        self.dh8, self.dh8t = e(M, 2 * F, grad_fmt), e(2 * F, M, grad_fmt)
        self.a8t, self.n8t, self.dn = e(F, M), e(K, M), b(M, K)
        self.workspace = torch.empty(fp8_layernorm_bwd_workspace(M, K), dtype=torch.uint8,
                                     device=device)

    @property
    def nbytes(self) -> int:
        return sum(t.nbytes for t in vars(self).values() if isinstance(t, (BlockFp8, torch.Tensor)))


class Fp8BlockMlp:
    """The MLP for ``M`` tokens: owns its weights' FP8 copies, what it keeps from forward
    to backward, and its results.

    ``gamma``, ``beta`` [K]; ``W1`` [2F, K]; ``W2`` [K, F], F a multiple of 128.
    ``grad_fmt``: format of the gradients' FP8 operands.  ``scratch``: another layer's, to
    share; a set of its own when None.  Everything is enqueued on the given (else the
    current) stream with no host synchronisation, so a step can be captured into a CUDA
    graph."""

    def __init__(self, gamma: torch.Tensor, beta: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                 M: int, eps: float = 1e-5, grad_fmt: int = E5M2, stream=None,
                 scratch: BlockMlpScratch | None = None):
        K, F = W2.shape
        if tuple(W1.shape) != (2 * F, K):
            raise ValueError(f"W1 must be [{2 * F}, {K}] for W2 {tuple(W2.shape)}")
        if F % 128:
            raise ValueError(f"W2's columns must be a multiple of 128, got {F}")
        dev = W1.device
        if scratch is None:
            with _on_stream(stream, dev):
                scratch = BlockMlpScratch(M, K, F, grad_fmt, dev)
        elif scratch.key != (M, K, F, grad_fmt):
            raise ValueError(f"scratch is of (M, K, F, grad_fmt) {scratch.key}, "
                             f"not {(M, K, F, grad_fmt)}")
        elif scratch.workspace.device != dev:
            raise ValueError(f"scratch is on {scratch.workspace.device}, the weights on {dev}")
        self.gamma, self.beta, self.eps, self.grad_fmt = gamma, beta, eps, grad_fmt
        self.M, self.K, self.F, self.scratch = M, K, F, scratch
        e = lambda r, c, block=1: BlockFp8.empty(r, c, E4M3, block, device=dev)
        b = lambda r, c: torch.empty((r, c), dtype=torch.bfloat16, device=dev)
        v = lambda n: torch.empty(n, dtype=torch.float32, device=dev)
        with _on_stream(stream, dev):
            # weights, in tiles of 128 x 128, and their transposes for the input gradients
            self.W1q, self.W1t = e(2 * F, K, 128), e(K, 2 * F, 128)
            self.W2q, self.W2t = e(K, F, 128), e(F, K, 128)
            # kept from forward to backward
            self.x8, self.h8, self.mean, self.rstd = e(M, K), e(M, 2 * F), v(M), v(M)
            # results
            self.y, self.dx = b(M, K), b(M, K)
            self.dW1, self.dW2, self.dgamma, self.dbeta = b(2 * F, K), b(K, F), v(K), v(K)
        self._kept = False    # nothing yet
        self.load_weights(W1, W2, stream)
        _log.info("FP8 block-scaled MLP [%d -> %d -> %d], %d tokens: E4M3 forward, %s backward, "
                  "%.1f MB kept per pass, %.1f MB of scratch", K, F, K, M,
                  "E5M2" if grad_fmt == E5M2 else "E4M3", self.saved_bytes / 1e6,
                  scratch.nbytes / 1e6)

    @property
    def saved_bytes(self) -> int:
        """Bytes kept from the forward to the backward pass; ``scratch.nbytes`` are needed
        besides, once for all layers that share it."""
        return self.x8.nbytes + self.h8.nbytes + 8 * self.M

    def load_weights(self, W1: torch.Tensor, W2: torch.Tensor, stream=None) -> None:
        """Quantizes new weights (after an optimizer step)."""
        fp8_block_quantize(W1, self.W1q, self.W1t, stream)
        fp8_block_quantize(W2, self.W2q, self.W2t, stream)

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """y [M, K] (bfloat16) of x [M, K]; keeps x and h in 8 bits."""
        if tuple(x.shape) != (self.M, self.K):
            raise ValueError(f"x must be [{self.M}, {self.K}], got {tuple(x.shape)}")
        s = self.scratch
        fp8_layernorm_fwd(x, self.gamma, self.beta, self.eps, self.mean, self.rstd, y8=s.n8,
                          x8=self.x8, stream=stream)
        fp8_block_gemm_tn(s.n8, self.W1q, s.h, stream)
        fp8_swiglu_fwd(s.h, s.a8, self.h8, stream)
        fp8_block_gemm_tn(s.a8, self.W2q, self.y, stream)
        self._kept = True
        return self.y

    def backward(self, dy: torch.Tensor, stream=None):
        """(dx, dW1, dW2, dgamma, dbeta) of the last forward; dy [M, K]."""
        if tuple(dy.shape) != (self.M, self.K):
            raise ValueError(f"dy must be [{self.M}, {self.K}], got {tuple(dy.shape)}")
        if not self._kept:
            raise RuntimeError("backward needs a forward before it")
        s = self.scratch
        fp8_block_quantize(dy, s.dy8, s.dy8t, stream)
        fp8_block_gemm_tn(s.dy8, self.W2t, s.da, stream)
        fp8_swiglu_bwd(s.da, self.h8, s.dh8, s.dh8t, s.a8t, stream)
        fp8_block_gemm_tn(s.dy8t, s.a8t, self.dW2, stream)
        fp8_block_gemm_tn(s.dh8, self.W1t, s.dn, stream)
        fp8_layernorm_recompute(self.x8, self.gamma, self.beta, self.mean, self.rstd, s.n8t,
                                stream)
        fp8_block_gemm_tn(s.dh8t, s.n8t, self.dW1, stream)
        fp8_layernorm_bwd(s.dn, self.x8, self.gamma, self.mean, self.rstd, self.dx, self.dgamma,
                          self.dbeta, s.workspace, stream)
        return self.dx, self.dW1, self.dW2, self.dgamma, self.dbeta
