"""MLPs in block-scaled FP8, from the block-scaled operators of api: Fp8BlockMlp, LayerNorm +
SwiGLU, and Fp8GatedMlp, a pre-norm residual layer with the RMS norm and the gated product
in one kernel each (its own docstring says more).

LayerNorm + SwiGLU:

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

from .api import (E4M3, E5M2, BlockFp8, fp8_block_gemm_swiglu_bwd, fp8_block_gemm_swiglu_fwd,
                  fp8_block_gemm_tn, fp8_block_quantize, fp8_layernorm_bwd,
                  fp8_layernorm_bwd_workspace, fp8_layernorm_fwd, fp8_layernorm_recompute,
                  fp8_rmsnorm_bwd, fp8_rmsnorm_bwd_workspace, fp8_rmsnorm_fwd,
                  fp8_rmsnorm_recompute, fp8_swiglu_bwd, fp8_swiglu_fwd, _on_stream)

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


class GatedMlpScratch:
    """What the passes of an Fp8GatedMlp of ``M`` tokens, [K -> F -> K], need while they run.
    Any number of layers of these sizes may share one, if their passes do not overlap on the GPU
    (one stream, or streams that wait for one another)."""

    def __init__(self, M: int, K: int, F: int, grad_fmt: int = E5M2, device="cuda"):
        self.key = (M, K, F, grad_fmt)
        e = lambda r, c, fmt=E4M3: BlockFp8.empty(r, c, fmt, device=device)
        # forward: the norm's output, the gated product
        self.n8, self.a8 = e(M, K), e(M, F)
        # backward: the gradients and their transposes, both outputs again
        self.dy8, self.dy8t = e(M, K, grad_fmt), e(K, M, grad_fmt)
        self.dh8, self.dh8t = e(M, 2 * F, grad_fmt), e(2 * F, M, grad_fmt)
        self.a8t, self.n8t = e(F, M), e(K, M)
        self.dn = torch.empty((M, K), dtype=torch.bfloat16, device=device)
        self.workspace = torch.empty(fp8_rmsnorm_bwd_workspace(M, K), dtype=torch.uint8,
                                     device=device)

    @property
    def nbytes(self) -> int:
        return sum(t.nbytes for t in vars(self).values() if isinstance(t, (BlockFp8, torch.Tensor)))


class Fp8GatedMlp:
    """A pre-norm residual MLP layer for ``M`` tokens:

        s = x + residual;  n = RMSNorm(s);  [g | u] = n W1^T;  y = (SiLU(g) u) W2^T

    whose y and s are the next layer's x and residual.  The residual's addition is part of the
    norm's kernel and SwiGLU part of the product's, forward and backward; h = [g | u] and its
    gradient are never in 16 bits.  From forward to backward the layer keeps s and h, both in
    8 bits, and a statistic per token.  It owns its weights' FP8 copies and its results.

    ``gamma`` [K]; ``W1`` [2F, K]; ``W2`` [K, F], F a multiple of 128.  ``grad_fmt``: format of
    the gradients' FP8 operands.  ``scratch``: another layer's, to share; a set of its own when
    None.  Everything is enqueued on the given (else the current) stream with no host
    synchronisation, so a step can be captured into a CUDA graph."""

    def __init__(self, gamma: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, M: int,
                 eps: float = 1e-6, grad_fmt: int = E5M2, stream=None,
                 scratch: GatedMlpScratch | None = None):
        K, F = W2.shape
        if tuple(W1.shape) != (2 * F, K):
            raise ValueError(f"W1 must be [{2 * F}, {K}] for W2 {tuple(W2.shape)}")
        if F % 128:
            raise ValueError(f"W2's columns must be a multiple of 128, got {F}")
        dev = W1.device
        if scratch is None:
            with _on_stream(stream, dev):
                scratch = GatedMlpScratch(M, K, F, grad_fmt, dev)
        elif scratch.key != (M, K, F, grad_fmt):
            raise ValueError(f"scratch is of (M, K, F, grad_fmt) {scratch.key}, "
                             f"not {(M, K, F, grad_fmt)}")
        elif scratch.workspace.device != dev:
            raise ValueError(f"scratch is on {scratch.workspace.device}, the weights on {dev}")
        self.gamma, self.eps, self.grad_fmt = gamma, eps, grad_fmt
        self.M, self.K, self.F, self.scratch = M, K, F, scratch
        e = lambda r, c, block=1: BlockFp8.empty(r, c, E4M3, block, device=dev)
        b = lambda r, c: torch.empty((r, c), dtype=torch.bfloat16, device=dev)
        v = lambda n: torch.empty(n, dtype=torch.float32, device=dev)
        with _on_stream(stream, dev):
            # weights, in tiles of 128 x 128, and their transposes for the input gradients
            self.W1q, self.W1t = e(2 * F, K, 128), e(K, 2 * F, 128)
            self.W2q, self.W2t = e(K, F, 128), e(F, K, 128)
            # kept from forward to backward
            self.x8, self.h8, self.rstd = e(M, K), e(M, 2 * F), v(M)
            # results
            self.y, self.s, self.dx = b(M, K), b(M, K), b(M, K)
            self.dW1, self.dW2, self.dgamma = b(2 * F, K), b(K, F), v(K)
        self._kept = False    # nothing yet
        self.load_weights(W1, W2, stream)
        _log.info("FP8 gated MLP [%d -> %d -> %d], %d tokens: E4M3 forward, %s backward, "
                  "%.1f MB kept per pass, %.1f MB of scratch", K, F, K, M,
                  "E5M2" if grad_fmt == E5M2 else "E4M3", self.saved_bytes / 1e6,
                  scratch.nbytes / 1e6)

    @property
    def saved_bytes(self) -> int:
        """Bytes kept from the forward to the backward pass; ``scratch.nbytes`` are needed
        besides, once for all layers that share it."""
        return self.x8.nbytes + self.h8.nbytes + 4 * self.M

    def load_weights(self, W1: torch.Tensor, W2: torch.Tensor, stream=None) -> None:
        """Quantizes new weights (after an optimizer step)."""
        fp8_block_quantize(W1, self.W1q, self.W1t, stream)
        fp8_block_quantize(W2, self.W2q, self.W2t, stream)

    def _check(self, t: torch.Tensor | None, name: str) -> None:
        if t is not None and (tuple(t.shape) != (self.M, self.K) or t.dtype != torch.bfloat16):
            raise ValueError(f"{name} must be [{self.M}, {self.K}] in bfloat16, got "
                             f"{tuple(t.shape)} in {t.dtype}")

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, stream=None):
        """(y, s) [M, K] (bfloat16) of x and the residual [M, K] (none: s is x); keeps s and h
        in 8 bits."""
        self._check(x, "x")
        self._check(residual, "residual")
        c = self.scratch
        fp8_rmsnorm_fwd(x, self.gamma, self.eps, self.rstd, residual=residual,
                        sum=None if residual is None else self.s, y8=c.n8, x8=self.x8,
                        stream=stream)
        fp8_block_gemm_swiglu_fwd(c.n8, self.W1q, c.a8, self.h8, stream)
        fp8_block_gemm_tn(c.a8, self.W2q, self.y, stream)
        self._kept = True
        return self.y, x if residual is None else self.s

    def backward(self, dy: torch.Tensor, ds: torch.Tensor | None = None, stream=None):
        """(dx, dW1, dW2, dgamma) of the last forward from the gradients of y and of s (None:
        s has no other use); dx [M, K] is the gradient of x and of the residual alike."""
        self._check(dy, "dy")
        self._check(ds, "ds")
        if not self._kept:
            raise RuntimeError("backward needs a forward before it")
        c = self.scratch
        fp8_block_quantize(dy, c.dy8, c.dy8t, stream)
        fp8_block_gemm_swiglu_bwd(c.dy8, self.W2t, self.h8, c.dh8, c.dh8t, c.a8t, stream)
        fp8_block_gemm_tn(c.dy8t, c.a8t, self.dW2, stream)
        fp8_block_gemm_tn(c.dh8, self.W1t, c.dn, stream)
        fp8_rmsnorm_recompute(self.x8, self.gamma, self.rstd, c.n8t, stream)
        fp8_block_gemm_tn(c.dh8t, c.n8t, self.dW1, stream)
        fp8_rmsnorm_bwd(c.dn, self.x8, self.gamma, self.rstd, self.dx, self.dgamma, ds,
                        c.workspace, stream)
        return self.dx, self.dW1, self.dW2, self.dgamma
