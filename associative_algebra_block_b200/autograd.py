"""torch.autograd wrappers of the algebraic SwiGLU FFN and of the layer norm
ahead of it (libaal calls only).

``swiglu(law, q, rule, X, Wg, Wu, Wd)`` returns Y = (silu(X*Wg) . (X*Wu)) * Wd
with every product row-typed, and differentiates through ``aal_swiglu_bwd``.
The forward keeps its activation H for the backward; the backward allocates
the pre-activation and gradient workspaces it passes to the library.

``layer_norm(X, gamma, beta)`` is the norm of X's rows, and with ``residual``
the pair (norm of X + residual, the sum).  ``swiglu_block`` is the pre-norm
feed-forward sublayer X + swiglu(layer_norm(X)).  All arithmetic but that
sublayer's residual add runs in the CUDA library.

To capture a backward into a CUDA graph, first let go of every eager graph that
reaches the same leaves (its losses and outputs), as torch requires.
"""
from __future__ import annotations

import torch

from . import (_workspace_keep, aal_layer_norm_bwd, aal_layer_norm_bwd_workspace_size, aal_layer_norm_fwd,
               aal_set_workspace, aal_swiglu_bwd, aal_swiglu_fwd)


class _SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, law, q, rule, X, Wg, Wu, Wd):
        M, D, F = X.shape[0], X.shape[1], Wg.shape[1]
        H = torch.empty(M, F, dtype=X.dtype, device=X.device)
        Y = torch.empty(M, D, dtype=X.dtype, device=X.device)
        aal_swiglu_fwd(law, q, rule, X, Wg, Wu, Wd, H, Y)
        ctx.law, ctx.q, ctx.rule = law, q, rule
        ctx.save_for_backward(X, Wg, Wu, Wd, H)
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, Wg, Wu, Wd, H = ctx.saved_tensors
        dY = dY.contiguous()
        ws = [torch.empty_like(H) for _ in range(4)]  # G, U, dG, dU
        dX, dWg, dWu, dWd = (torch.empty_like(t) for t in (X, Wg, Wu, Wd))
        aal_swiglu_bwd(ctx.law, ctx.q, ctx.rule, X, Wg, Wu, Wd, H, dY, *ws, dX, dWg, dWu, dWd)
        return None, None, None, dX, dWg, dWu, dWd


def swiglu(law, q, rule, X, Wg, Wu, Wd):
    """Differentiable algebraic SwiGLU FFN on row-major CUDA tensors."""
    return _SwiGLU.apply(law, q, rule, X, Wg, Wu, Wd)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, gamma, beta, eps, residual):
        Y = torch.empty(X.shape, dtype=X.dtype, device=X.device)
        S = X if residual is None else torch.empty_like(Y)
        mean, rstd = (torch.empty(X.shape[0], dtype=torch.float32, device=X.device) for _ in range(2))
        aal_layer_norm_fwd(X, gamma, beta, Y, eps, R=residual, S=None if residual is None else S, mean=mean, rstd=rstd)
        ctx.has_residual = residual is not None
        ctx.beta_dtype = None if beta is None else beta.dtype
        ctx.save_for_backward(S, gamma, mean, rstd)
        return (Y, S) if ctx.has_residual else Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY, dS=None):
        S, gamma, mean, rstd = ctx.saved_tensors
        need_x, need_g, need_b, _, need_r = ctx.needs_input_grad
        M, d = S.shape
        dX = torch.empty(M, d, dtype=S.dtype, device=S.device) if need_x or need_r else None
        dgamma = torch.empty_like(gamma) if need_g else None
        dbeta = torch.empty(d, dtype=ctx.beta_dtype, device=S.device) if need_b else None
        # the column sums' workspace, in place of the thread's own for this call
        kept = getattr(_workspace_keep, "t", None)
        n = aal_layer_norm_bwd_workspace_size(M, d) if need_g or need_b else 0
        aal_set_workspace(torch.empty(n, dtype=torch.uint8, device=S.device) if n else None)
        try:
            aal_layer_norm_bwd(S, gamma, mean, rstd, dY.contiguous(), dX=dX, dgamma=dgamma, dbeta=dbeta,
                               dR=dS.contiguous() if dS is not None and dX is not None else None)
        finally:
            aal_set_workspace(kept)
        return dX if need_x else None, dgamma, dbeta, None, dX if need_r else None


def layer_norm(X, gamma=None, beta=None, eps=1e-5, residual=None):
    """Differentiable layer norm of the rows of X [M, d]; with ``residual``
    returns (norm of X + residual, X + residual)."""
    return _LayerNorm.apply(X, gamma, beta, eps, residual)


def swiglu_block(law, q, rule, X, gamma, beta, Wg, Wu, Wd, eps=1e-5):
    """Differentiable pre-norm feed-forward sublayer X + swiglu(layer_norm(X))."""
    return X + swiglu(law, q, rule, layer_norm(X, gamma, beta, eps), Wg, Wu, Wd)
