"""PyTorch autograd wrapper of the C ABI (argument marshalling only).

``bam_attention`` is differentiable in q, k, v, the three per-head prior
parameters and the SSMax scale s: its forward calls ``bam_attn_fwd`` and
keeps O and the LSE, its backward calls ``bam_attn_bwd``.  Both run in the
library's CUDA kernels; nothing here computes a step of the method.

With ``prior=BAM_PRIOR_THETA`` the prior tensors are the BAM README's
theta_alpha, theta_beta, theta_mu ("Implementation Details":
b = -exp(theta_alpha) (|d - mu| + eps)^theta_beta, mu = 2 sinh(theta_mu)),
so the module's parameters can be trained as the authors parameterise them.
"""

from __future__ import annotations

import torch

from . import bam_attn as ba


def _rows_of(g):
    """A gradient as the library reads it: bf16, contiguous, its first row on 16 bytes (one
    of a slice may begin anywhere)."""
    g = g.to(torch.bfloat16).contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class BamAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, alpha, beta, mu, s, causal, ssmax, prior, eps, o_dtype):
        o, lse = ba.attention_forward(q, k, v, alpha, beta, mu, s, eps=eps, causal=causal,
                                      ssmax=ssmax, o_dtype=o_dtype, prior=prior)
        ctx.save_for_backward(q, k, v, o, lse, alpha, beta, mu, s)
        ctx.cfg = (causal, ssmax, prior, eps)
        return o

    @staticmethod
    def backward(ctx, dO):
        q, k, v, o, lse, alpha, beta, mu, s = ctx.saved_tensors
        causal, ssmax, prior, eps = ctx.cfg
        dq, dk, dv, da, db, dm, ds = ba.attention_backward(
            q, k, v, o, lse, _rows_of(dO), alpha, beta, mu, s, eps=eps, causal=causal, ssmax=ssmax,
            prior=prior)
        return (dq, dk, dv, da, db, dm, ds if s is not None else None,
                None, None, None, None, None)


def bam_attention(q, k, v, alpha, beta, mu, s=None, *, causal=True, ssmax=False,
                  prior=ba.BAM_PRIOR_ALPHA, eps=1e-5, o_dtype=None):
    """GGD-BAM attention with autograd.

    q, k, v: bf16 CUDA tensors [B, H, T, 64] (contiguous).  alpha, beta, mu
    (and s when ssmax): fp32 CUDA tensors [H].  Returns O [B, H, T, 64] in
    ``o_dtype`` (default bf16; fp32 keeps the parity-grade output).  The
    incoming gradient of O is rounded to bf16 for the backward kernel.
    """
    if ssmax and s is None:
        raise ValueError("ssmax needs the per-head scale s")
    o_dtype = o_dtype or torch.bfloat16
    return BamAttention.apply(q, k, v, alpha, beta, mu, s if ssmax else None, bool(causal),
                              bool(ssmax), int(prior), float(eps), o_dtype)


class QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, rope, eps):
        out = ba.qk_norm_forward(q, k, q_weight, k_weight, positions, rope, eps)
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        ctx.cfg = (rope, eps)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, positions = ctx.saved_tensors
        rope, eps = ctx.cfg
        dq, dk, dqw, dkw = ba.qk_norm_backward(q, k, _rows_of(dq_out), _rows_of(dk_out), q_weight, k_weight,
                                               positions, rope, eps)
        return dq, dk, dqw, dkw, None, None, None


def qk_norm(q, k, q_weight, k_weight, positions=None, rope=None, eps=1e-6):
    """Norms of queries and keys for each head and their rotation, with autograd.

    q: bf16 CUDA tensor [B, H, T, 64], k: [B, Hkv, T, 64], rows of 64 contiguous
    and 16-byte aligned (slices of a projection's output need no copy).
    q_weight, k_weight: fp32 [64], or [H, 64] and [Hkv, 64].  positions: int32
    [B, T] or None (0, 1, ..); rope: ``bam_attn.make_rope(...)`` or None.
    Returns contiguous (q_out, k_out), as ``bam_attention`` takes them.  Gradients
    are of the first order.

    Captured into a CUDA graph, take the gradients inside the capture with
    ``torch.autograd.grad``, and let go of every eager graph of the same leaves
    before: PyTorch ties a leaf's accumulation to the stream of the oldest graph
    that is alive, and a captured backward that reaches for that stream fails, which
    can end the process.
    """
    return QkNorm.apply(q, k, q_weight, k_weight, positions, rope, float(eps))
