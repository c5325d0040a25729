"""Trainer-side asymmetric W4A16 QAT (QUADS, arXiv 2607.15810, section 3.2).

The learner fake-quantizes its weights with the same NVFP4 operator the
rollout kernels use, and keeps its activations in bf16:

  forward   W_hat = QDQ_W(W),  Y = X W_hat^T                         Eq. (12)
  backward  dL/dW ~= dL/dW_hat (straight-through),  dL/dX = dY W_hat  Eq. (13)

QDQ_W is `quads_nvfp4_weight_qdq` itself: one dynamic fp32 tensor scale per
expert matrix, E4M3 scales over 16-element blocks along K, E2M1 codes with
ties to even -- the call that produces the rollout's NVFP4 weights.  Its bf16
output is the round-to-nearest-even bf16 of the exact decode v * s_b * s_t,
so the learner sees, bit for bit, the bf16 image of the values the rollout's
W4A4 GEMM multiplies (Eq. (16): the weight term of the mismatch vanishes);
where s_t is a power of two the two are the same numbers.

The matrix product of the learner is the trainer's own (torch); the QDQ node
runs in the library, and so do the losses on its logits: the log-probabilities
of the rollout's tokens with the entropy (`token_logprobs`, the quantity that
the method aligns between rollout and learner) and the distillation from
another model's top alternatives (`distill_loss`).

Forward and backward of the losses may be captured into a HIP graph.  As with
any of torch's operators, take the captured gradients with torch.autograd.grad,
or call .backward() only while no eager result of the same leaves is alive:
torch would wait, inside the capture, for the stream of the eager one.
"""

import torch

from . import (quads_nvfp4_weight_qdq, quads_token_logprob, quads_token_logprob_backward,
               quads_topk_distill, quads_topk_distill_backward)


class WeightQDQ(torch.autograd.Function):
    """W_hat = QDQ_W(W) for bf16 W [E, N, K] or [N, K]; straight-through gradient."""

    @staticmethod
    def forward(ctx, w):
        if w.dtype != torch.bfloat16:
            raise TypeError("QAT master weights are bf16")
        w3 = w.detach().contiguous()
        squeeze = w3.dim() == 2
        if squeeze:
            w3 = w3.unsqueeze(0)
        if w3.dim() != 3:
            raise ValueError("weights must be [N, K] or [E, N, K]")
        _nib, _scale, _ts, dq = quads_nvfp4_weight_qdq(w3.view(torch.int16), want_dq=True)
        out = dq.view(torch.bfloat16)
        return out[0] if squeeze else out

    @staticmethod
    def backward(ctx, grad):
        return grad                                  # Eq. (13): straight through


def weight_qdq(w):
    """QDQ_W(w) with the straight-through gradient (Eq. (12), (13))."""
    return WeightQDQ.apply(w)


def qat_linear(x, w):
    """Learner forward of one projection under W4A16 QAT: x [.., K] bf16, w [N, K] bf16 master.

    Leading dimensions of x are flattened so that torch runs plain 2-D
    products (forward and backward), never batched ones."""
    k = x.shape[-1]
    y = torch.nn.functional.linear(x.reshape(-1, k), weight_qdq(w))
    return y.reshape(*x.shape[:-1], w.shape[0])


class TokenLogprobs(torch.autograd.Function):
    """(ln p[ids], entropy) of softmax(inv_temp * logits); gradient for the logits."""

    @staticmethod
    def forward(ctx, logits, ids, inv_temp):
        r = quads_token_logprob(logits, ids, inv_temp=inv_temp)
        ctx.save_for_backward(logits, ids, r["stats"], r["entropy"])
        ctx.inv_temp = inv_temp
        ctx.set_materialize_grads(False)
        return r["logp"], r["entropy"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logp, g_entropy):
        if g_logp is None and g_entropy is None:
            return None, None, None
        logits, ids, stats, entropy = ctx.saved_tensors
        return quads_token_logprob_backward(logits, ids, stats, entropy, g_logp, g_entropy,
                                            inv_temp=ctx.inv_temp), None, None


def token_logprobs(logits, ids, inv_temp=1.0):
    """Log-probabilities (fp32) of the tokens ids int32 and the entropies of the rows of logits
    [..., V] (float32 or bf16), differentiable in the logits.  An id outside [0, V) marks a
    position without a token: its log-probability is 0, without a gradient."""
    if ids.shape != logits.shape[:-1]:
        raise ValueError("ids must have the shape of the logits without the last dimension")
    lp, h = TokenLogprobs.apply(logits.reshape(-1, logits.shape[-1]), ids.reshape(-1),
                                float(inv_temp))
    return lp.reshape(ids.shape), h.reshape(ids.shape)


class DistillLoss(torch.autograd.Function):
    """Loss per row from a teacher's top alternatives; gradient for the logits."""

    @staticmethod
    def forward(ctx, logits, t_val, t_id, weight, inv_temp, renorm):
        loss, stats = quads_topk_distill(logits, t_val, t_id, weight, inv_temp, renorm)
        ctx.save_for_backward(logits, t_val, t_id, weight, stats)
        ctx.inv_temp, ctx.renorm = inv_temp, renorm
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        logits, t_val, t_id, weight, stats = ctx.saved_tensors
        return (quads_topk_distill_backward(logits, t_val, t_id, stats, g, weight, ctx.inv_temp,
                                            ctx.renorm), None, None, None, None, None)


def distill_loss(logits, t_val, t_id, weight=None, inv_temp=1.0, renorm=True):
    """Distillation loss (fp32) of each row of logits [..., V] from a teacher's alternatives
    t_val fp32 and t_id int32 [..., topk] (`quads_token_logprob`'s top_logp and top_id of the
    teacher's logits): w sum_i q_i (ln q_i - ln p_i), q the teacher's probabilities, over the
    list renormalised (`renorm`) or as they stand.  Differentiable in the logits only."""
    lead = logits.shape[:-1]
    if t_val.shape[:-1] != lead or t_id.shape != t_val.shape:
        raise ValueError("t_val and t_id must be [..., topk] over the logits' rows")
    if weight is not None and weight.shape != lead:
        raise ValueError("weight must have one entry per row of the logits")
    if t_val.requires_grad or (weight is not None and weight.requires_grad):
        raise ValueError("distill_loss has no gradient for the teacher's values or the weights")
    k = t_val.shape[-1]
    loss = DistillLoss.apply(logits.reshape(-1, logits.shape[-1]), t_val.reshape(-1, k),
                             t_id.reshape(-1, k),
                             None if weight is None else weight.reshape(-1), float(inv_temp),
                             bool(renorm))
    return loss.reshape(lead)
