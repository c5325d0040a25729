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

Forward and backward of these operators may be captured into a HIP graph.  As with
any of torch's operators, take the captured gradients with torch.autograd.grad,
or call .backward() only while no eager result of the same leaves is alive:
torch would wait, inside the capture, for the stream of the eager one.
"""

import torch

from . import (OUT_BF16, OUT_F32, quads_moe_route, quads_moe_route_backward, quads_moe_sort,
               quads_moe_unsort, quads_moe_unsort_backward, quads_nvfp4_weight_qdq, quads_rmsnorm,
               quads_rmsnorm_backward, quads_token_logprob, quads_token_logprob_backward,
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


def _code(dtype):
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("the type must be torch.float32 or torch.bfloat16")
    return OUT_BF16 if dtype == torch.bfloat16 else OUT_F32


class RMSNorm(torch.autograd.Function):
    """(y, h) of h = x + residual, y = h / sqrt(mean h^2 + eps) * weight, over the last dimension.

    The leading dimensions are taken in here: an input's gradient must reach autograd as the one
    tensor object that dx and dres are, so that the first leaf copies it.  Reshaped outside, it
    would become two views of one memory, which both leaves keep, and add to twice.
    """

    @staticmethod
    def forward(ctx, x, residual, weight, eps, out_dtype):
        n, shape = x.shape[-1], x.shape
        rows = x.reshape(-1, n)
        r = quads_rmsnorm(rows, weight, eps, None if residual is None else residual.reshape(-1, n),
                          _code(out_dtype))
        # not views: they may be changed in place as any operator's results
        y, h = (v if v is None or v.shape == shape else torch.ops.aten._unsafe_view(v, shape)
                for v in (r["y"], r.get("sum")))
        ctx.save_for_backward(x if h is None else h, weight)
        ctx.eps, ctx.x_dtype, ctx.added = eps, x.dtype, h is not None
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g, g_sum):
        h, weight = ctx.saved_tensors
        for_x, for_res, for_w = ctx.needs_input_grad[:3]
        for_res = for_res and ctx.added
        if g is None:
            if g_sum is None:
                return None, None, None, None, None
            return g_sum.to(ctx.x_dtype) if for_x else None, g_sum if for_res else None, None, None, None
        n, any_rows = h.shape[-1], for_x or for_res
        # an input that needs no gradient gets none; where only the weight does, dx is written all
        # the same, in the narrow type, and without h's other gradient
        g_sum = g_sum.reshape(-1, n) if any_rows and g_sum is not None else None
        dx, dres, dw = quads_rmsnorm_backward(
            g.reshape(-1, n), h.reshape(-1, n), weight, ctx.eps, g_sum,
            ctx.x_dtype if for_x else h.dtype if for_res else torch.bfloat16, for_w, for_res)
        one = dres is dx
        dx = dx.view(h.shape)
        if for_res:
            dres = dx if one else dres.view(h.shape)
        return dx if for_x else None, dres if for_res else None, dw, None, None


def rms_norm(x, weight=None, eps=1e-6, residual=None, out_dtype=None):
    """Root-mean-square norm over the last dimension of x [..., H] (float32 or bf16), times
    weight [H].  With a residual of x's shape: (y, h), the norm of h = x + residual and h itself
    in the residual's type, the next residual.  y has the type out_dtype (h's).  Differentiable
    in x, residual and weight."""
    for t in (x, weight, residual):
        if t is not None:
            _code(t.dtype)
    if residual is not None and residual.shape != x.shape:
        raise ValueError("residual must have the shape of x")
    if out_dtype is None:
        out_dtype = x.dtype if residual is None else residual.dtype
    y, h = RMSNorm.apply(x, residual, weight, float(eps), out_dtype)
    return y if residual is None else (y, h)


class Route(torch.autograd.Function):
    """(weights, ids) of the topk experts of each row of logits; gradient for the logits."""

    @staticmethod
    def forward(ctx, logits, topk, renorm):
        ids, w = quads_moe_route(logits, topk, renorm)
        ctx.save_for_backward(logits, ids, w)
        ctx.renorm = renorm
        ctx.mark_non_differentiable(ids)
        return w, ids

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g, _):
        logits, ids, w = ctx.saved_tensors
        return quads_moe_route_backward(logits, ids, w, g, ctx.renorm), None, None


def route(logits, topk, renorm=True):
    """Routing weights (fp32) and ids (int32) [..., topk] of the experts with the largest logits
    [..., E] (float32 or bf16): softmax over all experts, or over the chosen ones (renorm).
    Differentiable in the logits, through the weights of the chosen experts."""
    _code(logits.dtype)
    w, ids = Route.apply(logits.reshape(-1, logits.shape[-1]), int(topk), bool(renorm))
    shape = logits.shape[:-1] + (int(topk),)
    return w.reshape(shape), ids.reshape(shape)


class SortTokens(torch.autograd.Function):
    """Rows of x copied to the packed rows that pos names; the gradient adds them up again."""

    @staticmethod
    def forward(ctx, x, pos, topk, rows):
        ctx.save_for_backward(pos)
        ctx.topk, ctx.dtype = topk, x.dtype
        return quads_moe_sort(x, pos, topk, rows)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        pos, = ctx.saved_tensors
        return quads_moe_unsort(g, pos, ctx.topk, out_dtype=_code(ctx.dtype)), None, None, None


def sort_tokens(x, pos, topk, rows=None):
    """Tokens x [T, H] (float32 or bf16) in expert order [rows, H]: row pos[t * topk + s] is x[t].
    rows None: pos is a permutation of the T * topk rows (`quads_moe_pack`'s).  With rows given,
    slots whose pos is outside [0, rows) are left out and rows without a slot are 0; no row has
    two slots.  Differentiable in x."""
    _code(x.dtype)
    return SortTokens.apply(x, pos, int(topk), rows)


class UnsortTokens(torch.autograd.Function):
    """Weighted sums of the packed rows that pos names; gradient for the rows and the weights."""

    @staticmethod
    def forward(ctx, y, pos, topk, topk_w, out_dtype, rows):
        ctx.save_for_backward(y, pos, topk_w)
        ctx.topk, ctx.rows = topk, rows
        return quads_moe_unsort(y, pos, topk, topk_w, _code(out_dtype))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        y, pos, topk_w = ctx.saved_tensors
        dy, dw = quads_moe_unsort_backward(g, y, pos, ctx.topk, topk_w, ctx.rows,
                                           ctx.needs_input_grad[0], ctx.needs_input_grad[3])
        return dy, None, None, dw, None, None


def unsort_tokens(y, pos, topk, topk_w=None, out_dtype=torch.float32, rows=None):
    """Experts' rows y [rows, H] (float32 or bf16) back in token order [T, H]: the sum over a
    token's slots of topk_w[t, s] * y[pos[t * topk + s]] (topk_w fp32 [T, topk], None: 1).  rows
    as in sort_tokens: None says that pos is a permutation of y's rows; otherwise y's number of
    rows, and rows without a slot get a zero gradient.  Differentiable in y and topk_w."""
    _code(y.dtype)
    if y.shape[0] != (pos.numel() if rows is None else rows):
        raise ValueError("y must have T * topk rows, or as many as rows says")
    return UnsortTokens.apply(y, pos, int(topk), topk_w, out_dtype, rows)
