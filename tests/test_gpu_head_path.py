"""The output head's operators used together, as a rollout and its learner use
them: the W4A16 product's logits, their tokens' log-probabilities and top
alternatives, the distillation loss of a learner on those, and its gradient
down to the master weights; and the accuracy sweep's head workload (QUADS,
arXiv 2607.15810, Table 3) against the oracle."""

import numpy as np
import pytest
import torch

import synth
from nvfp4_w4a4_quantized_act_amd import qat
from nvfp4_w4a4_quantized_act_amd import sweep as S
from oracle import formats as F
from oracle import head as OH
from oracle import moe as OM
from oracle import nvfp4 as ON
from oracle import rac as OR

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


def up(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(DEV).view(torch.bfloat16)


def test_sweep_head_matches_oracle(Q):
    """Logits: |x w| sums S of at most 600 here; the product's bound is 180 u S, the GEMM's 1e-5 S
    = 168 u S, so a log-probability (two logits' errors) is off by at most 2 * 360 u S < 0.03 in
    the worst case; roundings of random sign leave sqrt(K) rather than K of them, a hundredth of
    that.  The figures are held to 2e-4 and a relative 1e-3."""
    sizes = dict(m=48, k_dim=512, n=2000)
    got = S.sweep_head(Q, torch, synth, torch.device(DEV), **sizes)
    d = synth.make(2, **dict(S.HEAD, **sizes))
    x = F.bf16_to_f64(d["x"])
    w = ON.weight_qdq(d["w"])[:3]
    learner, _ = OH.w4a16(x, w, [0, sizes["m"]])
    ids = S.sample_tokens(learner)
    lp = OH.token_logprob(learner, ids)["logp"]
    assert [g["k"] for g in got] == [0, 64, 128, 256, 384, 512]
    for g in got:
        k = g["k"]
        o = OR.rac_quantize(x, k)
        r = (o["r_nib"], o["r_scale"], o["r_ts"]) if k else None
        y, _ = OM.grouped_gemm((o["nib"], o["scale"], o["ts"]), r, o["sel"], w,
                               [0, sizes["m"]])
        p = OH.token_logprob(y, ids, topk=S.HEAD_TOP)
        gap = np.abs(lp - p["logp"])
        div = OH.distill(learner, p["top_logp"], p["top_id"], renorm=False).mean()
        for key, want in (("max_gap", gap.max()), ("mean_gap", gap.mean()), ("divergence", div)):
            assert abs(g[key] - want) <= 2e-4 + 1e-3 * abs(want), (k, key, g[key], want)
    assert got[-1]["mean_gap"] < 0.3 * got[0]["mean_gap"]     # RAC narrows the gap
    assert "head | 12.5 % | 64 |" in S.head_table(got)


def test_rollout_to_learner(Q):
    """Teacher: the W4A16 head's logits for one decode step, their top alternatives.  Student: a
    QAT head on the same hidden states, distilled; its master weights' gradient is dz^T x
    (straight through, Eq. (13)) with dz the oracle's for the student's own bf16 logits."""
    t, k, v, top = 24, 256, 1500, 32
    rng = np.random.default_rng(3)
    xb = synth.activations(rng, rng, t, k, "normal", 3.0, 3, 10.0)[0]
    wt = up(synth.weights(rng, 1, v, k, std=0.05))
    ws = up(synth.weights(rng, 1, v, k, std=0.05))[0].clone().requires_grad_()
    x = up(xb)
    wq = Q.quads_nvfp4_weight_qdq(wt.view(torch.int16))[:3]
    teacher = Q.quads_moe_w4a16_gemv(x, wq, v)
    ids = teacher.argmax(1).int()
    r = Q.quads_token_logprob(teacher, ids, topk=top)
    assert torch.equal(r["top_id"][:, 0], ids) and torch.equal(r["top_logp"][:, 0], r["logp"])
    # the teacher's logits are the oracle's
    want, bound = OH.w4a16(F.bf16_to_f64(xb), [a.cpu().numpy() for a in wq], [0, t])
    assert (np.abs(teacher.cpu().numpy() - want) <= 177 * U * bound).all()

    z = qat.qat_linear(x, ws)
    z.retain_grad()
    loss = qat.distill_loss(z, r["top_logp"], r["top_id"])
    lp, h = qat.token_logprobs(z, ids)
    (loss.mean() - 0.1 * lp.mean() - 0.01 * h.mean()).backward()
    torch.cuda.synchronize()
    zr = z.detach().double().cpu().numpy()
    tv, ti = r["top_logp"].cpu().numpy(), r["top_id"].cpu().numpy()
    one = np.full(t, 1.0 / t)
    dz = OH.distill_grad(zr, tv, ti, one) + OH.token_logprob_grad(zr, ids.cpu().numpy(), -0.1 * one,
                                                                  -0.01 * one)
    # z's gradient: two bf16 tensors (half a step each, of terms of at most 1 / t and 0.2 / t),
    # their bf16 sum (half a step)
    got = z.grad.double().cpu().numpy()
    p = np.exp(OH.log_softmax(zr, 1.0))
    a, b = np.abs(OH.distill_grad(zr, tv, ti, one)), 0.2 / t * p + 0.1 / t * (p > 0)
    assert (np.abs(got - dz) <= 2.0 ** -8 * (a + b + np.abs(dz)) + 1e-6 / t).all()
    # the weights' gradient of z's own gradient: a bf16 product with fp32 sums
    gw = got.T @ F.bf16_to_f64(xb)
    sw = np.abs(got).T @ np.abs(F.bf16_to_f64(xb))
    assert ws.grad.shape == ws.shape
    err = np.abs(ws.grad.double().cpu().numpy() - gw)
    assert (err <= 2.0 ** -8 * np.abs(gw) + (t + 8) * U * sw).all()


def test_experts_layer_of_one_step(Q):
    """A MoE layer of one decode step in W4A16: packing, both products (SwiGLU in the first), the
    combine, against the oracle's layer on the GPU's own intermediate values."""
    t, e, topk, h, i = 7, 16, 4, 256, 96
    d = synth.make(4, t=t, e=e, h=h, i=i, topk=topk)
    x = up(d["x"])
    w13 = Q.quads_nvfp4_weight_qdq(up(d["w13"]).view(torch.int16))[:3]
    w2 = Q.quads_nvfp4_weight_qdq(up(d["w2"]).view(torch.int16))[:3]
    off, rt, pos = Q.quads_moe_pack(torch.from_numpy(d["topk_ids"]).to(DEV), e)
    hb = Q.quads_moe_w4a16_gemv(x, w13, 2 * i, offsets=off, row_token=rt, epilogue=Q.EPI_SWIGLU,
                                out_dtype=Q.OUT_BF16)
    y = Q.quads_moe_w4a16_gemv(hb, w2, h, offsets=off)
    out = Q.quads_moe_combine(y, pos, torch.from_numpy(d["topk_w"]).to(DEV))
    torch.cuda.synchronize()
    offn, rtn, posn = OM.pack_routes(d["topk_ids"], e)
    y1, _ = OH.w4a16(F.bf16_to_f64(d["x"]), ON.weight_qdq(d["w13"])[:3], offn, rtn)
    want_h = F.bf16_to_f64(OM.swiglu(y1))
    got_h = F.bf16_to_f64(hb.cpu().numpy().view(np.uint16))
    assert (np.abs(got_h - want_h) <= 2.0 ** -7 * np.abs(want_h) + 1e-6).all()   # one bf16 step
    y2, b2 = OH.w4a16(got_h, ON.weight_qdq(d["w2"])[:3], offn)
    assert (np.abs(y.cpu().numpy() - y2) <= 177 * U * b2).all()
    want = OM.combine(y.cpu().numpy(), posn, d["topk_w"], t, topk)
    bound = OM.combine(np.abs(y.cpu().numpy()), posn, np.abs(d["topk_w"]), t, topk)
    assert (np.abs(out.cpu().numpy() - want) <= topk * U * bound + 1e-30).all()
