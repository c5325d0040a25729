"""What is measured of the output head: the W4A16 product with NVFP4 weights, the log probabilities of
given tokens with their entropy and top alternatives, and the distillation loss from a teacher's top
alternatives, forward and backward.

Where `own` is false, run() computes the operators in plain torch, in 32 bits, rounded once at the end;
where it is true it makes the library's calls.  exact() states them in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda:0"
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------- cases --

def product(name, rows, k, n, out, e=1, topk=1, swiglu=False):
    """`rows` tokens, each routed to `topk` of `e` experts (e = 1: a dense layer)."""
    return dict(name=name, op="product", rows=rows, k=k, n=n, out=out, e=e, topk=topk, swiglu=swiglu)


def logprob(name, t, v, dtype, top, train=False, inv_temp=1.0, masked=0.0):
    return dict(name=name, op="logprob", t=t, v=v, dtype=dtype, top=top, train=train,
                inv_temp=inv_temp, masked=masked)


def distill(name, t, v, dtype, top, fused, renorm, inv_temp=1.0):
    return dict(name=name, op="distill", t=t, v=v, dtype=dtype, top=top, fused=fused, renorm=renorm,
                inv_temp=inv_temp)


def listed():
    return [
        # the smallest dense layer of the synthetic workloads, one token: what a call costs
        product("product_1x256x128", 1, 256, 128, "f32"),
        # the head of a decode step for one request: the whole matrix for one row
        product("product_head_1", 1, 4096, 131072, "f32"),
        # a head with an odd number of features for a small batch
        product("product_head_13_odd", 13, 2048, 100003, "bf16"),
        # the experts' gate/up projection of the 64-token decode step
        product("product_experts_64", 64, 2048, 1536, "bf16", e=128, topk=8, swiglu=True),
        # one sampled token's log probability with its alternatives: latency
        logprob("logprob_1", 1, 32768, "f32", 20),
        # a decode step's batch, part of the vocabulary masked, sampled at a temperature
        logprob("logprob_64", 64, 131072, "f32", 20, inv_temp=1.25, masked=0.3),
        # scoring a batch of rollouts with the learner
        logprob("logprob_4096", 4096, 131072, "bf16", 8),
        # the policy's loss on a short batch, an odd vocabulary in fp32
        logprob("logprob_train_1023_odd", 1023, 50001, "f32", 0, train=True),
        # the policy's loss on a long batch
        logprob("logprob_train_4096", 4096, 65536, "bf16", 0, train=True, inv_temp=0.7),
        # distillation of a few rows, log probabilities as they stand, through forward and backward
        distill("distill_33_odd", 33, 50001, "f32", 16, fused=False, renorm=False),
        # a distillation step over a vocabulary whose fp32 row is larger than a work-group's registers
        distill("distill_1000_wide", 1000, 100001, "f32", 20, fused=True, renorm=True),
        # a distillation step over a long batch
        distill("distill_4096", 4096, 131072, "bf16", 64, fused=True, renorm=True, inv_temp=0.5),
    ]


def log_range(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "logprob", "distill"])
    if op == "product":
        e = rng.choice([1, 1, log_range(rng, 2, 128)])
        topk = rng.randint(1, min(8, e))
        rows = log_range(rng, 1, 64)
        k = 16 * log_range(rng, 16, 256)
        n = log_range(rng, 128, min(131072, (1 << 29) // (e * k)))
        swiglu = rng.random() < 0.4
        return product("", rows, k, n + n % 2 if swiglu else n,
                       "bf16" if swiglu else rng.choice(["bf16", "f32"]), e, topk, swiglu)
    v = log_range(rng, 1000, 131072)
    t = log_range(rng, 1, min(4096, (1 << 28) // v))
    dtype = rng.choice(["bf16", "f32"])
    inv_temp = rng.choice([0.5, 1.0, 1.3])
    if op == "logprob":
        train = rng.random() < 0.5
        return logprob("", t, v, dtype, 0 if train else rng.choice([0, log_range(rng, 1, 128)]),
                       train, inv_temp, rng.choice([0.0, 0.5]))
    return distill("", t, v, dtype, log_range(rng, 1, 128), rng.random() < 0.6, rng.random() < 0.5,
                   inv_temp)


# ------------------------------------------------------------------------------------------ inputs --

def nvfp4_weights(g, e, n, k):
    """NVFP4 of N(0, 0.02) weights [e, n, k]: codes two to a byte, E4M3 scales per 16, one fp32 scale per expert."""
    nib = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((e, n, k // 16), dtype=torch.uint8, device=DEV)
    ts = torch.empty(max(e, 4), dtype=torch.float32, device=DEV)[:e]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for i in range(e):
        w = torch.randn((n, k), generator=g, device=DEV) * 0.02
        ts[i] = w.abs().max() / 2688.0
        b = w.view(n, k // 16, 16)
        s = (b.abs().amax(-1) / (6.0 * ts[i])).clamp_(max=448.0).to(torch.float8_e4m3fn)
        q = b / (s.float() * ts[i]).clamp_(min=1e-30)[..., None]
        code = torch.bucketize(q.abs(), edges).to(torch.uint8) + (q < 0).to(torch.uint8) * 8
        code = code.view(n, k)
        nib[i] = code[:, 0::2] | (code[:, 1::2] << 4)
        scale[i] = s.view(torch.uint8)
    return nib, scale, ts


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "product":
        t, e, topk, k = case["rows"], case["e"], case["topk"], case["k"]
        x = torch.randn((t, k), generator=g, device=DEV)
        x[:, torch.randperm(k, generator=g, device=DEV)[:max(1, k // 100)]] *= 20.0   # outlier channels
        s = dict(x=x.bfloat16(), w=nvfp4_weights(g, e, case["n"], k), offsets=None, row_token=None)
        if e > 1:
            ids = torch.rand((t, e), generator=g, device=DEV).argsort(1)[:, :topk].reshape(-1)
            order = ids.argsort(stable=True)
            counts = torch.bincount(ids, minlength=e)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
            s["row_token"] = (order // topk).int()
            s["most"] = int(counts.max())
        return dict(s, case=case)
    t, v, dtype = case["t"], case["v"], FLOATS[case["dtype"]]
    z = torch.randn((t, v), generator=g, device=DEV) * 2.0
    u = torch.rand((t, v), generator=g, device=DEV) * (v / 12.0)
    z = torch.where(u < 1.0, z - 1.5 * torch.log(u.clamp_(min=1e-6)), z)     # about 12 peaks in a row
    del u
    row = torch.arange(t, device=DEV)
    if case["op"] == "logprob":
        if case["masked"]:
            z.masked_fill_(torch.rand((1, v), generator=g, device=DEV) < case["masked"], -math.inf)
        z = z.to(dtype)
        noise = torch.empty((t, v), device=DEV).exponential_(generator=g).log_()
        ids = (z.float() * case["inv_temp"] - noise).argmax(1).int()
        if t > 1:
            ids[row % 16 == 5] = -1                               # prompt positions: no target
        return dict(case=case, logits=z, ids=ids,
                    g_logp=torch.randn(t, generator=g, device=DEV),
                    g_entropy=torch.randn(t, generator=g, device=DEV) * 0.1)
    teacher = z + torch.randn((t, v), generator=g, device=DEV) * 0.5
    val, ids = teacher.topk(case["top"], 1)
    val = val - teacher.logsumexp(1, keepdim=True)
    ids = ids.int()
    del teacher
    if case["top"] > 2:
        ids[row % 8 == 3, case["top"] - 2:] = -1                  # rows with fewer alternatives
    weight = torch.rand(t, generator=g, device=DEV) + 0.5
    weight[row % 8 == 6] = 0.0                                    # padded positions
    return dict(case=case, logits=z.to(dtype), t_val=val.contiguous(), t_id=ids.contiguous(),
                weight=weight, g=torch.rand(t, generator=g, device=DEV) + 0.5)


# --------------------------------------------------------------------------------------------- run --

def run(state):
    return {"product": run_product, "logprob": run_logprob, "distill": run_distill}[state["case"]["op"]](state)


def run_product(s):
    c = s["case"]
    if own:
        import nvfp4_w4a4_quantized_act_amd as Q
        out = Q.quads_moe_w4a16_gemv(s["x"], s["w"], c["n"], offsets=s["offsets"], row_token=s["row_token"],
                                     epilogue=Q.EPI_SWIGLU if c["swiglu"] else Q.EPI_NONE,
                                     out_dtype=Q.OUT_BF16 if c["out"] == "bf16" else Q.OUT_F32)
        return out.view(FLOATS[c["out"]])
    nib, scale, ts = s["w"]
    e, n, k = c["e"], c["n"], c["k"]
    value = torch.tensor([sign * m for sign in (1.0, -1.0) for m in E2M1], device=DEV)
    code = torch.stack([nib & 15, nib >> 4], -1).view(e, n, k // 16, 16)
    w = value[code.int()] * (scale.view(torch.float8_e4m3fn).float() * ts[:, None, None])[..., None]
    w = w.view(e, n, k)
    x = s["x"].float()
    if e == 1:
        y = x @ w[0].t()
    else:
        rows = s["row_token"].shape[0]
        p = torch.arange(rows, device=DEV)
        of = torch.searchsorted(s["offsets"][1:].long(), p, right=True)
        at = p - s["offsets"].long()[of]
        xe = torch.zeros((e, s["most"], k), device=DEV)
        xe[of, at] = x[s["row_token"].long()]
        y = torch.bmm(w, xe.transpose(1, 2).contiguous())[of, :, at]
    if c["swiglu"]:
        gate, up = y[:, :n // 2], y[:, n // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(FLOATS[c["out"]])


def run_logprob(s):
    c = s["case"]
    logits, ids, it = s["logits"], s["ids"], c["inv_temp"]
    if own:
        import nvfp4_w4a4_quantized_act_amd as Q
        r = Q.quads_token_logprob(logits, ids, inv_temp=it, topk=c["top"])
        if c["train"]:
            r["dlogits"] = Q.quads_token_logprob_backward(logits, ids, r["stats"], r["entropy"], s["g_logp"],
                                                          s["g_entropy"], inv_temp=it)
        return r
    z = logits.float()
    m = z.amax(1, keepdim=True)
    d = (z - m) * it
    ex = torch.exp(d)
    log_sum = ex.sum(1, keepdim=True).log()
    lp = d - log_sum
    p = torch.exp(lp)
    weighted = torch.where(p > 0, p * lp, 0.0)
    entropy = -weighted.sum(1)
    have = (ids >= 0) & (ids < c["v"])
    at = torch.where(have, ids, 0).long()[:, None]
    r = dict(logp=torch.where(have, lp.gather(1, at)[:, 0], 0.0), entropy=entropy,
             stats=torch.cat([m, log_sum], 1))
    if c["top"]:
        # one whole number per entry, larger for a larger value and then for a lower index
        bits = (z + 0.0).view(torch.int32)
        rank = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32)
        rank += torch.arange(c["v"] - 1, -1, -1, device=DEV)
        top = rank.topk(c["top"], 1)[1]
        r["top_id"], r["top_logp"] = top.int(), lp.gather(1, top)
    if c["train"]:
        g_lp = torch.where(have, s["g_logp"], 0.0)[:, None]
        grad = -(g_lp * p) - s["g_entropy"][:, None] * (weighted + p * entropy[:, None])
        grad.scatter_add_(1, at, g_lp)
        r["dlogits"] = (grad * it).to(logits.dtype)
    return r


def run_distill(s):
    c = s["case"]
    logits, t_val, t_id, weight, it = s["logits"], s["t_val"], s["t_id"], s["weight"], c["inv_temp"]
    if own:
        import nvfp4_w4a4_quantized_act_amd as Q
        if c["fused"]:
            loss, grad = Q.quads_topk_distill_grad(logits, t_val, t_id, weight, inv_temp=it, renorm=c["renorm"])
        else:
            loss, stats = Q.quads_topk_distill(logits, t_val, t_id, weight, inv_temp=it, renorm=c["renorm"])
            grad = Q.quads_topk_distill_backward(logits, t_val, t_id, stats, s["g"], weight, inv_temp=it,
                                                 renorm=c["renorm"])
        return dict(loss=loss, dlogits=grad)
    d = (logits.float() - logits.float().amax(1, keepdim=True)) * it
    lp = d - torch.exp(d).sum(1, keepdim=True).log()
    have = (t_id >= 0) & (t_id < c["v"])
    at = torch.where(have, t_id, 0).long()
    if c["renorm"]:
        t = torch.where(have, t_val * it, -math.inf)
        t = t - t.amax(1, keepdim=True)
        log_q = t - torch.exp(t).sum(1, keepdim=True).log()
    else:
        log_q = torch.where(have, t_val, -math.inf)
    q = torch.exp(log_q)
    loss = weight * torch.where(q > 0, q * (log_q - lp.gather(1, at)), 0.0).sum(1)
    grad = torch.exp(lp) * q.sum(1, keepdim=True)
    grad.scatter_add_(1, at, -q)
    by = weight * it if c["fused"] else weight * it * s["g"]
    return dict(loss=loss, dlogits=(grad * by[:, None]).to(logits.dtype))


# -------------------------------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "product":
        t, e, topk, k, n = (case[x] for x in ("rows", "e", "topk", "k", "n"))
        rows = t * topk
        active = e * (1.0 - (1.0 - topk / e) ** t) if e > 1 else 1.0     # experts some token is routed to
        cols = n // 2 if case["swiglu"] else n
        size = 2 if case["out"] == "bf16" else 4
        return dict(bytes=active * (n * k * 0.5625 + 4) + 2.0 * t * k + rows * cols * size,
                    flops=2.0 * rows * n * k)
    t, v = case["t"], case["v"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprob":
        passes = 2 if case["train"] else 1                          # the logits in, their gradients out
        return dict(bytes=float(t) * v * size * passes + t * (20.0 + 8 * case["top"]),
                    flops=float(t) * v * (14 if case["train"] else 6))
    live = t - sum(1 for i in range(t) if i % 8 == 6)               # padded rows are only written
    return dict(bytes=(live * float(v) + float(t) * v) * size + t * (12.0 + 8 * case["top"]),
                flops=live * float(v) * 9)


# ------------------------------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"product": exact_product, "logprob": exact_logprob, "distill": exact_distill}[case["op"]](case, s)


def exact_product(c, s):
    nib, scale, ts = s["w"]
    n, k = c["n"], c["k"]
    off = s["offsets"].tolist() if s["offsets"] is not None else [0, c["rows"]]
    rt = s["row_token"].long() if s["row_token"] is not None else torch.arange(c["rows"], device=DEV)
    y = torch.zeros((off[-1], n), dtype=torch.float64, device=DEV)
    for i in range(c["e"]):
        if off[i] == off[i + 1]:
            continue
        for n0 in range(0, n, 16384):
            b = nib[i, n0:n0 + 16384].long()
            code = torch.empty((b.shape[0], k), dtype=torch.int64, device=DEV)
            code[:, 0::2], code[:, 1::2] = b % 16, b // 16
            m = code % 8
            # E2M1: one mantissa bit, exponent (m >> 1) - 1, no hidden bit where the exponent field is 0
            w = torch.where(m < 2, 0.5 * m.double(), (2 + m % 2).double() * torch.exp2((m // 2).double() - 2))
            w = torch.where(code >= 8, -w, w)
            c8 = scale[i, n0:n0 + 16384].long()
            sb = torch.where(c8 < 8, c8.double() / 512, (8 + c8 % 8).double() * torch.exp2((c8 // 8).double() - 10))
            w = w * sb.repeat_interleave(16, 1) * ts[i].double()
            xr = s["x"][rt[off[i]:off[i + 1]]].double()
            y[off[i]:off[i + 1], n0:n0 + 16384] = xr @ w.t().contiguous()
    if c["swiglu"]:
        y = y[:, :n // 2] * torch.sigmoid(y[:, :n // 2]) * y[:, n // 2:]
    return y


def exact_logprob(c, s):
    t, v = c["t"], c["v"]
    f64 = dict(dtype=torch.float64, device=DEV)
    r = dict(logp=torch.zeros(t, **f64), entropy=torch.zeros(t, **f64), stats=torch.zeros((t, 2), **f64))
    if c["top"]:
        r["top_id"], r["top_logp"] = None, torch.zeros((t, c["top"]), **f64)
    if c["train"]:
        r["dlogits"] = torch.zeros((t, v), **f64)
    for a in range(0, t, 512):
        b = slice(a, min(t, a + 512))
        z = s["logits"][b].double()
        y = z * c["inv_temp"]
        lse = torch.logsumexp(y, 1)
        ids = s["ids"][b].long()
        have = (ids >= 0).double()
        lp = y - lse[:, None]
        p = lp.exp()
        plogp = torch.special.entr(p)                               # -p ln p, 0 where p = 0
        r["entropy"][b] = plogp.sum(1)
        picked = lp[torch.arange(len(ids), device=DEV), ids.clamp(min=0)]
        r["logp"][b] = torch.where(ids >= 0, picked, 0.0)
        r["stats"][b, 0] = z.max(1)[0]
        r["stats"][b, 1] = lse - z.max(1)[0] * c["inv_temp"]
        if c["top"]:
            r["top_logp"][b] = lp.topk(c["top"], 1)[0]
        if c["train"]:
            gl, ge = s["g_logp"][b].double() * have, s["g_entropy"][b].double()
            hot = torch.nn.functional.one_hot(ids.clamp(min=0), v).double()
            r["dlogits"][b] = c["inv_temp"] * (gl[:, None] * (hot - p)
                                               + ge[:, None] * (plogp - p * r["entropy"][b][:, None]))
    return r


def exact_distill(c, s):
    t, v, it = c["t"], c["v"], c["inv_temp"]
    loss = torch.zeros(t, dtype=torch.float64, device=DEV)
    grad = torch.zeros((t, v), dtype=torch.float64, device=DEV)
    for a in range(0, t, 512):
        b = slice(a, min(t, a + 512))
        y = s["logits"][b].double() * it
        lp = y - torch.logsumexp(y, 1, keepdim=True)
        ids, val = s["t_id"][b].long(), s["t_val"][b].double()
        full = torch.zeros((len(ids), v + 1), dtype=torch.float64, device=DEV)   # last column: no token
        q = torch.exp(val * it if c["renorm"] else val) * (ids >= 0)
        if c["renorm"]:
            q = q / q.sum(1, keepdim=True)
        full.scatter_add_(1, torch.where(ids < 0, v, ids), q)
        full = full[:, :v]
        w = s["weight"][b].double()
        loss[b] = w * (torch.special.xlogy(full, full) - full * lp).sum(1)
        by = w * it if c["fused"] else w * it * s["g"][b].double()
        grad[b] = by[:, None] * (full.sum(1, keepdim=True) * lp.exp() - full)
    return dict(loss=loss, dlogits=grad)
