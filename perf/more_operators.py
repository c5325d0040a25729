"""What is measured of the layer around the experts: the residual's addition with the root-mean-square norm
(bf16, fp32 or MX FP8 output, forward and backward), the router's top experts (forward and backward), and the
tokens sorted by expert and back with the routing weights applied (forward and backward).

Where `own` is false, run() computes the operators in plain torch, in 32 bits (in 64 where a value next to a
border of the 8-bit format decides), rounded once at the end; where it is true it makes the library's calls.
exact() states them in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda:0"
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases --

def norm(name, t, h, x, res, out, train=False):
    """t rows of h channels: x and the residual stream ("" for none) in their types, the output's format."""
    return dict(name=name, op="norm", t=t, h=h, x=x, res=res, out=out, train=train)


def route(name, t, e, topk, dtype, renorm, train=False):
    return dict(name=name, op="route", t=t, e=e, topk=topk, dtype=dtype, renorm=renorm, train=train)


def sort(name, t, h, e, topk, dtype, out, train=False, capacity=0):
    """t tokens to topk of e experts and back; capacity: rows that each expert has room for (0: as many as come)."""
    return dict(name=name, op="sort", t=t, h=h, e=e, topk=topk, dtype=dtype, out=out, train=train,
                capacity=capacity)


def listed():
    return [
        # one token of a decode step into the 8-bit experts: what a call costs
        norm("norm_1", 1, 2048, "bf16", "bf16", "fp8"),
        # a decode step's batch: the experts' fp32 sum into the bf16 residual stream, bf16 for the quantizers
        norm("norm_64", 64, 4096, "f32", "bf16", "bf16"),
        # the same of a long prefill, for the 8-bit product
        norm("norm_16384_fp8", 16384, 4096, "f32", "bf16", "fp8"),
        # short rows: one norm per attention head
        norm("norm_heads", 131072, 128, "bf16", "", "bf16"),
        # the learner's layer, forward and backward
        norm("norm_train_4096", 4096, 2048, "bf16", "bf16", "bf16", train=True),
        # an odd width and number of rows in fp32
        norm("norm_train_odd", 777, 5001, "f32", "f32", "f32", train=True),
        # a decode step's routing
        route("route_64", 64, 128, 8, "f32", True),
        # the learner's routing of a long batch, weights as the softmax over all experts gives them
        route("route_train_16384", 16384, 64, 8, "bf16", False, train=True),
        # a decode step's tokens to 128 experts and back
        sort("sort_64", 64, 2048, 128, 8, "bf16", "f32"),
        # experts with room for a limited number of rows, odd sizes, fp32
        sort("sort_train_odd", 333, 1001, 16, 3, "f32", "f32", train=True, capacity=67),
        # the learner's layer
        sort("sort_train_4096", 4096, 2048, 128, 8, "bf16", "bf16", train=True),
        # a long batch through wide experts
        sort("sort_train_16384", 16384, 4096, 64, 8, "bf16", "bf16", train=True),
    ]


def log_range(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "sort", "sort"])
    if op == "norm":
        h = log_range(rng, 16, 20000)
        train = rng.random() < 0.5
        out = rng.choice(["bf16", "f32"] if train else ["bf16", "f32", "fp8", "fp8"])
        if out == "fp8":
            h = (h + 31) // 32 * 32
        res = rng.choice(["", "bf16", "f32"])
        x = res if train and res else rng.choice(["bf16", "f32"])
        return norm("", log_range(rng, 1, max(1, min(65536, (1 << 25) // h))), h, x, res, out, train)
    if op == "route":
        e = log_range(rng, 4, 512)
        return route("", log_range(rng, 1, min(65536, (1 << 23) // e)), e, rng.randint(1, min(12, e)),
                     rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.random() < 0.5)
    e = log_range(rng, 2, 256)
    topk = rng.randint(1, min(8, e))
    h = log_range(rng, 16, 8192)
    t = log_range(rng, 1, max(1, min(16384, (1 << 27) // (h * topk))))
    return sort("", t, h, e, topk, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.random() < 0.6,
                rng.choice([0, 0, -(-t * topk * 5 // (4 * e))]))


# ------------------------------------------------------------------------------------------ inputs --

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rand(*shape, by=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=DEV) * by).to(dtype)

    s = dict(case=case)
    t = case["t"]
    if case["op"] == "norm":
        h = case["h"]
        far = torch.ones(h, device=DEV)
        far[torch.randperm(h, generator=g, device=DEV)[:max(1, h // 100)]] = 20.0      # outlier channels
        level = torch.exp(rand(t, 1, by=0.5))                                          # of each token
        s["x"] = (rand(t, h) * far * level).to(FLOATS[case["x"]])
        s["residual"] = (rand(t, h) * far * level * 2.0).to(FLOATS[case["res"]]) if case["res"] else None
        s["weight"] = (1.0 + rand(h, by=0.2)).to(FLOATS[case["x"]])
        if case["train"]:
            s["g"] = rand(t, h, by=0.1, dtype=FLOATS[case["out"]])
            s["g_sum"] = rand(t, h, by=0.1, dtype=FLOATS[case["res"]]) if case["res"] else None
    elif case["op"] == "route":
        s["logits"] = rand(t, case["e"], by=1.5, dtype=FLOATS[case["dtype"]])
        if case["train"]:
            s["g"] = rand(t, case["topk"])
    else:
        h, e, topk, c = case["h"], case["e"], case["topk"], case["capacity"]
        dtype = FLOATS[case["dtype"]]
        popular = rand(1, e, by=0.5)                                                   # some experts more than others
        top = (rand(t, e) + popular).topk(topk, 1)
        ids = top[1].reshape(-1)
        order = ids.argsort(stable=True)
        rank = torch.empty_like(order)
        rank[order] = torch.arange(t * topk, device=DEV)
        if c:                                                                          # what finds no room is left out
            first = torch.bincount(ids, minlength=e).cumsum(0) - torch.bincount(ids, minlength=e)
            at = rank - first[ids]
            rank = torch.where(at < c, ids * c + at, -1)
        s["pos"] = rank.int()
        s["rows"] = e * c if c else t * topk
        s["topk_w"] = torch.softmax(top[0], 1)
        s["x"] = rand(t, h, dtype=dtype)
        s["y"] = rand(s["rows"], h, by=0.3, dtype=dtype)                               # what the experts answer
        if case["train"]:
            s["g"] = rand(t, h, by=0.1, dtype=FLOATS[case["out"]])
            s["g_sorted"] = rand(s["rows"], h, by=0.1, dtype=dtype)
    return s


# --------------------------------------------------------------------------------------------- run --

def run(state):
    return {"norm": run_norm, "route": run_route, "sort": run_sort}[state["case"]["op"]](state)


def run_norm(s):
    c = s["case"]
    x, res, weight = s["x"], s["residual"], s["weight"]
    if own:
        import nvfp4_w4a4_quantized_act_amd as Q
        out = {"bf16": Q.OUT_BF16, "f32": Q.OUT_F32, "fp8": Q.OUT_MX_FP8}[c["out"]]
        r = Q.quads_rmsnorm(x, weight, EPS, residual=res, out_dtype=out)
        if c["out"] == "fp8":
            r["codes"] = r["codes"].view(torch.float8_e4m3fn)
        if c["train"]:
            r["dx"], _, r["dweight"] = Q.quads_rmsnorm_backward(s["g"], r.get("sum", x), weight, EPS,
                                                                g_sum=s["g_sum"])
        return r
    r = {}
    h = x
    if res is not None:
        h = r["sum"] = (x.float() + res.float()).to(res.dtype)
    if c["out"] == "fp8":
        h, w = h.double(), weight.double()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w
        blocks = y.view(c["t"], c["h"] // 32, 32)
        top = blocks.abs().amax(2)
        e = torch.where(top > 0, torch.frexp(top)[1] - 9, -127).clamp(-127, 127)
        v = torch.ldexp(blocks, -e[..., None]).clamp(-448.0, 448.0)
        step = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1].clamp(min=-5) - 4)   # the e4m3 grid's, at v
        r["codes"] = (torch.round(v / step) * step).view(c["t"], c["h"]).to(torch.float8_e4m3fn)
        r["scales"] = (e + 127).to(torch.uint8)
        return r
    h, w = h.float(), weight.float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * rstd
    r["y"] = (n * w).to(FLOATS[c["out"]])
    if c["train"]:
        g = s["g"].float()
        wg = g * w
        dx = rstd * (wg - n * (n * wg).mean(1, keepdim=True))
        if res is not None:
            dx = dx + s["g_sum"].float()
        r["dx"], r["dweight"] = dx.to(x.dtype), (g * n).sum(0).to(weight.dtype)
    return r


def run_route(s):
    c = s["case"]
    logits, topk, renorm = s["logits"], c["topk"], c["renorm"]
    if own:
        import nvfp4_w4a4_quantized_act_amd as Q
        ids, w = Q.quads_moe_route(logits, topk, renorm=renorm)
        r = dict(ids=ids, w=w)
        if c["train"]:
            r["dlogits"] = Q.quads_moe_route_backward(logits, ids, w, s["g"], renorm=renorm)
        return r
    z = logits.float()
    # one whole number per entry, larger for a larger value and then for a lower index
    bits = (z + 0.0).view(torch.int32)
    rank = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32)
    rank += torch.arange(c["e"] - 1, -1, -1, device=DEV)
    ids = rank.topk(topk, 1)[1]
    ex = torch.exp(z - z.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True)
    w = p.gather(1, ids)
    if renorm:
        w = ex.gather(1, ids)
        w = w / w.sum(1, keepdim=True)
    r = dict(ids=ids.int(), w=w)
    if c["train"]:
        gw = s["g"] * w
        if renorm:
            grad = torch.zeros_like(z).scatter_(1, ids, gw - w * gw.sum(1, keepdim=True))
        else:
            grad = (-p * gw.sum(1, keepdim=True)).scatter_add_(1, ids, gw)
        r["dlogits"] = grad.to(logits.dtype)
    return r


def run_sort(s):
    c = s["case"]
    x, y, pos, w, topk = s["x"], s["y"], s["pos"], s["topk_w"], c["topk"]
    rows = s["rows"] if c["capacity"] else None
    if own:
        import nvfp4_w4a4_quantized_act_amd as Q
        out = Q.OUT_BF16 if c["out"] == "bf16" else Q.OUT_F32
        r = dict(sorted=Q.quads_moe_sort(x, pos, topk, rows=rows), out=Q.quads_moe_unsort(y, pos, topk, w, out_dtype=out))
        if c["train"]:
            r["dy"], r["dw"] = Q.quads_moe_unsort_backward(s["g"], y, pos, topk, w, rows=rows)
            r["dx"] = Q.quads_moe_unsort(s["g_sorted"], pos, topk,
                                         out_dtype=Q.OUT_BF16 if c["dtype"] == "bf16" else Q.OUT_F32)
        return r
    t, h = c["t"], c["h"]
    have = pos >= 0
    at = torch.where(have, pos, s["rows"]).long()                    # what is left out goes to a row behind the last
    wide = torch.zeros((s["rows"] + 1, h), dtype=x.dtype, device=DEV)
    wide[at] = x.repeat_interleave(topk, 0)
    r = dict(sorted=wide[:-1])
    w = torch.where(have.view(t, topk), w, 0.0)

    def picked(rows_of):
        v = rows_of[torch.where(have, pos, 0).long()].float()
        return torch.where(have[:, None], v, 0.0).view(t, topk, h)

    yt = picked(y)
    r["out"] = (yt * w[..., None]).sum(1).to(FLOATS[c["out"]])
    if c["train"]:
        g = s["g"].float()
        dy = torch.zeros((s["rows"] + 1, h), dtype=y.dtype, device=DEV)
        dy[at] = (w[..., None] * g[:, None, :]).view(t * topk, h).to(y.dtype)
        r["dy"] = dy[:-1]
        r["dw"] = (yt * g[:, None, :]).sum(2)
        del yt
        r["dx"] = picked(s["g_sorted"]).sum(1).to(x.dtype)
    return r


# -------------------------------------------------------------------------------------------- work --

def work(case):
    size = {"bf16": 2.0, "f32": 4.0, "fp8": 1.0 + 1.0 / 32, "": 0.0}
    t = float(case["t"])
    if case["op"] == "norm":
        n = t * case["h"]
        x, res, out = size[case["x"]], size[case["res"]], size[case["out"]]
        total = n * (x + 2 * res + out) + case["h"] * x
        if case["train"]:                  # the gradients in, the summed rows again (they cannot stay), dx and dw out
            total += n * (out + res + (res or x) + x) + case["h"] * 2 * x
        return dict(bytes=total, flops=n * (14.0 if case["train"] else 5.0))
    if case["op"] == "route":
        n, k = t * case["e"], t * case["topk"]
        return dict(bytes=n * size[case["dtype"]] * (2 if case["train"] else 1) + k * (12 if case["train"] else 8),
                    flops=n * (8.0 if case["train"] else 4.0))
    h, k = case["h"], t * case["topk"]
    rows = float(case["e"] * case["capacity"]) if case["capacity"] else k
    live = min(rows, k)
    d, out = size[case["dtype"]], size[case["out"]]
    total = t * h * d + rows * h * d + live * h * d + t * h * out + k * 8
    flops = 2 * live * h
    if case["train"]:                      # the output's gradient and y in, dy and dw out; the sorted rows' in, dx out
        total += t * h * out + live * h * d + rows * h * d + k * 8 + live * h * d + t * h * d
        flops *= 4
    return dict(bytes=total, flops=flops)


# ------------------------------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "route": exact_route, "sort": exact_sort}[case["op"]](case, s)


def e4m3_grid():
    """The 127 finite magnitudes, in the order of their codes."""
    code = torch.arange(127, dtype=torch.float64, device=DEV)
    exponent, mantissa = torch.div(code, 8, rounding_mode="floor"), code % 8
    return torch.where(exponent == 0, mantissa * 2.0 ** -9, (8 + mantissa) * torch.pow(2.0, exponent - 10))


def exact_norm(c, s):
    x, res, w = s["x"].double(), s["residual"], s["weight"].double()
    r = {}
    h = x
    if res is not None:
        # rounded to the residual's type from the sum in fp32, as the operator is defined
        h = s["x"].float().add(res.float()).to(res.dtype).double()
        r["sum"] = h
    n = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / c["h"] + EPS)
    y = n * w
    if c["out"] == "fp8":
        grid = e4m3_grid()
        r["codes"], r["scales"] = torch.empty_like(y), None
        for a in range(0, c["t"], 2048):
            b = y[a:a + 2048].reshape(-1, 32)
            top = b.abs().max(1, keepdim=True)[0]
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
            e = torch.where(torch.pow(2.0, e) > top, e - 1, e)
            e = torch.where(torch.pow(2.0, e + 1) <= top, e + 1, e)
            e = torch.where(top > 0, (e - 8).clamp(-127, 127), -127.0)
            v = b.abs() * torch.pow(2.0, -e)
            low = (torch.searchsorted(grid, v.clamp(max=448.0), right=True) - 1).clamp(0, 126)
            high = (low + 1).clamp(max=126)
            below, above = v - grid[low], grid[high] - v
            up = (above < below) | ((above == below) & (low % 2 == 1))
            q = torch.where(up, grid[high], grid[low])
            r["codes"][a:a + 2048] = torch.copysign(q, b).view(-1, c["h"])
        return r
    r["y"] = y
    if c["train"]:
        g = s["g"].double()
        size = torch.sqrt((h * h).sum(1, keepdim=True) / c["h"] + EPS)
        along = (g * w * n).sum(1, keepdim=True) / c["h"]
        r["dx"] = (g * w - along * n) / size
        if res is not None:
            r["dx"] = r["dx"] + s["g_sum"].double()
        r["dweight"] = torch.einsum("th,th->h", g, n)
    return r


def exact_route(c, s):
    z = s["logits"].double()
    e, topk = c["e"], c["topk"]
    p = torch.softmax(z, 1)
    best = z.topk(topk, 1)[0]                                        # values only: equal ones need no order
    total = torch.logsumexp(best if c["renorm"] else z, 1, keepdim=True)
    r = dict(ids=None, w=torch.exp(best - total))
    if c["train"]:
        order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :topk]
        hot = torch.zeros((c["t"], e), dtype=torch.float64, device=DEV)
        hot[torch.arange(c["t"], device=DEV)[:, None], order] = s["g"].double() * r["w"]
        share = torch.where(torch.zeros_like(hot).scatter(1, order, 1.0) > 0, torch.exp(z - total), 0.0) if c["renorm"] else p
        r["dlogits"] = hot - share * hot.sum(1, keepdim=True)
    return r


def exact_sort(c, s):
    t, h, topk, rows = c["t"], c["h"], c["topk"], s["rows"]
    pos = s["pos"].long().view(t, topk)
    f64 = dict(dtype=torch.float64, device=DEV)
    r = dict(sorted=torch.zeros((rows, h), **f64), out=torch.zeros((t, h), **f64))
    if c["train"]:
        r.update(dy=torch.zeros((rows, h), **f64), dw=torch.zeros((t, topk), **f64), dx=torch.zeros((t, h), **f64))
    for k in range(topk):
        tok = torch.nonzero(pos[:, k] >= 0)[:, 0]
        at = pos[tok, k]
        w = s["topk_w"][tok, k].double()[:, None]
        r["sorted"].index_copy_(0, at, s["x"][tok].double())
        y = s["y"][at].double()
        r["out"].index_add_(0, tok, y * w)
        if c["train"]:
            g = s["g"][tok].double()
            r["dy"].index_copy_(0, at, g * w)
            r["dw"][tok, k] = torch.linalg.vecdot(g, y)
            r["dx"].index_add_(0, tok, s["g_sorted"][at].double())
    return r
