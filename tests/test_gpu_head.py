"""Log-probabilities, distillation and their gradients on the GPU against
oracle/head.py in fp64.

Tolerances, derived (u = 2^-24, half a step of fp32).  With d = it (z - m):
  * the kernel reaches d (or d / ln 2) by at most 6 roundings, so its error is
    at most 6 u |d|; terms with |d| > 104 are below the smallest fp32 number;
  * a term e^d then has the relative error 6 u |d| + 4 u (exponential to 2
    ulps), and a sum in which no term meets more than n additions adds n u.  A
    row is summed by at least 256 threads, then over threads and parts of the
    row: n <= V / 256 + 64.  The log-sum s takes one more logarithm (2 ulps of
    s, and 2 u).  Hence |err s| <= err_s = (6 min(D, 104) + n + 8 + 4 |s|) u,
    D = max |d| over unmasked entries;
  * ln p = d - s: err_lp = 6 u |d| + err_s + 2 u |ln p|;
  * H = s - sum p d: p has the relative error err_s + 6 u |d| + 8 u, so
    err_H = err_s + sum p |d| (err_s + 6 u |d| + (n + 12) u) + 2 u H + 2 u s;
  * a gradient is made of terms of p with p's relative error
    err_p = err_lp + 8 u, plus 4 roundings of each term and of the sum, plus
    half a step of the output's type and the smallest subnormal.  The hardware's
    exponential gives 0 below the smallest normal number, 2^-126: p has that
    absolute error too, and a term is p times its other factors, so 2^-126
    times those factors is added.
"""

import numpy as np
import pytest
import torch

from oracle import head as OH

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


@pytest.fixture(scope="module")
def qat():
    from nvfp4_w4a4_quantized_act_amd import qat as m
    return m


def make(t, v, dtype, seed=0, scale=2.0, masked=0.0, ld=None, empty=()):
    """Logits on the GPU (a view with row stride ld) and their exact values in fp64."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((t, v), generator=g) * scale
    if masked:
        z[torch.rand((t, v), generator=g) < masked] = -float("inf")
    for r in empty:
        z[r] = -float("inf")
    z = z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    full = torch.full((t, ld or v), 7.5, dtype=z.dtype)
    full[:, :v] = z
    return full.to(DEV)[:, :v], z.double().numpy()


def errors_of(z, it):
    """ln p and err_s, err_lp, err_H of the derivation."""
    v = z.shape[1]
    m, s = OH.row_stats(z, it)
    lp = OH.log_softmax(z, it)
    d = np.where(np.isneginf(z), 0.0, it * (z - np.where(np.isneginf(m), 0, m)[:, None]))
    n = v / 256 + 64
    es = (6 * np.minimum(np.abs(d).max(1), 104) + n + 8 + 4 * np.abs(s)) * U
    fin = np.where(np.isneginf(lp), 0.0, lp)
    elp = 6 * U * np.abs(d) + es[:, None] + 2 * U * np.abs(fin)
    p = np.exp(lp)
    eh = es + (p * np.abs(d) * (es[:, None] + 6 * U * np.abs(d) + (n + 12) * U)).sum(1)
    eh += 2 * U * (np.abs(s) + (p * np.abs(fin)).sum(1))
    return lp, es, elp, eh


def close(got, want, tol):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True)
    err = np.abs(got[fin] - want[fin])
    tol = np.broadcast_to(tol, want.shape)[fin]
    assert np.isfinite(got[fin]).all()
    bad = err > tol
    assert not bad.any(), (float(err[bad].max()), float((err / np.maximum(tol, 1e-300)).max()),
                           int(bad.sum()), np.argwhere(bad)[:4].tolist())


def tokens(z, seed):
    t, v = z.shape
    ids = np.random.default_rng(seed).integers(0, v, t).astype(np.int32)
    for i, x in ((1, -1), (2, v), (3, -2 ** 31), (4, 2 ** 31 - 1)):
        if t > 5:
            ids[i] = x
    return ids


def check_logprob(Q, z, zr, it, topk, seed=1, want_entropy=True):
    t, v = zr.shape
    ids = tokens(zr, seed)
    print(f"logprob T={t} V={v} ld={z.stride(0)} {z.dtype} it={it} k={topk}", flush=True)
    r = Q.quads_token_logprob(z, torch.from_numpy(ids).to(DEV), it, topk, want_entropy)
    torch.cuda.synchronize()
    e = OH.token_logprob(zr, ids, it, topk)
    lp, es, elp, eh = errors_of(zr, it)
    have = (ids >= 0) & (ids < v)
    at = np.where(have, ids, 0)
    close(r["logp"], e["logp"], np.where(have, elp[np.arange(t), at], 0.0))
    if want_entropy:
        close(r["entropy"], e["entropy"], eh)
    assert np.array_equal(r["stats"][:, 0].cpu().numpy().astype(np.float64), e["stats"][:, 0])
    close(r["stats"][:, 1], e["stats"][:, 1], es)
    if topk:
        assert np.array_equal(r["top_id"].cpu().numpy(), e["top_id"])
        close(r["top_logp"], e["top_logp"], np.take_along_axis(elp, e["top_id"].astype(int), 1))
    return ids, r, e, (lp, es, elp, eh)


def check_grad(Q, z, zr, it, ids, r, e, b, dtype, which="both", out=None):
    t, v = zr.shape
    lp, es, elp, eh = b
    rng = np.random.default_rng(7)
    gl = rng.normal(size=t).astype(np.float32) if which != "entropy" else None
    gh = rng.normal(size=t).astype(np.float32) if which != "logp" else None
    up = lambda a: None if a is None else torch.from_numpy(a).to(DEV)
    dz = Q.quads_token_logprob_backward(z, up(ids) if gl is not None else None, r["stats"],
                                        r["entropy"] if gh is not None else None, up(gl), up(gh),
                                        it, out=out)
    torch.cuda.synchronize()
    assert dz.dtype == z.dtype and tuple(dz.shape) == (t, v)
    want = OH.token_logprob_grad(zr, ids, gl, gh, it)
    p = np.exp(lp)
    fin = np.where(np.isneginf(lp), 0.0, lp)
    ep = elp + 8 * U
    tol = np.zeros((t, v))
    if gl is not None:
        have = (ids >= 0) & (ids < v)
        a = np.where(have, np.abs(gl), 0.0)[:, None]
        hot = np.zeros((t, v))
        hot[np.arange(t), np.where(have, ids, 0)] = 1
        tol += a * (p * (ep + 4 * U) + hot * 4 * U + 2.0 ** -126)
    if gh is not None:
        a = np.abs(gh)[:, None]
        tol += a * 2.0 ** -126 * (np.abs(fin) + np.abs(e["entropy"])[:, None])
        tol += a * p * (np.abs(fin + e["entropy"][:, None]) * (ep + 4 * U) + elp + eh[:, None]
                    + 4 * U * (np.abs(fin) + e["entropy"][:, None]))
    tol = it * tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + TINY[dtype]
    close(dz, want, tol)
    return dz


SHAPES = [(1, 1, None), (1, 7, None), (7, 64, None), (6, 257, 264), (9, 1000, None),
          (6, 4097, None), (300, 515, None), (2, 16385, 16392), (33, 32768, None),
          (3, 50001, None), (2, 131072, None), (1, 300001, None),
          (2050, 515, 520), (2048, 2048, None), (4100, 37, None)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v,ld", SHAPES)
def test_logprob_and_gradient(Q, t, v, ld, dtype):
    it = 0.7 if v % 2 else 1.0
    z, zr = make(t, v, dtype, seed=v, ld=ld)
    ids, r, e, b = check_logprob(Q, z, zr, it, min(v, 20))
    check_grad(Q, z, zr, it, ids, r, e, b, dtype)
    if ld:                                                   # the padding is not written
        full = torch.full((t, ld), 3.0, dtype=z.dtype, device=DEV)
        check_grad(Q, z, zr, it, ids, r, e, b, dtype, out=full[:, :v])
        assert bool((full[:, v:] == 3.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v,masked", [(8, 1000, 0.5), (6, 20000, 0.999), (9, 70001, 0.3),
                                        (2100, 1001, 0.97)])
def test_masked_rows(Q, t, v, masked, dtype):
    """-inf entries, rows with fewer unmasked entries than alternatives, rows with none."""
    z, zr = make(t, v, dtype, seed=4, masked=masked, empty=(0, 5))
    ids, r, e, b = check_logprob(Q, z, zr, 1.3, 40)
    check_grad(Q, z, zr, 1.3, ids, r, e, b, dtype)


@pytest.mark.parametrize("which", ["logp", "entropy"])
def test_one_gradient_and_in_place(Q, which):
    z, zr = make(6, 3001, "f32", seed=8)
    ids, r, e, b = check_logprob(Q, z, zr, 1.0, 0)
    want = check_grad(Q, z, zr, 1.0, ids, r, e, b, "f32", which)
    got = check_grad(Q, z, zr, 1.0, ids, r, e, b, "f32", which, out=z)
    assert got.data_ptr() == z.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(1, 40000), (300, 40000), (3, 200000), (5, 30000), (600, 20000),
                                 (4096, 2000)])
@pytest.mark.parametrize("kind", ["constant", "two", "rising", "falling", "zeros", "late"])
def test_alternatives_in_hard_rows(Q, kind, t, v, dtype):
    """Ties by index (signed zeros are equal), ordered rows, the largest entries last."""
    i = torch.arange(v, dtype=torch.float32)
    row = {"constant": torch.full((v,), -3.25), "two": (i % 3 == 1).float(),
           "rising": i / 1024, "falling": -i / 1024,
           "zeros": torch.where(i % 2 == 0, 0.0, -0.0),
           "late": torch.where(i >= v - 100, 1.0 + i % 7, -5.0)}[kind]
    row = row.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    z = row.to(DEV).repeat(t, 1)
    zr = row.double().numpy()[None]
    r = Q.quads_token_logprob(z, None, 1.0, 128)
    torch.cuda.synchronize()
    e = OH.token_logprob(zr, None, 1.0, 128)
    _, es, elp, eh = errors_of(zr, 1.0)
    assert "logp" not in r
    assert np.array_equal(r["top_id"].cpu().numpy(), np.repeat(e["top_id"], t, 0))
    close(r["top_logp"], np.repeat(e["top_logp"], t, 0),
          np.take_along_axis(elp, e["top_id"].astype(int), 1))
    close(r["entropy"], np.repeat(e["entropy"], t), eh)


@pytest.mark.parametrize("k", [1, 2, 3, 31, 64, 65, 128])
def test_counts_of_alternatives(Q, k):
    for t, v in ((2, 9000), (2, k), (400, 2049), (4096, 2000)):
        z, zr = make(t, v, "bf16", seed=k, scale=1.0)
        check_logprob(Q, z, zr, 1.0, k, want_entropy=False)


def test_large_and_small_logits(Q):
    """Rows far from 0, and far apart entries: only differences to the maximum count."""
    z, zr = make(6, 5000, "f32", seed=2, scale=30.0)
    z += 1000.0
    zr = z.double().cpu().numpy()
    ids, r, e, b = check_logprob(Q, z, zr, 1.0, 8)
    check_grad(Q, z, zr, 1.0, ids, r, e, b, "f32")
    z = torch.full((6, 5000), -3.0e38, device=DEV)
    z[:, 17] = 3.0e38
    r = Q.quads_token_logprob(z, torch.full((6,), 17, dtype=torch.int32, device=DEV), 1.0, 2)
    assert r["logp"].tolist() == [0.0] * 6 and r["entropy"].tolist() == [0.0] * 6
    assert r["top_id"].tolist() == [[17, 0]] * 6


@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_are_not_numbers(Q, bad, dtype):
    """NaN or +inf spoils its own row only; alternatives stay distinct indices of the row."""
    for t, v in ((3, 700), (3, 70001), (300, 5000), (5, 30000), (2048, 1500)):
        z, zr = make(t, v, dtype, seed=3)
        z[1, v // 2] = bad
        ids = torch.zeros(t, dtype=torch.int32, device=DEV)
        r = Q.quads_token_logprob(z, ids, 1.0, 16)
        dz = Q.quads_token_logprob_backward(z, ids, r["stats"], r["entropy"],
                                            torch.ones(t, device=DEV), torch.ones(t, device=DEV))
        torch.cuda.synchronize()
        for key in ("logp", "entropy"):
            nan = torch.isnan(r[key]).tolist()
            assert nan[1] and sum(nan) == 1, key
        assert bool(torch.isnan(dz[1]).all())
        top = r["top_id"][1].tolist()
        assert len(set(top)) == 16 and min(top) >= 0 and max(top) < v
        keep = [i for i in range(t) if i != 1]
        e = OH.token_logprob(zr[keep], None, 1.0, 16)
        assert np.array_equal(r["top_id"][keep].cpu().numpy(), e["top_id"])
        assert not bool(torch.isnan(dz[keep]).any())


# ------------------------------------------------------------------ distillation --

def lists(zr, k, seed, it, renorm):
    """A teacher's list near the row's largest entries, with left-out and repeated ids."""
    t, v = zr.shape
    rng = np.random.default_rng(seed)
    noisy = np.where(np.isneginf(zr), -50.0, zr) + rng.normal(size=(t, v))
    t_id = np.argsort(-noisy, axis=1, kind="stable")[:, :k].astype(np.int32)
    if t_id.shape[1] < k:                                    # fewer entries than the list holds
        t_id = np.concatenate([t_id, np.full((t, k - v), -1, np.int32)], 1)
    t_val = np.sort(rng.normal(size=(t, k)), axis=1)[:, ::-1].astype(np.float32)
    if not renorm:
        t_val = (t_val - np.log(np.exp(t_val.astype(np.float64)).sum(1, keepdims=True))
                 - 0.1).astype(np.float32)
    if t > 5:
        t_id[1, k // 2:] = -1
        t_id[2, :] = v                                       # nothing in the list
        t_id[3, -1] = t_id[3, 0]
        t_val[4, k // 2:] = -np.inf
    return t_val, t_id


def distill_tolerance(zr, t_val, t_id, w, g, it, renorm, dtype, want_dz):
    """As above; q has the relative error 12 u (1 + |ln q|) + (topk + 8) u, and it enters the
    loss once as a factor and once as a logarithm."""
    t, v = zr.shape
    k = t_val.shape[1]
    lp, es, elp, _ = errors_of(zr, it)
    q, lq = OH.teacher(t_val, t_id, v, it, renorm)
    at = np.where(q > 0, t_id.astype(np.int64), 0)
    y = np.where(np.isneginf(t_val), 0.0, t_val.astype(np.float64))
    eq = (12 * (1 + np.where(q > 0, np.abs(lq), 0)) + (k + 8)
          + 6 * it * np.abs(y).max(1, keepdims=True)) * U
    lpi = np.take_along_axis(lp, at, 1)
    elpi = np.take_along_axis(elp, at, 1)
    with np.errstate(invalid="ignore"):
        part = np.where(q > 0, np.abs(lq) + np.abs(lpi), 0.0)
        tol = np.where(q > 0, q * (np.abs(lq - lpi) * eq + eq + elpi + (k + 4) * U * part), 0).sum(1)
    with np.errstate(invalid="ignore"):                      # (an infinite loss has no tolerance)
        tol_loss = np.abs(w) * (tol * (1 + U) + 4 * U * np.where(q > 0, q * part, 0).sum(1))
    p = np.exp(lp)
    big = q.sum(1, keepdims=True)
    tol = big * (p * (elp + 8 * U + eq.max(1, keepdims=True) + (k + 8) * U) + 2.0 ** -126)
    for i in range(t):
        for j in range(k):
            if q[i, j] > 0:
                tol[i, t_id[i, j]] += q[i, j] * (eq[i, j] + (k + 8) * U)
    by = np.abs(w * g * it)[:, None]
    tol_dz = by * tol * (1 + HALF[dtype]) + (HALF[dtype] + 4 * U) * np.abs(want_dz) + TINY[dtype]
    return tol_loss, tol_dz


def check_distill(Q, z, zr, k, it, renorm, dtype, seed=1, weights=True, out=None):
    t, v = zr.shape
    print(f"distill T={t} V={v} ld={z.stride(0)} {dtype} k={k} it={it} renorm={renorm}", flush=True)
    t_val, t_id = lists(zr, k, seed, it, renorm)
    rng = np.random.default_rng(seed + 1)
    w = rng.uniform(0.2, 2.0, t).astype(np.float32)
    g = rng.normal(size=t).astype(np.float32)
    w[rng.random(t) < 0.2] = 0.0
    if t > 5:
        w[1:5] = 1.5
    if not weights:
        w[:] = 1.0
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    args = (z, up(t_val), up(t_id))
    wt = up(w) if weights else None
    loss, stats = Q.quads_topk_distill(*args, wt, it, renorm)
    dz = Q.quads_topk_distill_backward(*args, stats, up(g), wt, it, renorm)
    loss2, dz2 = Q.quads_topk_distill_grad(*args, wt, it, renorm, out=out)
    torch.cuda.synchronize()
    want = OH.distill(zr, t_val, t_id, w, it, renorm)
    one = np.ones(t)
    for got, gg in ((dz, g.astype(np.float64)), (dz2, one)):
        want_dz = OH.distill_grad(zr, t_val, t_id, gg, w, it, renorm)
        tol, tol_dz = distill_tolerance(zr, t_val, t_id, w.astype(np.float64), gg, it, renorm,
                                        dtype, want_dz)
        close(got, want_dz, tol_dz)
    close(loss, want, tol)
    close(loss2, want, tol)
    m, s = OH.row_stats(zr, it)
    live = w != 0
    assert np.array_equal(stats[:, 0].cpu().numpy()[live].astype(np.float64), m[live])
    assert not stats.cpu().numpy()[~live].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,v,ld,k", [(1, 1, None, 1), (8, 9, None, 12), (7, 1000, 1008, 128),
                                      (300, 700, None, 5), (6, 4097, None, 16),
                                      (9, 32768, None, 64), (270, 16384, None, 20),
                                      (6, 50001, None, 20), (6, 131072, None, 64),
                                      (1, 300001, None, 3), (70, 140001, None, 2),
                                      (5, 131081, 131088, 9)])
def test_distill(Q, t, v, ld, k, renorm, dtype):
    z, zr = make(t, v, dtype, seed=v + k, ld=ld)
    check_distill(Q, z, zr, k, 0.6 if k % 2 else 1.0, renorm, dtype)


@pytest.mark.parametrize("t,v,ld,dtype,k", [
    (2100, 1, None, "bf16", 1), (2061, 7, None, "bf16", 3), (2050, 9, None, "f32", 2),
    (2049, 17, 24, "bf16", 17), (2100, 700, None, "bf16", 5), (2053, 1025, 1032, "f32", 70), (2048, 16383, None, "f32", 9),
    (1030, 32771, 32776, "bf16", 20), (1025, 16405, None, "f32", 4), (515, 65539, None, "bf16", 64),
    (4200, 1027, None, "f32", 11), (4097, 8200, None, "bf16", 20), (2049, 8203, 8204, "f32", 6),
    (513, 65537, None, "f32", 33), (512, 131081, None, "bf16", 128),
    (2048, 1024, None, "f32", 36), (2200, 2041, None, "bf16", 40), (2300, 4096, None, "f32", 8)])
def test_distill_many_rows(Q, t, v, ld, dtype, k):
    """Loss and gradient of many rows in one call: rows held by each size of work-group, rows
    longer than its registers, partial vectors at both ends, rows of weight 0 in between, lists
    with repeated and left-out ids.  Every seventh row against the oracle, all rows against the
    backward call's gradient (both are within the tolerance, so they differ by twice that)."""
    print(f"distill rows T={t} V={v} ld={ld} {dtype} k={k}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device=DEV).manual_seed(v)
    full = torch.full((t, ld or v), 7.5, dtype=dt, device=DEV)
    full[:, :v] = torch.randn((t, v), generator=g, device=DEV) * 2
    z = full[:, :v]
    z[3::50] = -float("inf")
    z[5::50, : v // 2] = -float("inf")
    t_val, t_id = (z.float() + torch.randn((t, v), generator=g, device=DEV)).topk(k, 1)
    t_val, t_id = t_val.clamp(min=-60.0), t_id.int()
    t_id[1::9, k // 2:] = -1
    t_id[2::9] = v
    t_id[4::9, -1] = t_id[4::9, 0]
    t_id[6::9, 0] = v - 1
    t_id[7::9, 0] = 0
    w = torch.rand(t, generator=g, device=DEV) + 0.5
    w[::5] = 0.0
    loss, dz = Q.quads_topk_distill_grad(z, t_val, t_id, w, 0.8)
    loss1, stats = Q.quads_topk_distill(z, t_val, t_id, w, 0.8)
    dz1 = Q.quads_topk_distill_backward(z, t_val, t_id, stats, torch.ones(t, device=DEV), w, 0.8)
    torch.cuda.synchronize()
    assert bool((full[:, v:] == 7.5).all())
    rows = np.unique(np.r_[np.arange(0, t, 7 if v < 20000 else 31), t - 1])
    zr = z[rows].double().cpu().numpy()
    tv, ti, wr = (a[rows].cpu().numpy() for a in (t_val, t_id, w))
    one = np.ones(len(rows))
    want = OH.distill(zr, tv, ti, wr, 0.8)
    want_dz = OH.distill_grad(zr, tv, ti, one, wr, 0.8)
    tol, tol_dz = distill_tolerance(zr, tv, ti, wr.astype(np.float64), one, 0.8, True, dtype,
                                    want_dz)
    for a, b in ((loss, dz), (loss1, dz1)):
        close(a[rows], want, tol)
        close(b[rows], want_dz, tol_dz)
    # fp32: p to about (6 |d| + V / 256 + 64) u from either side, |d| < 100; bf16: two half steps
    rel = 2 * (700 + v / 256) * U + (2 ** -7 if dtype == "bf16" else 0)
    scale = torch.maximum(dz.float().abs(), dz1.float().abs())
    diff = (dz.float() - dz1.float()).abs()
    at_list = torch.zeros((t, v), device=DEV)
    at_list.scatter_(1, t_id.clamp(0, v - 1).long(), 1.0)        # differences of near numbers
    assert bool((diff <= rel * (scale + 2.0 * at_list) + 2.0 ** -120).all())
    out = z.clone() if ld is None else z                         # in place
    _, dz2 = Q.quads_topk_distill_grad(out, t_val, t_id, w, 0.8, out=out)
    assert torch.equal(dz2, dz)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_masked_rows_and_in_place(Q, dtype):
    z, zr = make(9, 5003, dtype, seed=6, masked=0.4, empty=(6,))
    check_distill(Q, z, zr, 10, 1.0, True, dtype)
    z, zr = make(300, 5003, dtype, seed=7, masked=0.4)
    check_distill(Q, z, zr, 10, 1.0, True, dtype, weights=False, out=z)


def test_distill_weight_zero_reads_nothing(Q):
    """Rows of weight 0 may hold anything."""
    for t, v in ((4, 3000), (300, 3000), (4, 200000)):
        z, _ = make(t, v, "f32", seed=1)
        z[2] = float("nan")
        w = torch.ones(t, device=DEV)
        w[2] = 0.0
        tv = torch.zeros((t, 4), device=DEV)
        ti = torch.arange(4, dtype=torch.int32, device=DEV).repeat(t, 1)
        loss, dz = Q.quads_topk_distill_grad(z, tv, ti, w)
        loss2, stats = Q.quads_topk_distill(z, tv, ti, w)
        dz2 = Q.quads_topk_distill_backward(z, tv, ti, stats, torch.ones(t, device=DEV), w)
        for a, d in ((loss, dz), (loss2, dz2)):
            assert a[2].item() == 0.0 and not bool(d[2].any())
            assert bool(torch.isfinite(a).all()) and bool(torch.isfinite(d).all())


def test_distill_without_teacher_entries_has_no_gradient(Q):
    z, _ = make(3, 500, "f32")
    ti = torch.full((3, 7), -1, dtype=torch.int32, device=DEV)
    for renorm in (True, False):
        loss, dz = Q.quads_topk_distill_grad(z, torch.zeros((3, 7), device=DEV), ti, renorm=renorm)
        assert not bool(loss.any()) and not bool(dz.any())


# ------------------------------------------------------------------- how it is used --

def test_same_inputs_same_bits(Q):
    for t, v in ((1, 131072), (64, 50001), (300, 9000)):
        z, zr = make(t, v, "f32", seed=9)
        tv, ti = lists(zr, 16, 3, 1.0, True)
        tv, ti = torch.from_numpy(tv).to(DEV), torch.from_numpy(ti).to(DEV)
        runs = []
        for _ in range(2):
            r = Q.quads_token_logprob(z, ti[:, 0].contiguous(), 1.0, 50)
            loss, dz = Q.quads_topk_distill_grad(z, tv, ti)
            runs.append([*r.values(), loss, dz])
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_autograd_over_three_dimensions(Q, qat):
    z0, zr = make(12, 999, "bf16", seed=5)
    ids = tokens(zr, 2)
    z = z0.reshape(3, 4, 999).clone().requires_grad_()
    lp, h = qat.token_logprobs(z, torch.from_numpy(ids).to(DEV).reshape(3, 4), 0.8)
    (lp.sum() + 0.5 * h.sum()).backward()                    # broadcast (stride 0) gradients
    r = Q.quads_token_logprob(z0, torch.from_numpy(ids).to(DEV), 0.8)
    one = torch.ones(12, device=DEV)
    want = Q.quads_token_logprob_backward(z0, torch.from_numpy(ids).to(DEV), r["stats"],
                                          r["entropy"], one, 0.5 * one, 0.8)
    assert torch.equal(z.grad.reshape(12, 999), want) and torch.equal(lp.reshape(-1), r["logp"])
    z.grad = None
    lp, _ = qat.token_logprobs(z, torch.from_numpy(ids).to(DEV).reshape(3, 4), 0.8)
    lp.mean().backward()                                     # the entropy is not used
    want = Q.quads_token_logprob_backward(z0, torch.from_numpy(ids).to(DEV), r["stats"], None,
                                          one / 12, None, 0.8)
    assert torch.equal(z.grad.reshape(12, 999), want)
    tv, ti = lists(zr, 6, 3, 1.0, True)
    tv, ti = torch.from_numpy(tv).to(DEV), torch.from_numpy(ti).to(DEV)
    w = torch.linspace(0, 2, 12, device=DEV)
    z.grad = None
    loss = qat.distill_loss(z, tv.reshape(3, 4, 6), ti.reshape(3, 4, 6), w.reshape(3, 4))
    loss.sum().backward()
    loss2, stats = Q.quads_topk_distill(z0, tv, ti, w)
    want = Q.quads_topk_distill_backward(z0, tv, ti, stats, one, w)
    assert torch.equal(loss.reshape(-1), loss2) and torch.equal(z.grad.reshape(12, 999), want)


def test_gradients_against_differences(qat):
    """Central differences in fp64 of the oracle around the kernel's own gradient."""
    z, zr = make(4, 33, "f32", seed=11)
    ids = np.array([0, 5, 32, 7], np.int32)
    zt = z.clone().requires_grad_()
    lp, h = qat.token_logprobs(zt, torch.from_numpy(ids).to(DEV))
    (lp.sum() - 0.3 * h.sum()).backward()
    got = zt.grad.double().cpu().numpy()

    def f(a):
        r = OH.token_logprob(a, ids)
        return r["logp"].sum() - 0.3 * r["entropy"].sum()
    step = 1e-5
    for i in range(4):
        for j in range(33):
            a, b = zr.copy(), zr.copy()
            a[i, j] += step
            b[i, j] -= step
            # third derivatives below 10: step^2; fp64 sums of about 20: 1e-14 / step; fp32: 2e-6
            assert abs(got[i, j] - (f(a) - f(b)) / (2 * step)) < 3e-6


def test_strides_and_alignment(Q):
    """Transposed, offset and broadcast logits are copied; results equal the dense ones."""
    z, zr = make(6, 500, "f32", seed=1)
    ids = torch.from_numpy(tokens(zr, 1)).to(DEV)
    want = Q.quads_token_logprob(z, ids, 1.0, 5)
    wide = torch.zeros((6, 520), device=DEV)
    wide[:, 3:503] = z
    for view in (z.t().contiguous().t(), wide[:, 3:503]):
        got = Q.quads_token_logprob(view, ids, 1.0, 5)
        assert all(torch.equal(got[k], want[k]) for k in want)
    got = Q.quads_token_logprob(z[2:3].expand(6, 500), ids, 1.0, 5)
    assert torch.equal(got["top_id"], want["top_id"][2:3].expand(6, 5))
    got = Q.quads_token_logprob(z[1:], ids[1:], 1.0, 5)      # ids at an odd word
    assert all(torch.equal(got[k], want[k][1:]) for k in want)


def test_rows_far_apart(Q, qat):
    """The last positions of [B, S, V] logits: read where they are, a dense gradient."""
    z = make(12, 520, "f32", seed=4)[0].reshape(4, 3, 520)
    last, dense = z[:, -1], z[:, -1].contiguous()
    ids = torch.tensor([3, 519, -1, 0], dtype=torch.int32, device=DEV)
    tv, ti = torch.zeros((4, 2), device=DEV), torch.tensor([[1, 9]] * 4, dtype=torch.int32,
                                                           device=DEV)
    one = torch.ones(4, device=DEV)

    def calls(x):
        r = Q.quads_token_logprob(x, ids, 1.0, 5)
        loss, st = Q.quads_topk_distill(x, tv, ti)
        grads = [Q.quads_token_logprob_backward(x, ids, r["stats"], r["entropy"], one, one),
                 Q.quads_topk_distill_backward(x, tv, ti, st, one),
                 Q.quads_topk_distill_grad(x, tv, ti)[1]]
        assert all(g.is_contiguous() for g in grads)
        return [*r.values(), loss, st, *grads]
    assert all(torch.equal(a, b) for a, b in zip(calls(last), calls(dense)))
    out = torch.full_like(z, 7.0)                            # in place of rows far apart
    Q.quads_topk_distill_grad(last, tv, ti, out=out[:, -1])
    assert torch.equal(out[:, -1], Q.quads_topk_distill_grad(dense, tv, ti)[1])
    assert bool((out[:, :-1] == 7.0).all())
    full = z.clone().requires_grad_()
    lp, _ = qat.token_logprobs(full[:, -1], ids)
    lp.sum().backward()
    assert not bool(full.grad[:, :-1].any()) and bool(full.grad[0, -1].any())


def test_empty_calls(Q):
    z = torch.empty((0, 100), device=DEV)
    r = Q.quads_token_logprob(z, torch.empty(0, dtype=torch.int32, device=DEV), 1.0, 3)
    assert tuple(r["top_id"].shape) == (0, 3) and r["logp"].numel() == 0
    loss, dz = Q.quads_topk_distill_grad(z, torch.empty((0, 2), device=DEV),
                                         torch.empty((0, 2), dtype=torch.int32, device=DEV))
    assert loss.numel() == 0 and tuple(dz.shape) == (0, 100)


def test_refusals(Q):
    z, _ = make(4, 100, "f32")
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        Q.quads_token_logprob(z, ids.long())
    with pytest.raises(TypeError):
        Q.quads_token_logprob(z.half(), ids)
    with pytest.raises(ValueError):
        Q.quads_token_logprob(z, ids[:3])
    with pytest.raises(ValueError):
        Q.quads_token_logprob(z, ids.cpu())
    with pytest.raises(ValueError):
        Q.quads_token_logprob(z[0], ids)
    with pytest.raises(Q.QuadsError):
        Q.quads_token_logprob(z, ids, topk=101)
    with pytest.raises(Q.QuadsError):
        Q.quads_token_logprob(z, ids, topk=-1)
    with pytest.raises(Q.QuadsError):
        Q.quads_token_logprob(z, ids, inv_temp=0.0)
    with pytest.raises(Q.QuadsError):
        Q.quads_topk_distill(z, torch.zeros((4, 0), device=DEV),
                             torch.zeros((4, 0), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        Q.quads_topk_distill(z, torch.zeros((4, 3), device=DEV),
                             torch.zeros((4, 2), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        Q.quads_topk_distill_grad(z, torch.zeros((4, 3), device=DEV),
                                  torch.zeros((4, 3), dtype=torch.int32, device=DEV),
                                  out=torch.empty((4, 100), dtype=torch.bfloat16, device=DEV))


def test_other_stream(Q):
    z, zr = make(64, 50001, "f32", seed=2)
    ids = torch.from_numpy(tokens(zr, 1)).to(DEV)
    want = Q.quads_token_logprob(z, ids, 1.0, 10)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = Q.quads_token_logprob(z, ids, 1.0, 10)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_two_streams_at_once(Q):
    """Calls that overlap in time (each with a workspace of its own) do not meet."""
    zs = [make(40, 90001, "f32", seed=s)[0] for s in (3, 4)]
    ids = torch.zeros(40, dtype=torch.int32, device=DEV)
    want = [Q.quads_token_logprob(z, ids, 1.0, 30) for z in zs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = Q.quads_token_logprob(zs[i], ids, 1.0, 30)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in b)


def test_bit_patterns(Q):
    """bf16 as int16 or uint16 bits: the same results, gradients in the same type."""
    z, zr = make(6, 700, "bf16", seed=3)
    ids = torch.from_numpy(tokens(zr, 1)).to(DEV)
    one = torch.ones(6, device=DEV)
    want = Q.quads_token_logprob(z, ids, 1.0, 4)
    dz = Q.quads_token_logprob_backward(z, ids, want["stats"], want["entropy"], one, one)
    for dt in (torch.int16, torch.uint16):
        got = Q.quads_token_logprob(z.view(dt), ids, 1.0, 4)
        assert all(torch.equal(got[k], want[k]) for k in want)
        d = Q.quads_token_logprob_backward(z.view(dt), ids, want["stats"], want["entropy"], one,
                                           one)
        assert d.dtype == dt and torch.equal(d.view(torch.int16), dz.view(torch.int16))


@pytest.mark.parametrize("t,v", [(3, 70001), (300, 5000)])
def test_graph_replays(Q, t, v):
    """Captured forward, backward and distillation, replayed on new inputs with eager work
    between the replays."""
    z, zr = make(t, v, "f32", seed=2)
    ids = torch.from_numpy(tokens(zr, 1)).to(DEV)
    tv, ti = lists(zr, 8, 3, 1.0, True)
    tv, ti = torch.from_numpy(tv).to(DEV), torch.from_numpy(ti).to(DEV)
    g = torch.ones(t, device=DEV)

    def step(x):
        r = Q.quads_token_logprob(x, ids, 1.0, 8)
        dz = Q.quads_token_logprob_backward(x, ids, r["stats"], r["entropy"], g, g)
        loss, dd = Q.quads_topk_distill_grad(x, tv, ti)
        l2, st = Q.quads_topk_distill(x, tv, ti)
        return [*r.values(), dz, loss, dd, l2, Q.quads_topk_distill_backward(x, tv, ti, st, g)]
    step(z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(z)
    for seed in (20, 21, 22):
        new, _ = make(t, v, "f32", seed=seed)
        z.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in held]
        want = step(new)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_in_a_graph(Q, qat):
    """Forward and gradient of the autograd functions captured on leaves of their own, replayed
    on new logits with eager work between the replays."""
    t, v = 40, 9001
    ids = torch.arange(t, dtype=torch.int32, device=DEV)
    tv = torch.zeros((t, 4), device=DEV)
    ti = torch.randint(0, v, (t, 4), generator=torch.Generator().manual_seed(1)).int().to(DEV)
    g = torch.linspace(-1, 1, t, device=DEV)

    def step(x):
        lp, h = qat.token_logprobs(x, ids, 0.9)
        loss = qat.distill_loss(x, tv, ti)
        return [lp.detach(), h.detach(), loss.detach(),
                *torch.autograd.grad([lp, h, loss], [x], [g, 0.5 * g, g])]
    step(make(t, v, "f32", seed=1)[0].requires_grad_())
    z = make(t, v, "f32", seed=2)[0].requires_grad_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(z)
    for seed in (5, 6, 7):
        new = make(t, v, "f32", seed=seed)[0]
        with torch.no_grad():
            z.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in held]
        want = step(new.requires_grad_())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
