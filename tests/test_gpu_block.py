"""The layer around the experts on the GPU against oracle/block.py in fp64: the
residual's addition with the norm, routing, tokens in expert order and back, and
their gradients.

Tolerances, derived (u = 2^-24, half a step of fp32; HALF of the output's type):
  * h is one fp32 sum and one rounding: the oracle's bits.
  * y in fp32 or bf16: r = 1 / sqrt(..) comes from fp64 and is rounded (u), h r and
    (h r) w round once each: 3 u |y|, then the output's half step (none more for
    fp32); 2^-126 where h r is subnormal.
  * MX FP8: y is formed in fp64, about 2^-51 off, and a code or a scale differs only
    where y is that close to a border: the oracle's bits.
  * dh: n = h r (2 u), w g (u), c = mean n w g: its terms carry u and its own rounding
    u |c|, its fp64 sum nothing; the fused n c + w g rounds once, the product with r
    twice (r's own u), the sum with g_sum once.  With M = mean |n w g|:
    r u (|w g| + |n| M + 4 |n c| + |w g - n c|) + 2 u |r (w g - n c)| + u |dh|.
  * dweight: terms g n with n's 2 u, one rounding per addition, at most T of them (any
    order of T terms): (T + 3) u sum |g n|.
  * a routing term e^(z - m): z - m rounds (u |d|), its product with log2 e and that
    constant again (2 u |d|), the exponential 2 ulps (4 u); a sum meets at most
    n = min(E / 8, 64) + 12 + topk additions; one division (2 ulps).  err_w =
    w (3 u |d| + 4 u + [the terms' mean of the same] + (n + 4) u) + 2^-126.
  * a routing gradient: products a_i = g_i w_i and their sums (topk + 3 roundings), p
    with err_w: sum |a| p (err_p / p + (topk + 6) u), and at the chosen experts
    |a_i| (err_w / w + (topk + 6) u) more, |w_i| A's likewise.
  * sort: a copy.  unsort: one fused multiply-add a slot, topk u sum |w y|.  dy: one
    product, u |dy|.  dw: products of two fp32 numbers in fused sums; a thread adds up
    at most H / 64 + 16 of them before at most 8 more additions: (H / 64 + 24) u sum |g y|.
"""

import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import moe as OM

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"
TINY = 2.0 ** -126
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(t, h, dtype, seed, by=1.0, ld=None):
    """[t, h] on the GPU (a view with row stride ld, other values between the rows) and its
    values."""
    g = torch.Generator().manual_seed(seed)
    full = torch.full((t, ld or h), 7.5, dtype=TYPES[dtype])
    full[:, :h] = (torch.randn((t, h), generator=g) * by).to(TYPES[dtype])
    v = full.to(DEV)[:, :h]
    return v, f64(v)


def close(got, want, tol):
    got = f64(got)
    assert got.shape == want.shape
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True)
    err = np.abs(got[fin] - want[fin])
    tol = np.broadcast_to(tol, want.shape)[fin]
    bad = ~(err <= tol)
    assert not bad.any(), (float(err[bad].max()), float((err / np.maximum(tol, 1e-300)).max()),
                           int(bad.sum()), np.argwhere(bad)[:4].tolist())


# ------------------------------------------------------------------------------------- norm --

def norm_inputs(t, h, xt, rt, wt, seed, ldx=None, ldr=None, by=1.0):
    x, xr = rows(t, h, xt, seed, by, ldx)
    res, rr = rows(t, h, rt, seed + 1, 2.0 * by, ldr) if rt else (None, None)
    w, wr = (None, None)
    if wt:
        w = (1.0 + 0.3 * torch.randn(h, generator=torch.Generator().manual_seed(seed + 2)))
        w = w.to(TYPES[wt]).to(DEV)
        wr = f64(w)
    want = xr if rt is None else OB.add(xr, rr, rt == "bf16")
    return x, res, w, want, wr


def check_norm(Q, t, h, xt, rt, wt, out, seed=0, eps=EPS, **kw):
    print(f"norm T={t} H={h} x={xt} res={rt} w={wt} out={out} {kw}", flush=True)
    x, res, w, hr, wr = norm_inputs(t, h, xt, rt, wt, seed, **kw)
    code = {"f32": Q.OUT_F32, "bf16": Q.OUT_BF16, "fp8": Q.OUT_MX_FP8}[out]
    r = Q.quads_rmsnorm(x, w, eps, res, code, want_amax=out == "bf16")
    torch.cuda.synchronize()
    if rt:
        assert r["sum"].dtype == res.dtype and np.array_equal(f64(r["sum"]), hr)
    y, _ = OB.rmsnorm(hr, wr, eps)
    if out == "fp8":
        codes, scales = OB.rmsnorm_mx(hr, wr, eps)
        assert np.array_equal(r["scales"].cpu().numpy(), scales)
        assert np.array_equal(r["codes"].cpu().numpy(), codes)
    else:
        assert r["y"].dtype == TYPES[out]
        close(r["y"], y, (3 * U + (HALF[out] if out == "bf16" else 0)) * (1 + 2 ** -7) * np.abs(y)
              + TINY)
    if out == "bf16":
        top = r["y"].view(torch.int16).to(torch.int32).bitwise_and(0x7FFF).max().item()
        assert r["amax_part"].shape[0] == Q.quads_rmsnorm_amax_groups(t, h)
        assert r["amax_part"].max().item() == top and r["amax_part"].min().item() >= 0
    return x, res, w, hr, wr, r


WIDTHS = (1, 2, 7, 8, 9, 31, 33, 64, 100, 127, 128, 129, 257, 512, 513, 1000, 1024, 1031, 2047, 2048,
          2056, 4095, 4096, 4104, 5001, 8191, 8192, 8200, 16384, 16385, 20000, 40007)


@pytest.mark.parametrize("h", WIDTHS)
def test_norm_widths(Q, h):
    t = 5 if h > 9000 else 67
    check_norm(Q, t, h, "bf16", "bf16", "bf16", "bf16", seed=h)
    check_norm(Q, t, h, "f32", None, "f32", "f32", seed=h)


@pytest.mark.parametrize("h", [32, 64, 96, 128, 160, 512, 544, 1024, 2016, 2048, 4096, 4128, 8192, 8224,
                               16384, 20000, 40032])
def test_norm_mx_widths(Q, h):
    check_norm(Q, 4 if h > 9000 else 37, h, "bf16", "bf16", "bf16", "fp8", seed=h)
    check_norm(Q, 3, h, "f32", "bf16", "f32", "fp8", seed=h + 1)


@pytest.mark.parametrize("out", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("rt", [None, "f32", "bf16"])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_norm_types(Q, xt, rt, out):
    for h in (96, 2048):
        check_norm(Q, 13, h, xt, rt, "f32" if xt == "bf16" else "bf16", out, seed=3)
        check_norm(Q, 13, h, xt, rt, None, out, seed=4)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 15, 16, 17, 64, 255, 1025, 4099])
def test_norm_numbers_of_rows(Q, t):
    for h in (64, 800, 2048):
        check_norm(Q, t, h, "bf16", "bf16", "bf16", "bf16", seed=t)
    check_norm(Q, t, 288, "f32", "bf16", "f32", "fp8", seed=t)


@pytest.mark.parametrize("ldx,ldr", [(264, 256), (257, 263), (256, 1000), (4099, 301)])
def test_norm_row_strides(Q, ldx, ldr):
    for out in ("bf16", "f32", "fp8"):
        check_norm(Q, 19, 256, "bf16", "bf16", "bf16", out, ldx=ldx, ldr=ldr)
        check_norm(Q, 19, 256, "f32", "bf16", "f32", out, ldx=ldx, ldr=ldr)
    check_norm(Q, 19, 251, "bf16", "f32", "bf16", "bf16", ldx=ldx, ldr=ldr)


@pytest.mark.parametrize("by", [1e-30, 1e-12, 1e12, 1e30])
def test_norm_magnitudes(Q, by):
    """Squares below and beyond fp32's range."""
    for out in ("f32", "bf16", "fp8"):
        check_norm(Q, 6, 512, "f32", "f32", "f32", out, by=by, eps=1e-5)
        check_norm(Q, 6, 512, "bf16", "bf16", "bf16", out, by=by, eps=1e-70)


def test_norm_zero_rows_and_blocks(Q):
    x = torch.zeros((3, 128), dtype=torch.bfloat16, device=DEV)
    x[1, 40] = -1.5
    x[2] = -0.0
    r = Q.quads_rmsnorm(x, out_dtype=Q.OUT_MX_FP8)
    codes, scales = OB.rmsnorm_mx(f64(x), None, EPS)
    assert np.array_equal(r["codes"].cpu().numpy(), codes)
    assert np.array_equal(r["scales"].cpu().numpy(), scales) and scales[0].tolist() == [0] * 4
    for eps in (1e-6, 1e-70):
        for out in (Q.OUT_F32, Q.OUT_BF16):
            assert not f64(Q.quads_rmsnorm(x, eps=eps, out_dtype=out)["y"][[0, 2]]).any()
        dx, _, dw = Q.quads_rmsnorm_backward(x[[0, 2]], x[[0, 2]], torch.ones(128, device=DEV), eps)
        assert not f64(dx).any() and not f64(dw).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("h", [64, 2048, 20000])
def test_norm_not_finite(Q, h, bad):
    """Only the row that holds it shows it; an infinity's row is 0 elsewhere."""
    for out in (Q.OUT_F32, Q.OUT_BF16, Q.OUT_MX_FP8):
        x, _ = rows(9, h, "f32", 5)
        want = Q.quads_rmsnorm(x, out_dtype=out)
        x[4, 33] = bad
        got = Q.quads_rmsnorm(x, out_dtype=out)
        for k in want:
            a, b = want[k], got[k]
            keep = [i for i in range(9) if i != 4]
            assert torch.equal(a[keep], b[keep])
        y = got["codes"].view(torch.float8_e4m3fn).float() if out == Q.OUT_MX_FP8 else got["y"]
        y = f64(y[4])
        assert np.isnan(y[33])
        rest = np.delete(y, 33)
        assert np.isnan(rest).all() if np.isnan(bad) else not rest.any()


@pytest.mark.parametrize("h", [5, 61, 64, 130, 1001, 2048, 2049, 5001, 8191, 16384, 16385, 40000, 40001])
def test_norm_in_place(Q, h):
    """sum over the residual, y over x (through the C ABI)."""
    lib, t = Q.lib(), 7
    for sum_at in ("residual", "x", "new"):
        x, res, w, hr, wr = norm_inputs(t, h, "bf16", "bf16", "bf16", 3)
        y = torch.empty_like(x)
        total = {"residual": res, "x": x, "new": torch.empty_like(x)}[sum_at]
        if sum_at == "residual":
            y = x
        elif sum_at == "x":
            y = res
        torch.cuda.synchronize()
        assert lib.quads_rmsnorm(x.data_ptr(), 1, t, h, h, res.data_ptr(), 1, h, w.data_ptr(), 1,
                                 EPS, total.data_ptr(), y.data_ptr(), 1, None, None, 0, None) == 0
        torch.cuda.synchronize()
        want, _ = OB.rmsnorm(hr, wr, EPS)
        assert np.array_equal(f64(total), hr)
        close(y, want, (3 * U + HALF["bf16"]) * 1.01 * np.abs(want) + TINY)


def test_norm_without_the_sum(Q):
    for h in (256, 40000):
        x, res, w, hr, wr = norm_inputs(9, h, "f32", "bf16", "f32", 8)
        a = Q.quads_rmsnorm(x, w, EPS, res, want_sum=False)
        assert set(a) == {"y"}
        assert torch.equal(a["y"], Q.quads_rmsnorm(x, w, EPS, res)["y"])


def check_norm_grad(Q, t, h, gt, ht, wt, seed=0, xt=None, gs=True, ldh=None, eps=EPS, by=1.0):
    print(f"norm gradient T={t} H={h} g={gt} h={ht} w={wt} x={xt} g_sum={gs} ldh={ldh}", flush=True)
    x, _, w, hr, wr = norm_inputs(t, h, ht, None, wt, seed, ldx=ldh, by=by)
    g, gr = rows(t, h, gt, seed + 5, 0.1)
    s, sr = rows(t, h, ht, seed + 6, 0.1) if gs else (None, None)
    dx, dres, dw = Q.quads_rmsnorm_backward(g, x, w, eps, s, TYPES[xt] if xt else None)
    torch.cuda.synchronize()
    dh, dwr = OB.rmsnorm_grad(gr, hr, wr, eps, sr)
    r = OB.rmsnorm(hr, None, eps)[1]
    n, wg = hr * r, gr * (1.0 if wr is None else wr)
    c = (n * wg).mean(1, keepdims=True)
    m = np.abs(n * wg).mean(1, keepdims=True)
    tol = r * U * (np.abs(wg) + np.abs(n) * m + 4 * np.abs(n * c) + np.abs(wg - n * c))
    tol = (tol + 2 * U * np.abs(r * (wg - n * c)) + U * np.abs(dh)) * 1.01 + TINY * (1 + r)
    close(dx, dh, tol * (1 + HALF[xt or ht]) + HALF[xt or ht] * np.abs(dh))
    if xt and xt != ht:
        assert dx.dtype == TYPES[xt] and dres.dtype == TYPES[ht]
        close(dres, dh, tol * (1 + HALF[ht]) + HALF[ht] * np.abs(dh))
    else:
        assert dres is dx
    if wt:
        tw = (t + 3) * U * np.abs(gr * n).sum(0) * 1.01 + TINY
        close(dw, dwr, tw * (1 + HALF[wt]) + HALF[wt] * np.abs(dwr))
    else:
        assert dw is None
    return dx, dw


@pytest.mark.parametrize("h", WIDTHS)
def test_norm_grad_widths(Q, h):
    t = 5 if h > 9000 else 67
    check_norm_grad(Q, t, h, "bf16", "bf16", "bf16", seed=h)
    check_norm_grad(Q, t, h, "f32", "f32", "f32", seed=h, gs=False)


@pytest.mark.parametrize("ht", ["f32", "bf16"])
@pytest.mark.parametrize("gt", ["f32", "bf16"])
def test_norm_grad_types(Q, gt, ht):
    for wt in ("f32", "bf16", None):
        for xt in ("f32", "bf16"):
            for h in (100, 2048, 9000):
                check_norm_grad(Q, 21, h, gt, ht, wt, xt=xt)


@pytest.mark.parametrize("t", [1, 2, 3, 7, 8, 9, 63, 64, 257, 1030])
def test_norm_grad_numbers_of_rows(Q, t):
    for h in (64, 800, 2048):
        check_norm_grad(Q, t, h, "bf16", "bf16", "f32", seed=t, gs=t % 2 == 0)
    check_norm_grad(Q, t, 9001, "f32", "f32", "f32", seed=t)


def test_norm_grad_row_strides_and_magnitudes(Q):
    for h, ldh in ((256, 264), (251, 257), (256, 4099), (9000, 9003)):
        check_norm_grad(Q, 11, h, "bf16", "bf16", "bf16", ldh=ldh)
        check_norm_grad(Q, 11, h, "f32", "f32", "f32", ldh=ldh)
    for by in (1e-12, 1e12, 1e18):
        check_norm_grad(Q, 6, 512, "f32", "f32", "f32", by=by, gs=False)


def test_norm_grad_of_no_rows(Q):
    x = torch.zeros((0, 40), device=DEV)
    dx, _, dw = Q.quads_rmsnorm_backward(x, x, torch.ones(40, device=DEV))
    assert dx.shape == (0, 40) and dw.tolist() == [0.0] * 40
    assert Q.quads_rmsnorm(x)["y"].shape == (0, 40)


@pytest.mark.parametrize("h", [5, 61, 64, 130, 1001, 2048, 2049, 5001, 8191, 12000, 12001, 20001])
def test_norm_grad_in_place(Q, h):
    lib, t = Q.lib(), 70
    for at in ("g", "g_sum"):
        x, _, w, hr, wr = norm_inputs(t, h, "bf16", None, "bf16", 3)
        g, gr = rows(t, h, "bf16", 4)
        s, sr = rows(t, h, "bf16", 5)
        want = Q.quads_rmsnorm_backward(g, x, w, EPS, s)
        nws = lib.quads_rmsnorm_backward_ws(t, h, 1)
        ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=DEV)
        dw = torch.empty_like(w)
        dx = g if at == "g" else s
        torch.cuda.synchronize()
        assert lib.quads_rmsnorm_backward(g.data_ptr(), 1, x.data_ptr(), 1, t, h, h, w.data_ptr(), 1,
                                          EPS, s.data_ptr(), dx.data_ptr(), 1, None, dw.data_ptr(),
                                          ws.data_ptr(), nws, None) == 0
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[2])


def test_norm_grad_writes_both(Q):
    """dx and dres of one type, and of two, dres over g_sum (through the C ABI)."""
    lib, t = Q.lib(), 20
    for h in (100, 2048, 20000):
        for dt in ("bf16", "f32"):
            x, _, w, _, _ = norm_inputs(t, h, "bf16", None, "f32", 3)
            g, _ = rows(t, h, "f32", 4)
            s, _ = rows(t, h, "bf16", 5)
            want = Q.quads_rmsnorm_backward(g, x, w, EPS, s, TYPES[dt])
            nws = lib.quads_rmsnorm_backward_ws(t, h, 0)
            ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=DEV)
            dx = torch.empty((t, h), dtype=TYPES[dt], device=DEV)
            torch.cuda.synchronize()
            assert lib.quads_rmsnorm_backward(g.data_ptr(), 0, x.data_ptr(), 1, t, h, h, w.data_ptr(), 0,
                                              EPS, s.data_ptr(), dx.data_ptr(), 1 if dt == "bf16" else 0,
                                              s.data_ptr(), None, ws.data_ptr(), nws, None) == 0
            torch.cuda.synchronize()
            assert torch.equal(dx, want[0]) and torch.equal(s, want[1])


def test_norm_grad_not_finite(Q):
    for h in (256, 9000):
        x, _ = rows(9, h, "f32", 5)
        g, _ = rows(9, h, "f32", 6)
        w = torch.ones(h, device=DEV)
        a = Q.quads_rmsnorm_backward(g, x, w)
        g[4, 33] = float("nan")
        b = Q.quads_rmsnorm_backward(g, x, w)
        keep = [i for i in range(9) if i != 4]
        assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][4]).all()
        other = [i for i in range(h) if i != 33]
        assert torch.equal(a[2][other], b[2][other]) and torch.isnan(b[2][33])


# ---------------------------------------------------------------------------------- routing --

def logits(t, e, dtype, seed, masked=0.0, empty=(), ld=None, by=1.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((t, e), generator=g) * by
    if masked:
        z[torch.rand((t, e), generator=g) < masked] = -float("inf")
    for i in empty:
        z[i] = -float("inf")
    full = torch.full((t, ld or e), 99.0, dtype=TYPES[dtype])
    full[:, :e] = z.to(TYPES[dtype])
    v = full.to(DEV)[:, :e]
    return v, f64(v)


def route_errors(z, ids, topk, renorm):
    """(err of each expert's p, err of the chosen weights) of the derivation."""
    t, e = z.shape
    m = z.max(1, keepdims=True)
    d = np.where(np.isneginf(z), 0.0, np.abs(z - np.where(np.isneginf(m), 0.0, m)))
    term = 3 * U * np.minimum(d, 110) + 4 * U
    n = min(e / 8, 64) + 12 + topk
    p = OB.softmax(z)
    ep = p * (term + (p * term).sum(1, keepdims=True) + (n + 4) * U) + TINY
    at = ids.astype(np.int64)
    if not renorm:
        return ep, np.take_along_axis(ep, at, 1)
    w = OB.softmax(np.take_along_axis(z, at, 1))
    tk = np.take_along_axis(term, at, 1)
    return ep, w * (tk + (w * tk).sum(1, keepdims=True) + (n + 4) * U) + TINY


def check_route(Q, t, e, topk, dtype, renorm, seed=0, grad=True, **kw):
    print(f"route T={t} E={e} topk={topk} {dtype} renorm={renorm} {kw}", flush=True)
    z, zr = logits(t, e, dtype, seed, **kw)
    ids, w = Q.quads_moe_route(z, topk, renorm)
    torch.cuda.synchronize()
    eids, ew = OB.route(zr, topk, renorm)
    assert np.array_equal(ids.cpu().numpy(), eids)
    ep, err = route_errors(zr, eids, topk, renorm)
    close(w, ew, err)
    if not grad:
        return
    g, gr = rows(t, topk, "f32", seed + 1)
    dz = Q.quads_moe_route_backward(z, ids, w, g, renorm)
    torch.cuda.synchronize()
    assert dz.dtype == z.dtype and dz.is_contiguous()
    want = OB.route_grad(zr, eids, gr, renorm)
    p = OB.softmax(zr)
    a = np.abs(gr * ew)
    ea = np.abs(gr) * err + (topk + 6) * U * a
    tol = np.zeros((t, e))
    if renorm:
        np.put_along_axis(tol, eids.astype(np.int64),
                          ea + ew * ea.sum(1, keepdims=True) + (err + 6 * U * ew) * a.sum(1, keepdims=True),
                          1)
    else:
        tol = p * ea.sum(1, keepdims=True) + (ep + (topk + 6) * U * p) * a.sum(1, keepdims=True)
        add = np.zeros((t, e))
        np.put_along_axis(add, eids.astype(np.int64), ea, 1)
        tol = tol + add
    close(dz, want, (tol + U * np.abs(want)) * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + TINY)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("e", [1, 2, 3, 8, 16, 17, 32, 60, 64, 65, 100, 128, 129, 160, 256, 257, 384,
                               512, 513, 777, 1024, 1025, 2048, 4096])
def test_route_numbers_of_experts(Q, e, renorm):
    for topk in sorted({1, min(e, 2), min(e, 8), min(e, 64)}):
        check_route(Q, 19, e, topk, "f32", renorm, seed=e)
        check_route(Q, 19, e, topk, "bf16", renorm, seed=e)       # many equal logits


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 15, 16, 17, 33, 1000, 5003])
def test_route_numbers_of_tokens(Q, t):
    check_route(Q, t, 128, 8, "bf16", True, seed=t)
    check_route(Q, t, 60, 4, "f32", False, seed=t)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("e", [8, 64, 100, 500, 3000])
def test_route_masks(Q, e, renorm):
    """Masked experts, fewer than topk left, nothing left; a mask of the type's lowest value."""
    for dtype in ("f32", "bf16"):
        check_route(Q, 40, e, 6, dtype, renorm, masked=0.5, empty=(3, 17))
        check_route(Q, 40, e, 6, dtype, renorm, masked=1.0 - 3.0 / e, empty=(0,))
    z, _ = logits(6, e, "f32", 4)
    z[2, :e - 2] = torch.finfo(torch.float32).min
    zr = f64(z)
    ids, w = Q.quads_moe_route(z, 4, renorm)
    eids, ew = OB.route(zr, 4, renorm)
    assert np.array_equal(ids.cpu().numpy(), eids)
    close(w, ew, route_errors(zr, eids, 4, renorm)[1])


def test_route_row_stride_and_equal_logits(Q):
    for ld in (101, 128, 1000):
        check_route(Q, 23, 100, 8, "bf16", True, ld=ld)
        check_route(Q, 23, 100, 8, "f32", False, ld=ld)
    for e in (16, 128, 700):
        z = torch.zeros((3, e), device=DEV)
        z[0, ::2] = -0.0
        ids, w = Q.quads_moe_route(z, 8)
        assert ids.tolist() == [list(range(8))] * 3 and torch.equal(w, torch.full_like(w, 0.125))


@pytest.mark.parametrize("e", [8, 64, 65, 128, 200, 256, 512, 700, 2000])
def test_route_logits_one_step_apart(Q, e):
    """Neighbouring fp32 numbers, of both signs, with equal ones among them."""
    for seed, base in ((0, 1.0), (1, -2.5), (2, 1e-38), (3, -3e38)):
        rng = np.random.default_rng(seed)
        v = np.full((41, e), np.float32(base)).view(np.int32) + rng.integers(-40, 40, size=(41, e)).astype(np.int32)
        z = torch.from_numpy(v.view(np.float32)).to(DEV)
        z[5, : e // 2] = z[5, e // 2: 2 * (e // 2)]
        z[6:9] = torch.randn(3, e, device=DEV)
        for topk in (1, 5, min(e, 8)):
            ids, w = Q.quads_moe_route(z, topk, True)
            eids, ew = OB.route(f64(z), topk, True)
            assert np.array_equal(ids.cpu().numpy(), eids)
            close(w, ew, route_errors(f64(z), eids, topk, True)[1])


@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf")])
def test_route_not_finite(Q, bad):
    for e in (16, 100, 1000):
        for renorm in (False, True):
            z, _ = logits(5, e, "f32", 2)
            ids0, w0 = Q.quads_moe_route(z, 8, renorm)
            z[2, 7] = bad
            z[2, 9] = bad
            ids, w = Q.quads_moe_route(z, 8, renorm)
            keep = [0, 1, 3, 4]
            assert torch.equal(ids[keep], ids0[keep]) and torch.equal(w[keep], w0[keep])
            got = ids[2].tolist()
            assert len(set(got)) == 8 and min(got) >= 0 and max(got) < e
            assert torch.isnan(w[2]).any()


def test_route_backward_takes_ids_as_given(Q):
    """Repeated ids add up; ids outside [0, E) are left out; dlogits over the logits."""
    z, zr = logits(4, 20, "f32", 1)
    ids = torch.tensor([[3, 3, 19], [0, -1, 20], [5, 6, 7], [2 ** 31 - 1, -2 ** 31, 1]],
                       dtype=torch.int32, device=DEV)
    have = ((ids >= 0) & (ids < 20)).cpu().numpy()
    at = np.where(have, ids.cpu().numpy(), 0)
    p = OB.softmax(zr)
    w = np.where(have, np.take_along_axis(p, at, 1), 0.0)
    g = np.random.default_rng(0).normal(size=(4, 3))
    a = g * w
    want = -p * a.sum(1, keepdims=True)
    for t in range(4):
        for i in range(3):
            want[t, at[t, i]] += a[t, i]
    up = lambda v: torch.from_numpy(v.astype(np.float32)).to(DEV)
    wt = up(np.where(have, w, 77.0))
    gt = up(g)
    dz = Q.quads_moe_route_backward(z, ids, wt, gt, False)
    torch.cuda.synchronize()
    assert np.allclose(f64(dz), want, rtol=0, atol=1e-5)
    assert Q.lib().quads_moe_route_backward(z.data_ptr(), 0, 4, 20, 20, ids.data_ptr(), wt.data_ptr(),
                                            gt.data_ptr(), 3, 0, z.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(z, dz)


# ---------------------------------------------------------------------------------- sorting --

def placement(t, topk, e, seed, capacity=0, left_out=0.0):
    """(pos [t * topk], rows): by expert, with room for `capacity` rows each."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(-rng.normal(size=(t, e)), axis=1)[:, :topk]
    _, _, pos = OM.pack_routes(ids, e)
    n = t * topk
    if capacity:
        first = np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=e))])[:-1]
        flat = ids.reshape(-1)
        at = pos - first[flat]
        pos = np.where(at < capacity, flat * capacity + at, -1)
        n = e * capacity
    if left_out:
        drop = rng.random(pos.shape) < left_out
        pos = np.where(drop, rng.choice([-1, n, -2 ** 31, 2 ** 31 - 1], size=pos.shape), pos)
    return pos.astype(np.int32), n


def check_sort(Q, t, h, topk, e, dtype, gt, seed=0, capacity=0, left_out=0.0, weighted=True, ld=None):
    print(f"sort T={t} H={h} topk={topk} E={e} {dtype} g={gt} capacity={capacity} out={left_out} "
          f"w={weighted} ld={ld}", flush=True)
    posn, n = placement(t, topk, e, seed, capacity, left_out)
    given = n if capacity or left_out else None
    pos = torch.from_numpy(posn).to(DEV)
    x, xr = rows(t, h, dtype, seed + 1, ld=ld)
    y, yr = rows(n, h, dtype, seed + 2)
    g, gr = rows(t, h, gt, seed + 3)
    w = wr = None
    if weighted:
        w = torch.rand((t, topk), generator=torch.Generator().manual_seed(seed)).to(DEV)
        wr = f64(w)
    xs = Q.quads_moe_sort(x, pos, topk, given)
    outs = {k: Q.quads_moe_unsort(y, pos, topk, w, c)
            for k, c in (("f32", Q.OUT_F32), ("bf16", Q.OUT_BF16))}
    dy, dw = Q.quads_moe_unsort_backward(g, y, pos, topk, w, given)
    torch.cuda.synchronize()
    assert xs.dtype == x.dtype and np.array_equal(f64(xs), OB.sort(xr, posn, topk, n))
    want, size = OB.unsort(yr, posn, topk, wr)
    for k in outs:
        tol = topk * U * size * (1 + HALF[k]) + TINY
        close(outs[k], want, tol + (HALF[k] * np.abs(want) if k == "bf16" else 0))
    edy, edw, esz = OB.unsort_grad(gr, yr, posn, topk, wr)
    close(dy, edy, U * np.abs(edy) * (1 + HALF[dtype]) + HALF[dtype] * np.abs(edy) + TINY)
    if weighted:
        close(dw, edw, (h / 64 + 24) * U * esz + TINY)
    else:
        assert dw is None


@pytest.mark.parametrize("h", [1, 2, 5, 8, 15, 16, 63, 64, 65, 128, 250, 512, 513, 1000, 1001, 1024, 2048,
                               2049, 4096, 4100, 8192, 12000])
def test_sort_widths(Q, h):
    check_sort(Q, 37, h, 3, 8, "bf16", "bf16", seed=h)
    check_sort(Q, 21, h, 2, 5, "f32", "f32", seed=h, capacity=7)


@pytest.mark.parametrize("topk", [1, 2, 3, 4, 5, 7, 8, 9, 16, 33, 64])
def test_sort_slots(Q, topk):
    for weighted in (True, False):
        check_sort(Q, 11, 300, topk, max(topk, 4), "bf16", "f32", seed=topk, weighted=weighted)
        check_sort(Q, 11, 2048, topk, 64, "f32", "bf16", seed=topk, weighted=weighted, left_out=0.3)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 64, 257, 1500])
def test_sort_numbers_of_tokens(Q, t):
    check_sort(Q, t, 256, 4, 16, "bf16", "bf16", seed=t)
    check_sort(Q, t, 72, 8, 8, "bf16", "f32", seed=t, left_out=1.0)
    check_sort(Q, t, 2048, 8, 128, "bf16", "bf16", seed=t, capacity=1 + t // 16)


def test_sort_row_stride(Q):
    for ld in (130, 131, 4000):
        check_sort(Q, 9, 129, 2, 4, "bf16", "bf16", ld=ld)
        check_sort(Q, 9, 128, 2, 4, "f32", "f32", ld=ld)


def test_sort_leaves_other_rows_and_nan_weights(Q):
    """C ABI: rows without a slot stay as they were; a left-out slot's weight is not used, and a
    NaN in a row without a slot goes nowhere."""
    lib, t, h, k, n = Q.lib(), 3, 40, 2, 8
    posn = np.array([7, 0, -1, 3, 100, 5], np.int32)
    pos = torch.from_numpy(posn).to(DEV)
    x, xr = rows(t, h, "f32", 0)
    y, yr = rows(n, h, "f32", 1)
    y[1] = float("nan")
    out = torch.full((n, h), 9.0, device=DEV)
    dy = torch.full((n, h), 9.0, device=DEV)
    w = torch.tensor([[1.0, 2.0], [float("nan"), 3.0], [float("inf"), 4.0]], device=DEV)
    dw = torch.empty_like(w)
    o = torch.empty_like(x)
    assert lib.quads_moe_sort(x.data_ptr(), 0, t, h, h, pos.data_ptr(), k, n, 0, out.data_ptr(), None,
                              0, None) == 0
    assert lib.quads_moe_unsort(y.data_ptr(), 0, n, pos.data_ptr(), w.data_ptr(), t, k, h, o.data_ptr(), 0,
                                None) == 0
    assert lib.quads_moe_unsort_backward(x.data_ptr(), 0, y.data_ptr(), 0, n, pos.data_ptr(),
                                         w.data_ptr(), t, k, h, 0, dy.data_ptr(), dw.data_ptr(), None, 0,
                                         None) == 0
    torch.cuda.synchronize()
    assert np.array_equal(f64(out), OB.sort(xr, posn, k, n, 9.0))
    want, size = OB.unsort(yr, posn, k, np.array([[1, 2], [0, 3], [0, 4.0]]))
    close(o, want, 2 * U * size + TINY)
    assert f64(dy)[[1, 2, 4, 6]].tolist() == [[9.0] * h] * 4
    assert f64(dw)[1, 0] == 0 and f64(dw)[2, 0] == 0 and np.isfinite(f64(dw)).all()
    for h in (20, 900):                                          # a gradient that is not finite
        g = torch.full((t, h), float("inf"), device=DEV)
        g[:, 3] = float("nan")
        y = torch.ones((n, h), device=DEV)
        dy, dw = Q.quads_moe_unsort_backward(g, y, pos, k, w, rows=n)
        assert f64(dw)[1, 0] == 0 and f64(dw)[2, 0] == 0 and np.isnan(f64(dw)[0]).all()
        assert not f64(dy)[[1, 2, 4, 6]].any()


@pytest.mark.parametrize("before", ["slots", "negative", "rows", "ones"])
@pytest.mark.parametrize("h,room", [(1, 16), (12, 15), (250, 15), (2049, 15), (7, 300000), (100, 30000),
                                    (250, 15000), (1001, 3000), (9000, 300)])
def test_rows_without_a_slot_become_zero(Q, h, room, before):
    """Whatever the workspace held: slots of the call (as an earlier call leaves them), numbers that
    are none, row numbers.  `room` rows for each of 16 experts: outputs of 1 kB to 170 MB."""
    lib, t, k = Q.lib(), 70, 3
    posn, n = placement(t, k, 16, 1, capacity=room, left_out=0.2)
    pos = torch.from_numpy(posn).to(DEV)
    at = pos.long()
    have = (at >= 0) & (at < n)
    full = torch.zeros(n, dtype=torch.bool, device=DEV)
    full[at[have]] = True
    for dtype in ("bf16", "f32"):
        code = 1 if dtype == "bf16" else 0
        x, _ = rows(t, h, dtype, 0)
        w = torch.rand((t, k), device=DEV)
        y = torch.randn((n, h), device=DEV).to(TYPES[dtype])
        nws = lib.quads_moe_sort_ws(n, h, code, 1)
        size = n * h * y.element_size()
        assert nws == 0 if size <= 64 << 20 else nws >= 4 * n
        held = {"slots": torch.arange(nws // 4) % (t * k), "negative": torch.full((nws // 4,), -5),
                "rows": torch.arange(nws // 4), "ones": torch.full((nws // 4,), 2 ** 31 - 1)}[before]
        for call in ("sort", "gradient"):
            ws = held.int().to(DEV)
            out = torch.full((n, h), 9.0, dtype=TYPES[dtype], device=DEV)
            torch.cuda.synchronize()
            if call == "sort":
                assert lib.quads_moe_sort(x.data_ptr(), code, t, h, h, pos.data_ptr(), k, n, 1,
                                          out.data_ptr(), ws.data_ptr() if nws else None, nws, None) == 0
                want = x.repeat_interleave(k, 0)
            else:
                dw = torch.empty_like(w)
                assert lib.quads_moe_unsort_backward(x.data_ptr(), code, y.data_ptr(), code, n,
                                                     pos.data_ptr(), w.data_ptr(), t, k, h, 1, out.data_ptr(),
                                                     dw.data_ptr(), ws.data_ptr() if nws else None, nws,
                                                     None) == 0
                want = (x.float()[:, None] * w[..., None]).reshape(t * k, h).to(x.dtype)
            torch.cuda.synchronize()
            assert not out[~full].any()
            assert torch.equal(out[at[have]], want[have])


def test_more_rows_than_slots(Q):
    """Most rows without a slot; no tokens at all."""
    x, xr = rows(5, 300, "bf16", 0)
    pos = torch.tensor([199999, 3, 70001, 0, 12345], dtype=torch.int32, device=DEV)
    xs = Q.quads_moe_sort(x, pos, 1, rows=200000)
    got = torch.nonzero(xs.float().abs().sum(1))[:, 0].tolist()
    assert got == [0, 3, 12345, 70001, 199999]
    assert torch.equal(xs[pos.long()], x)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    for h in (300, 30000):                                       # 0.8 and 84 MB
        y = torch.ones((0, h), device=DEV)
        torch.full((700, h), 5.0, device=DEV)                    # the next allocation's memory
        assert not Q.quads_moe_sort(y, none, 2, rows=700).any()
        dy, dw = Q.quads_moe_unsort_backward(y, torch.ones((700, h), device=DEV), none, 2,
                                             torch.ones((0, 2), device=DEV), rows=700)
        assert dy.shape == (700, h) and not dy.any() and dw.shape == (0, 2)


def test_unsort_backward_over_y(Q):
    lib, t, h, k = Q.lib(), 50, 700, 4
    posn, n = placement(t, k, 16, 0)
    pos = torch.from_numpy(posn).to(DEV)
    g, _ = rows(t, h, "bf16", 1)
    y, _ = rows(n, h, "bf16", 2)
    w = torch.rand((t, k), device=DEV)
    dy, dw = Q.quads_moe_unsort_backward(g, y, pos, k, w)
    dw2 = torch.empty_like(dw)
    assert lib.quads_moe_unsort_backward(g.data_ptr(), 1, y.data_ptr(), 1, n, pos.data_ptr(),
                                         w.data_ptr(), t, k, h, 0, y.data_ptr(), dw2.data_ptr(), None, 0,
                                         None) == 0
    torch.cuda.synchronize()
    assert torch.equal(y, dy) and torch.equal(dw, dw2)


def test_sort_of_more_tokens_than_a_launch_has(Q):
    t, h = 2 ** 21 + 5, 16
    g = torch.Generator(device=DEV).manual_seed(0)
    pos = torch.randperm(t, generator=g, device=DEV, dtype=torch.int32)
    x = torch.randn((t, h), generator=g, device=DEV).bfloat16()
    at = pos.long()
    xs = Q.quads_moe_sort(x, pos, 1)
    assert torch.equal(xs[at], x)
    w = torch.rand((t, 1), generator=g, device=DEV)
    out = Q.quads_moe_unsort(xs, pos, 1, w)
    assert torch.equal(out, x.float() * w)                          # one product, rounded once
    dy, dw = Q.quads_moe_unsort_backward(out, xs, pos, 1, w)
    assert torch.equal(dy[at], (out * w).bfloat16())
    want = (out.double() * x.double()).sum(1, keepdim=True)
    assert ((dw.double() - want).abs() <= 25 * U * (out.double() * x.double()).abs().sum(1, keepdim=True)
            + TINY).all()


def test_sort_of_nothing(Q):
    z = torch.zeros((0, 16), device=DEV)
    pos = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert Q.quads_moe_sort(z, pos, 2).shape == (0, 16)
    assert f64(Q.quads_moe_sort(z, pos, 2, rows=3)).tolist() == [[0.0] * 16] * 3
    assert Q.quads_moe_unsort(z, pos, 2).shape == (0, 16)
    out = torch.full((4,), -1, dtype=torch.int32, device=DEV)       # every slot left out, no rows
    assert f64(Q.quads_moe_unsort(z, out, 2)).tolist() == [[0.0] * 16] * 2


def test_calls_are_refused(Q):
    x = torch.zeros((4, 32), device=DEV)
    pos = torch.zeros(8, dtype=torch.int32, device=DEV)
    w = torch.zeros((4, 2), device=DEV)
    with pytest.raises(ValueError, match="residual must have the shape"):
        Q.quads_rmsnorm(x, residual=x[:3])
    with pytest.raises(ValueError, match="weight must have the shape"):
        Q.quads_rmsnorm(x, torch.zeros(31, device=DEV))
    with pytest.raises(TypeError):
        Q.quads_rmsnorm(x.half())
    with pytest.raises(TypeError):
        Q.quads_rmsnorm_backward(x, x, g_sum=x.bfloat16())
    with pytest.raises(Q.QuadsError):
        Q.quads_rmsnorm(x[:, :24].contiguous(), out_dtype=Q.OUT_MX_FP8)
    with pytest.raises(Q.QuadsError):
        Q.quads_rmsnorm(x, eps=0.0)
    with pytest.raises(Q.QuadsError):
        Q.quads_rmsnorm(x, out_dtype=Q.OUT_F32, want_amax=True)
    for k in (0, 33):
        with pytest.raises(ValueError):
            Q.quads_moe_route(x, k)
    with pytest.raises(TypeError):
        Q.quads_moe_sort(x, pos.long(), 2)
    with pytest.raises(ValueError):
        Q.quads_moe_sort(x, pos[:7], 2)
    with pytest.raises(ValueError):
        Q.quads_moe_sort(x, pos[:6], 2)
    with pytest.raises(ValueError):
        Q.quads_moe_unsort(x, pos, 2, w[:3])
    with pytest.raises(ValueError):
        Q.quads_moe_unsort_backward(x, x, pos, 2, w)               # y has 4 rows, not 8
    with pytest.raises(ValueError, match="must be on"):
        Q.quads_moe_sort(x, pos.cpu(), 2)
