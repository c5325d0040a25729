"""The losses on the output head over the whole range of inverse temperatures
that they accept (0 < it <= 1e30), against oracle/head.py in fp64.

Logits are N(0, 4) / it, so that it z is ordinary; a teacher's values are of
every size, so that it t reaches far beyond what fp32 holds and its rounding to
fp32 (spacing 2^-23 of the value) beyond what exp spans.  The inverse
temperatures are fp32 numbers: it t is then exact in the oracle's fp64.

Tolerances (u = 2^-24, derivation of the logits' side in test_gpu_head): with
d = it (t - max t) formed in fp64 and rounded once,
  * e^d has the relative error (|d| + 2) u (its argument's rounding, and the
    exponential to 2 ulps) or is below 2^-126 and off by that much at most;
  * the list's sum s >= 1 has the mean of those, sum q |d| <= ln topk < 5, and
    topk + 8 additions (the wave's steps): (topk + 15) u; q = e^d / s then
    (|d| + topk + 18) u <= (|ln q| + topk + 23) u = eq;
  * ln q = d - ln s is off by elq = (topk + 18) u;
  * loss: every term q (ln q - ln p) by q (|ln q - ln p| eq + elq + err_lp),
    and topk + 8 roundings of the terms' sizes;
  * gradient by (Q p - q): Q p relative to itself by err_lp + 8 u + max eq +
    (topk + 8) u and by 2^-126, the entries' q by eq + (topk + 8) u, then half a
    step of the output's type."""

import numpy as np
import pytest
import torch

from oracle import head as OH
from test_gpu_head import HALF, TINY, U, check_grad, check_logprob, close, errors_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TEMPS = [1e-30, 1e-3, 1e9, 1e10, 1e11, 1e30]


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


def logits(t, v, dtype, it, seed):
    z = torch.randn((t, v), generator=torch.Generator().manual_seed(seed)) * 2 / it
    z = z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return z.to(DEV), z.double().numpy()


def lists(v, it):
    """[9, 6] values and ids: far apart, tied, near ones that the product with it rounds up and
    down, left-out entries above all others, masked entries, an empty list."""
    f = np.float32
    inf = f(np.inf)
    step = np.spacing(f(0.1))
    near = [f(0.1) - i * step for i in range(6)]
    small = [f(-0.7 * i / it) for i in range(6)]
    rows = [[-0.3, -1.3, -2.3, -0.30001, -5.0, -0.31], [3.1, 3.0, 3.1, 2.0, 1.0, 3.0], near, small,
            [1e30, 0.5, 0.25, 1e30, 0.5, -1.0], [3e9, 2e9, 1e9, -3e9, 0.0, 3e9],
            [-inf, -2.5, -inf, -2.5, -9.0, -2.75], [-inf] * 6, [-1e9, -1e9, -2e9, -3e9, -1e9, -inf]]
    t_val = np.array(rows, np.float32)
    t_id = np.stack([np.random.default_rng(r).permutation(v)[:6] for r in range(9)]).astype(np.int32)
    t_id[4, [0, 3]] = -1, v
    t_id[5, 5] = t_id[5, 0]
    return t_val, t_id


def tolerances(zr, t_val, t_id, by, it, dtype, want_dz):
    t, v = zr.shape
    k = t_val.shape[1]
    lp, _, elp, _ = errors_of(zr, it)
    q, lq = OH.teacher(t_val, t_id, v, it, True)
    lq = np.where(q > 0, lq, 0.0)
    at = np.where(q > 0, t_id.astype(np.int64), 0)
    eq = (np.abs(lq) + k + 23) * U
    lpi, elpi = np.take_along_axis(lp, at, 1), np.take_along_axis(elp, at, 1)
    part = np.abs(lq - lpi) * eq + (k + 18) * U + elpi + (k + 8) * U * (np.abs(lq) + np.abs(lpi))
    tol = (q * part).sum(1) + 2.0 ** -120
    p = np.exp(lp)
    dz = q.sum(1, keepdims=True) * (p * (elp + 8 * U + eq.max(1, keepdims=True) + (k + 8) * U)
                                    + 2.0 ** -126)
    for i in range(t):
        for j in range(k):
            if q[i, j] > 0:
                dz[i, t_id[i, j]] += q[i, j] * (eq[i, j] + (k + 8) * U) + 2.0 ** -126
    dz = np.abs(by)[:, None] * dz * (1 + HALF[dtype])
    return tol, dz + (HALF[dtype] + 4 * U) * np.abs(want_dz) + TINY[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("v", [300, 200001])
@pytest.mark.parametrize("it", TEMPS)
def test_teacher_at_every_temperature(Q, it, v, dtype):
    """q = softmax(it t) whatever it t is: one entry, or tied ones, where values are far apart."""
    it = float(np.float32(it))
    print(f"teacher V={v} {dtype} it={it}", flush=True)
    z, zr = logits(9, v, dtype, it, 5)
    t_val, t_id = lists(v, it)
    q, _ = OH.teacher(t_val, t_id, v, it, True)
    assert np.abs(q.sum(1) - (np.arange(9) != 7)).max() < 1e-12
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    args = (z, up(t_val), up(t_id))
    one = torch.ones(9, device=DEV)
    loss, stats = Q.quads_topk_distill(*args, None, it)
    dz = Q.quads_topk_distill_backward(*args, stats, one, None, it)
    loss2, dz2 = Q.quads_topk_distill_grad(*args, None, it)
    torch.cuda.synchronize()
    want = OH.distill(zr, t_val, t_id, None, it)
    want_dz = OH.distill_grad(zr, t_val, t_id, np.ones(9), None, it)
    tol, tol_dz = tolerances(zr, t_val, t_id, np.full(9, it), it, dtype, want_dz)
    for a, b in ((loss, dz), (loss2, dz2)):
        close(a, want, tol)
        close(b, want_dz, tol_dz)


def test_many_rows_and_autograd(Q):
    """The row-by-row form and the autograd function on the same lists."""
    from nvfp4_w4a4_quantized_act_amd import qat
    it, v = float(np.float32(1e10)), 1000
    t_val, t_id = lists(v, it)
    z, zr = logits(9, v, "f32", it, 6)
    n = 300
    rows = np.arange(n) % 9
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    zt = z[torch.from_numpy(rows).to(DEV)].reshape(30, 10, v).requires_grad_()
    tv, ti = up(t_val[rows]).reshape(30, 10, 6), up(t_id[rows]).reshape(30, 10, 6)
    loss = qat.distill_loss(zt, tv, ti, inv_temp=it)
    loss.sum().backward()
    loss2, dz2 = Q.quads_topk_distill_grad(zt.detach().reshape(n, v), tv.reshape(n, 6),
                                           ti.reshape(n, 6), None, it)
    torch.cuda.synchronize()
    want = OH.distill(zr, t_val, t_id, None, it)
    want_dz = OH.distill_grad(zr, t_val, t_id, np.ones(9), None, it)
    tol, tol_dz = tolerances(zr, t_val, t_id, np.full(9, it), it, "f32", want_dz)
    for a, b in ((loss.reshape(-1), zt.grad.reshape(n, v)), (loss2, dz2)):
        close(a, want[rows], tol[rows])
        close(b, want_dz[rows], tol_dz[rows])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(6, 300), (3, 70001), (2050, 515)])
@pytest.mark.parametrize("it", TEMPS)
def test_logprob_at_every_temperature(Q, it, t, v, dtype):
    it = float(np.float32(it))
    z, zr = logits(t, v, dtype, it, 7)
    ids, r, e, b = check_logprob(Q, z, zr, it, 20)
    check_grad(Q, z, zr, it, ids, r, e, b, dtype)
