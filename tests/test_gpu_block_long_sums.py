"""The norm weight's gradient over many rows: its fp32 chains are bounded, whatever T.

A thread adds up at most 64 rows before at most 127 sums of a work-group's parts are joined in
fp32; the rest is fp64.  dweight_j = sum_t g n: n = h r carries 2 u (here 1 u: h = 1), each fused
addition of the chain one u of the sum so far, all terms of one sign: (64 + 127 + 3) u of the sum,
(64 + 3) u where one row at a time fills a work-group.  The terms are so chosen that every addition
from some sum on rounds the same way, by nearly half a step: one chain over all of a work-group's
rows would be off by more than that."""

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def one_way(n):
    """v in [1/2, 1), exact in fp32: sums of v from 2^n on lose nearly half a step each."""
    return 0.5 + 2.0 ** (n - 24) - 2.0 ** -23


def chain(v, n):
    """n terms v added up in fp32."""
    s = np.float32(0)
    for _ in range(n):
        s = np.float32(s + np.float32(v))
    return float(s)


def test_the_terms_do_that():
    """On the CPU: 64 terms stay within 64 u, 512 or 1024 of them not within the bound."""
    for n, length, most in ((7, 512, 67), (8, 1024, 194)):
        v = one_way(n)
        assert float(np.float32(v)) == v
        assert abs(chain(v, 64) - 64 * v) <= 64 * U * 64 * v
        assert abs(chain(v, length) - length * v) > most * U * length * v


@pytest.mark.parametrize("t,h,bits,most", [
    (1 << 17, 8192, 7, 67),                  # a work-group of 1024 threads a row: 512 rows in turn each
    ((1 << 18) + 3, 8200, 7, 67),            # sixteen channels a thread, an odd width
    (1 << 18, 16392, 7, 67),                 # rows that are read twice: 512 runs of 512 rows
    ((1 << 25) + 5, 64, 8, 194),             # 128 rows at once, 1024 times
    (1 << 25, 8, 8, 194),
])
def test_many_rows(t, h, bits, most):
    print(f"norm gradient T={t} H={h}", flush=True)
    v = one_way(bits)
    x = torch.ones((t, h), dtype=torch.bfloat16, device=DEV)
    eps = 1.0 / (v * v) - 1.0                                    # r = v to fp64's rounding, v in fp32
    w = torch.ones(h, device=DEV)
    dx, _, dw = Q.quads_rmsnorm_backward(x, x, w, eps)
    torch.cuda.synchronize()
    want = t * v
    assert float((dw.double() - want).abs().max()) <= most * U * want
    del dx
    # and with terms of both signs, against fp64: the same bound of the sum of magnitudes
    g = torch.randn((1 << 12, h), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()
    for a in range(0, t, 1 << 12):
        x[a:a + (1 << 12)] = g[:min(1 << 12, t - a)]
    dx, _, dw = Q.quads_rmsnorm_backward(x, x, w, 1e-6)
    torch.cuda.synchronize()
    gd = g.double()
    n = gd * torch.rsqrt((gd * gd).mean(1, keepdim=True) + 1e-6)
    times = torch.full((1 << 12, 1), t >> 12, dtype=torch.float64, device=DEV)
    times[:t & 0xFFF] += 1
    want, size = (times * gd * n).sum(0), (times * (gd * n).abs()).sum(0)
    assert bool(((dw.double() - want).abs() <= (most + 1) * U * size).all())
    assert torch.equal(dx[-3:], Q.quads_rmsnorm_backward(x[-3:].clone(), x[-3:].clone(), w, 1e-6)[0])
