"""The longest chains of additions in the distillation's row sums, with data
whose roundings all go one way.

A bf16 row of up to 16 vectors of 8 entries per thread is summed by 64 threads
(up to 8192 entries) or 128 (up to 16384), so a term meets up to 16 * 8 additions
in its thread, 8 more for a partial vector, and 12 in the two wave sums: n = 148.
With u = 2^-24 the rest is test_gpu_head's derivation: terms off by 6 u |d| + 4 u,
the logarithm by 4 u |s|, so err_s = (6 |d| q_d + n + 8 + 4 |s|) u, where only the
terms' share q_d of the sum carries 6 |d|.

Here the first entry of each thread is 0 and all others are -16.75: e^-16.75 is
0.89 u, less than half a step of the sum, so that each of the thread's other 127
terms is lost, and the sum is 113 u too small."""

import numpy as np
import pytest
import torch

from oracle import head as OH

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
N = 16 * 8 + 8 + 12


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


@pytest.mark.parametrize("t,v", [(70, 8192), (2048, 8192), (70, 16384)])
def test_longest_chains(Q, t, v):
    print(f"chains T={t} V={v}", flush=True)
    row = np.full(v, -16.75)
    row[: v // 16: 8] = 0.0                                    # entry 0 of each thread's first vector
    z = torch.from_numpy(row).to(DEV).bfloat16().repeat(t, 1)
    tv = torch.zeros((t, 2), device=DEV)
    ti = torch.tensor([[0, v - 1]], dtype=torch.int32, device=DEV).repeat(t, 1)
    loss, stats = Q.quads_topk_distill(z, tv, ti)
    dz = Q.quads_topk_distill_backward(z, tv, ti, stats, torch.ones(t, device=DEV))
    loss2, dz2 = Q.quads_topk_distill_grad(z, tv, ti)
    torch.cuda.synchronize()
    one, ids, val = row[None], np.array([[0, v - 1]]), np.zeros((1, 2))
    _, s = OH.row_stats(one, 1.0)
    p = np.exp(OH.log_softmax(one, 1.0))[0]
    share = p[row < 0].sum()
    es = (6 * 16.75 * share + N + 8 + 4 * s[0]) * U
    assert np.abs(stats[:, 1].double().cpu().numpy() - s).max() <= es
    # loss: q = 1/2 twice (exact), ln q to 8 u, ln p to es and the last rounding
    want = OH.distill(one, val, ids)[0]
    el = es + (8 + 2 * (want + 1)) * U
    # gradient p - q: p to es, its own exponential and product; half a step of bf16
    want_dz = OH.distill_grad(one, val, ids, np.ones(1))[0]
    ez = p * (es + (6 * np.abs(row) + 12) * U) + 8 * U * np.abs(want_dz) + 2.0 ** -8 * np.abs(want_dz)
    for a, b in ((loss, dz), (loss2, dz2)):
        assert np.abs(a.double().cpu().numpy() - want).max() <= el
        assert (np.abs(b.double().cpu().numpy() - want_dz) <= ez + U * 2.0 ** -8).all()
