"""The norm at the ends of its range.

Where h r is below fp32's normal numbers (an eps far above the squares) it is off by at
most 3 * 2^-24 of the value and 2^-149 (|weight| + 1), as the header says: h r rounds to a
multiple of 2^-149, half of which is multiplied by the weight, and y itself to one."""

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q
from oracle import block as OB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("h", [7, 64, 1000, 2048, 20000, 40001])
def test_subnormal_rows(h):
    rng = np.random.default_rng(h)
    x = (rng.normal(size=(8, h)) * 10.0 ** rng.uniform(-30, 0, size=(8, 1))).astype(np.float32)
    for eps in (1e20, 1e60, 1e70):
        for by in (1.0, 1e30, 1e-10):
            w = (rng.normal(size=h) * by).astype(np.float32)
            y = Q.quads_rmsnorm(torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV), eps,
                                out_dtype=Q.OUT_F32)["y"].double().cpu().numpy()
            want, _ = OB.rmsnorm(x.astype(np.float64), w.astype(np.float64), eps)
            tol = 3 * 2.0 ** -24 * 1.01 * np.abs(want) + 2.0 ** -149 * (np.abs(w.astype(np.float64)) + 1)
            assert np.all(np.abs(y - want) <= tol)


@pytest.mark.parametrize("h", [32, 96, 2048, 20000])
def test_mx_codes_at_the_ends(h):
    """Blocks far below and above what scales reach, against the oracle; what is not finite."""
    rng = np.random.default_rng(h)
    for eps in (1e20, 1e60, 1e70, 1e-70):
        for by in (1e-40, 1e-20, 1.0, 1e37):
            x = (rng.normal(size=(3, h)).clip(-30, 30) * by).astype(np.float32)
            for wby in (1e-30, 1.0, 1e30):
                w = (rng.normal(size=h) * wby).astype(np.float32)
                r = Q.quads_rmsnorm(torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV), eps,
                                    out_dtype=Q.OUT_MX_FP8)
                codes, scales = OB.rmsnorm_mx(x.astype(np.float64), w.astype(np.float64), eps)
                assert np.array_equal(r["codes"].cpu().numpy(), codes)
                assert np.array_equal(r["scales"].cpu().numpy(), scales)
    x, w = torch.ones((1, h), device=DEV), torch.ones(h, device=DEV)
    w[5], w[6], w[7] = float("inf"), float("nan"), -float("inf")
    r = Q.quads_rmsnorm(x, w, out_dtype=Q.OUT_MX_FP8)
    codes = r["codes"][0].tolist()
    assert codes[5] == 126 and codes[6] & 127 == 127 and codes[7] == 254
    assert codes[:5] + codes[8:32] == [0] * 29
    # elsewhere y = 1 / sqrt(1 + 1e-6), just below 1: floor(log2 y) - 8 + 127 = 118
    assert r["scales"][0].tolist() == [254] + [118] * (h // 32 - 1)
