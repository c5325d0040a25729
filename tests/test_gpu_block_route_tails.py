"""The routing gradient of unlikely experts: dz_v = -p_v A, as exact in fp32 for an expert far
below the token's largest logit as for one near it.

One logit of a token is 0, the others lie so far below that z - m is exact and the sum over all
experts rounds to 1 (what is left of it is below 2 u of it).  Errors relative to dz_v: the
exponential 2 ulps (4 u); the forward call's sum (2 u), its division and the product g w (2 u);
here the sum (2 u), the division and the product with p_v (2 u): 12 u.  A power of two of a rounded
product z log2(e) would be off by up to half a step of that product, 44 u from z = -45 on."""

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q
from oracle import block as OB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [8, 60, 64, 128, 200, 512, 777, 1024, 4096])
def test_gradient_of_unlikely_experts(e, dtype):
    rng = np.random.default_rng(e)
    t = 97
    # sums of up to 4096 exp(-27) = 8e-9 are below 2 u = 1.2e-7; exp(-86) is above 2^-126
    z = torch.from_numpy(rng.uniform(-86.0, -27.0, size=(t, e)).astype(np.float32))
    z[torch.arange(t), torch.from_numpy(rng.integers(0, e, size=t))] = 0.0
    z[3] = torch.where(z[3] == 0.0, 0.0, -float("inf"))          # nothing else: gradient 0
    z = z.to(dtype).to(DEV)
    ids, w = Q.quads_moe_route(z, 1, renorm=False)
    g = torch.from_numpy(rng.normal(size=(t, 1)).astype(np.float32)).to(DEV)
    up = z.float()                                               # fp32 gradients of either type's values
    dz = Q.quads_moe_route_backward(up, ids, w, g, renorm=False).double().cpu().numpy()
    want = OB.route_grad(up.double().cpu().numpy(), ids.cpu().numpy(), g.double().cpu().numpy(), False)
    rest = np.ones((t, e), bool)
    np.put_along_axis(rest, ids.cpu().numpy().astype(np.int64), False, 1)   # a_i - p_i A cancels there
    err = np.abs(dz - want)[rest]
    size = np.abs(want)[rest]
    assert np.all(err <= 12 * U * size + 2.0 ** -126), float((err / np.maximum(size, 2.0 ** -126)).max() / U)
    # a bf16 gradient is that one, rounded: half a step more
    if dtype == torch.bfloat16:
        db = Q.quads_moe_route_backward(z, ids, w, g, renorm=False).double().cpu().numpy()
        assert np.all(np.abs(db - want)[rest] <= (2.0 ** -8 + 13 * U) * size + 2.0 ** -126)
    assert not dz[3].any()
