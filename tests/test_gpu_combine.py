"""The MoE combine at the ends of its range: numbers of slots, of tokens and of channels, equal
to the way back with weights bit for bit, and to fp64 within its topk roundings."""

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def inputs(t, k, n, dtype, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    y = torch.randn((t * k, n), generator=g, device=DEV).to(dtype)
    pos = torch.randperm(t * k, generator=g, device=DEV).int()
    return y, pos, torch.rand((t, k), generator=g, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,k,n", [(1, 1, 8), (1, 8, 2048), (3, 65, 40), (7, 100, 1000), (64, 8, 2048), (300, 2, 72),
                                   (33, 9, 264), (1000, 4, 136), (257, 7, 8200), (2, 3, 40000), (2100, 8, 2048)])
def test_combine_sizes(t, k, n, dtype):
    print(f"combine T={t} topk={k} N={n} {dtype}", flush=True)
    y, pos, w = inputs(t, k, n, dtype)
    code = Q.OUT_BF16 if dtype == torch.bfloat16 else Q.OUT_F32
    out = Q.quads_moe_combine(y, pos, w, y_dtype=code)
    torch.cuda.synchronize()
    v = y.double()[pos.long()].view(t, k, n) * w.double()[..., None]
    want, size = v.sum(1), v.abs().sum(1)
    assert bool(((out.double() - want).abs() <= k * U * size + 2.0 ** -149).all())
    if k <= 64:
        assert torch.equal(out, Q.quads_moe_unsort(y, pos, k, w))


def test_combine_of_many_tokens_and_of_long_rows():
    """More tokens than one launch has, and rows of more channels."""
    t = 2 ** 21 + 3
    y, pos, w = inputs(t, 2, 8, torch.bfloat16)
    out = Q.quads_moe_combine(y, pos, w, y_dtype=Q.OUT_BF16)
    v = y.double()[pos.long()].view(t, 2, 8) * w.double()[..., None]
    assert bool(((out.double() - v.sum(1)).abs() <= 2 * U * v.abs().sum(1) + 2.0 ** -149).all())
    for n in (2 ** 24 - 8, 2 ** 24, 2 ** 24 + 8, 2 ** 25 + 520):
        print(f"combine N={n}", flush=True)
        y, pos, w = inputs(2, 2, n, torch.bfloat16)
        out = Q.quads_moe_combine(y, pos, w, y_dtype=Q.OUT_BF16)
        v = y.double()[pos.long()].view(2, 2, n) * w.double()[..., None]
        assert bool(((out.double() - v.sum(1)).abs() <= 2 * U * v.abs().sum(1) + 2.0 ** -149).all())


def test_only_the_tokens_own_slots_add():
    """A sum that rounds to -0 stays -0, whatever the number of slots; a token's NaN is its own."""
    for k in (1, 3, 8, 9):
        y = torch.full((4 * k, 16), 1e-30, device=DEV)
        pos = torch.arange(4 * k, dtype=torch.int32, device=DEV)
        w = torch.full((4, k), -1e-30, device=DEV)
        y[k] = float("nan")
        for out in (Q.quads_moe_combine(y, pos, w), Q.quads_moe_unsort(y, pos, k, w)):
            o = out.cpu().numpy()
            assert np.isnan(o[1]).all()
            o = np.delete(o, 1, axis=0)
            assert not o.any() and np.signbit(o).all()
