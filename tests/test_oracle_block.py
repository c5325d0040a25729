"""Pins of oracle/block.py (CPU): against scalar loops, hand values and central
differences of its own outputs, with masked experts, ties, empty rows and slots
that are left out."""

import math

import numpy as np
import pytest

from oracle import block as OB
from oracle import formats as F
from oracle import moe as OM


def _differences(f, v, h=1e-6):
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        a, b = v.copy(), v.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


def test_bf16_round_matches_formats():
    v = np.random.default_rng(0).normal(size=4096).astype(np.float32)
    v[:5] = (1.00390625, 1.01171875, -1.00390625, 3.4e38, 1e-40)   # ties to even; overflow; tiny
    got = OB.bf16_round(v)
    assert got[:3].tolist() == [1.0, 1.015625, -1.0] and np.isinf(got[3])
    v[3] = 0.0
    assert np.array_equal(OB.bf16_round(v), F.bf16_to_f64(F.f64_to_bf16_rne(v.astype(np.float64))))
    assert np.isnan(OB.bf16_round([np.nan])[0])


def test_norm_by_hand():
    y, r = OB.rmsnorm([[3.0, -4.0]], [2.0, 0.5], 0.0 + 1e-300)
    assert r[0, 0] == pytest.approx(1 / math.sqrt(12.5))
    assert y[0].tolist() == pytest.approx([6 / math.sqrt(12.5), -2 / math.sqrt(12.5)])
    assert OB.rmsnorm(np.zeros((1, 4)), None, 1e-6)[0].tolist() == [[0.0] * 4]
    assert OB.add([1.0], [2.0 ** -9], True)[0] == 1.0            # rounded to the residual's type
    assert OB.add([1.0], [2.0 ** -9], False)[0] == 1.0 + 2.0 ** -9


def test_norm_mx_scales_by_the_largest():
    h = np.zeros((1, 64))
    h[0, 3], h[0, 40] = 8.0, -0.25
    codes, scales = OB.rmsnorm_mx(h, None, 1e-6)
    y = OB.rmsnorm(h, None, 1e-6)[0]
    e = np.floor(np.log2(np.abs(y[0, [3, 40]]))) - 8
    assert scales[0].tolist() == (e + 127).tolist()
    got = F.e4m3_decode(codes[0]) * np.exp2(np.repeat(e, 32))
    assert np.all(np.abs(got - y[0]) <= np.abs(y[0]) / 8)        # one step where 448 cuts off


@pytest.mark.parametrize("weighted", [True, False])
def test_norm_gradient_is_the_difference(weighted):
    rng = np.random.default_rng(1)
    h, g, gs = rng.normal(size=(3, 3, 7))
    w = rng.normal(size=7) if weighted else None
    dh, dw = OB.rmsnorm_grad(g, h, w, 0.1, gs)
    f = lambda a: (g * OB.rmsnorm(a, w, 0.1)[0]).sum() + (gs * a).sum()
    assert np.allclose(dh, _differences(f, h), atol=1e-8)
    if weighted:
        assert np.allclose(dw, _differences(lambda a: (g * OB.rmsnorm(h, a, 0.1)[0]).sum(), w),
                           atol=1e-8)


def test_route_ties_masks_and_empty():
    inf = np.inf
    z = np.array([[1.0, 3.0, 3.0, 0.0], [-inf, 2.0, -inf, -inf], [-inf] * 4, [0.0, -0.0, 0.0, -1.0]])
    ids, w = OB.route(z, 3, True)
    assert ids.tolist() == [[1, 2, 0], [1, 0, 2], [0, 1, 2], [0, 1, 2]]
    assert w[1].tolist() == [1.0, 0.0, 0.0] and not w[2].any()
    assert w[3].tolist() == pytest.approx([1 / 3] * 3)
    _, w = OB.route(z, 2, False)
    e = [math.exp(v - 3) for v in (1, 3, 3, 0)]
    assert w[0].tolist() == pytest.approx([1 / sum(e)] * 2)
    for renorm in (False, True):
        assert not OB.route_grad(z, ids, np.ones((4, 3)), renorm)[2].any()


@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference(renorm):
    rng = np.random.default_rng(2)
    z, g = rng.normal(size=(4, 6)) * 2, rng.normal(size=(4, 3))
    ids, _ = OB.route(z, 3, renorm)
    f = lambda a: (g * OB.route(a, 3, renorm)[1]).sum()
    assert np.allclose(OB.route_grad(z, ids, g, renorm), _differences(f, z), atol=1e-8)


def test_sorting_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    pos = [2, 0, -1, 1]                                          # token 1's first slot left out
    assert OB.sort(x, pos, 2, 4, 9.0).tolist() == [[1, 2], [3, 4], [1, 2], [9, 9]]
    y = np.array([[1.0, 1.0], [2.0, 0.0], [4.0, 8.0], [100.0, 100.0]])
    w = np.array([[0.5, 2.0], [7.0, 3.0]])
    assert OB.unsort(y, pos, 2, w)[0].tolist() == [[4.0, 6.0], [6.0, 0.0]]
    assert OB.unsort(y, pos, 2)[0].tolist() == [[5.0, 9.0], [2.0, 0.0]]
    dy, dw, _ = OB.unsort_grad([[1.0, 10.0], [2.0, 0.0]], y, pos, 2, w)
    assert dy.tolist() == [[2.0, 20.0], [6.0, 0.0], [0.5, 5.0], [0.0, 0.0]]
    assert dw.tolist() == [[84.0, 11.0], [0.0, 4.0]]


def test_sorting_gradients_are_the_differences():
    rng = np.random.default_rng(3)
    pos = np.array([4, 0, 2, 5, -1, 1])
    x, y, w = rng.normal(size=(3, 5)), rng.normal(size=(6, 5)), rng.normal(size=(3, 2))
    g, gs = rng.normal(size=(3, 5)), rng.normal(size=(6, 5))
    dy, dw, _ = OB.unsort_grad(g, y, pos, 2, w)
    assert np.allclose(dy, _differences(lambda a: (g * OB.unsort(a, pos, 2, w)[0]).sum(), y))
    assert np.allclose(dw, _differences(lambda a: (g * OB.unsort(y, pos, 2, a)[0]).sum(), w))
    assert np.allclose(OB.unsort(gs, pos, 2)[0],
                       _differences(lambda a: (gs * OB.sort(a, pos, 2, 6)).sum(), x))


def test_pack_then_back_is_the_weighted_sum():
    rng = np.random.default_rng(4)
    z = rng.normal(size=(9, 8))
    ids, w = OB.route(z, 3, True)
    _, _, pos = OM.pack_routes(ids, 8)
    x = rng.normal(size=(9, 4))
    xs = OB.sort(x, pos, 3, 27)
    assert np.allclose(OB.unsort(xs, pos, 3, w)[0], x)           # weights add up to 1
