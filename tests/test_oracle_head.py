"""Pins of oracle/head.py (CPU): against scalar loops, hand values and central
differences of its own losses, with masked entries, empty rows, ties, lists
with left-out and repeated ids."""

import math

import numpy as np
import pytest

from oracle import head as OH
from oracle import nvfp4 as ON
import synth


def _z(t=5, v=17, seed=0, masked=True):
    z = np.random.default_rng(seed).normal(size=(t, v)) * 2
    if masked:
        z[1, 3:9] = -np.inf
    return z


def test_logprob_by_hand():
    z = np.array([[0.0, math.log(3.0), -np.inf, 0.0]])
    r = OH.token_logprob(z, [1], 1.0, 4)
    assert r["logp"][0] == pytest.approx(math.log(0.6))
    assert r["entropy"][0] == pytest.approx(-(0.6 * math.log(0.6) + 0.4 * math.log(0.2)))
    assert r["stats"][0, 0] == math.log(3.0)
    assert r["stats"][0, 1] == pytest.approx(math.log(5.0 / 3.0))
    assert r["top_id"][0].tolist() == [1, 0, 3, 2]           # equal entries by index
    assert r["top_logp"][0, 3] == -np.inf


def test_logprob_loops_and_temperature():
    z, it = _z(), 0.7
    ids = np.array([0, 4, -1, 17, 16])                       # row 1: masked token; 2, 3: none
    r = OH.token_logprob(z, ids, it)
    for t in range(5):
        tot = sum(math.exp(it * a) for a in z[t] if a > -np.inf)
        p = [math.exp(it * a) / tot if a > -np.inf else 0.0 for a in z[t]]
        assert r["entropy"][t] == pytest.approx(-sum(a * math.log(a) for a in p if a > 0))
        if 0 <= ids[t] < 17:
            want = math.log(p[ids[t]]) if p[ids[t]] > 0 else -np.inf
            assert r["logp"][t] == pytest.approx(want)
        else:
            assert r["logp"][t] == 0.0


def test_empty_row():
    z = np.full((2, 6), -np.inf)
    z[1, 2] = 1.0
    r = OH.token_logprob(z, [3, 2], 1.0, 6)
    assert r["entropy"].tolist() == [0.0, 0.0] and r["logp"].tolist() == [-np.inf, 0.0]
    assert r["stats"][0].tolist() == [-np.inf, 0.0] and r["stats"][1].tolist() == [1.0, 0.0]
    assert r["top_id"].tolist() == [[0, 1, 2, 3, 4, 5], [2, 0, 1, 3, 4, 5]]
    assert not OH.token_logprob_grad(z, [3, 2], [1.0, 1.0], [1.0, 1.0])[0].any()


def _differences(f, z, h=1e-6):
    out = np.zeros_like(z)
    for i in range(z.shape[0]):
        for j in range(z.shape[1]):
            if np.isneginf(z[i, j]):
                continue
            a, b = z.copy(), z.copy()
            a[i, j] += h
            b[i, j] -= h
            out[i, j] = (f(a) - f(b)) / (2 * h)
    return out


@pytest.mark.parametrize("it", [0.5, 1.0, 1.3])
def test_logprob_gradient_is_the_difference_quotient(it):
    z = _z(seed=3)
    ids = np.array([0, 1, -1, 17, 16])
    gl = np.array([1.0, -0.5, 2.0, 3.0, 0.25])
    gh = np.array([0.3, 1.0, -0.2, 0.0, 0.7])

    def f(a):
        r = OH.token_logprob(a, ids, it)
        return float((gl * r["logp"]).sum() + (gh * r["entropy"]).sum())
    g = OH.token_logprob_grad(z, ids, gl, gh, it)
    assert np.abs(g - _differences(f, z)).max() < 1e-8       # h^2 plus eps / h


def _list():
    t_id = np.array([[0, 3], [2, 1], [5, 5], [-1, 9], [-1, 17]])   # repeated, left out, all out
    t_val = np.log(np.array([[0.5, 0.3], [0.9, 0.05], [0.25, 0.25], [0.4, 0.6], [0.1, 0.2]]))
    return t_val, t_id


def test_teacher():
    t_val, t_id = _list()
    q, lq = OH.teacher(t_val, t_id, 17, 1.0, True)
    assert q[0] == pytest.approx([0.625, 0.375]) and q[3].tolist() == [0.0, 1.0]
    assert q[4].tolist() == [0.0, 0.0] and lq[4].tolist() == [-np.inf, -np.inf]
    assert OH.teacher(t_val, t_id, 17, 2.0, True)[0][0] == pytest.approx([25 / 34, 9 / 34])
    assert OH.teacher(t_val, t_id, 17, 2.0, False)[0][3] == pytest.approx([0.0, 0.6])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("it", [1.0, 0.6])
def test_distill_loss_and_gradient(renorm, it):
    z = _z(seed=5)
    t_val, t_id = _list()
    w = np.array([1.0, 0.5, 2.0, 1.5, 1.0])
    g = np.array([1.0, 2.0, -0.5, 0.3, 1.0])
    loss = OH.distill(z, t_val, t_id, w, it, renorm)
    q, _ = OH.teacher(t_val, t_id, 17, it, renorm)
    lp = OH.log_softmax(z, it)
    for t in range(5):
        want = sum(q[t, i] * (math.log(q[t, i]) - lp[t, t_id[t, i]])
                   for i in range(2) if q[t, i] > 0)
        assert loss[t] == pytest.approx(w[t] * want)
    assert loss[4] == 0.0
    grad = OH.distill_grad(z, t_val, t_id, g, w, it, renorm)
    diff = _differences(lambda a: float((g * OH.distill(a, t_val, t_id, w, it, renorm)).sum()), z)
    assert np.abs(grad - diff).max() < 1e-8


def test_distill_zero_weight_and_masked_alternative():
    z = _z(seed=5)
    t_val, t_id = _list()
    z[0, 0] = -np.inf                                        # q > 0 where p = 0
    assert OH.distill(z, t_val, t_id)[0] == np.inf
    assert OH.distill(z, t_val, t_id, np.zeros(5))[0] == 0.0
    assert np.isfinite(OH.distill_grad(z, t_val, t_id, np.ones(5))).all()


def test_w4a16_loops():
    wb = synth.weights(np.random.default_rng(1), 2, 3, 32)
    w = ON.weight_qdq(wb)[:3]
    x = np.random.default_rng(2).normal(size=(4, 32))
    y, b = OH.w4a16(x, w, [0, 2, 3], [3, 0, 1])
    for p, (e, r) in enumerate([(0, 3), (0, 0), (1, 1)]):
        for n in range(3):
            wr = ON.dequantize_unscaled(w[0][e, n:n + 1], w[1][e, n:n + 1])[0] * float(w[2][e])
            assert y[p, n] == pytest.approx(sum(x[r, j] * wr[j] for j in range(32)))
            assert b[p, n] == pytest.approx(sum(abs(x[r, j] * wr[j]) for j in range(32)))
