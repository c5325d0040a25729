"""The autograd forms of the layer around the experts on the CPU, with plain torch
in the place of the library's calls: what a learner's leaves accumulate."""

import pytest
import torch

from nvfp4_w4a4_quantized_act_amd import qat

EPS = 1e-5


def plain_norm(x, weight=None, eps=EPS, residual=None, out_dtype=1, want_sum=True):
    """quads_rmsnorm's binding in plain torch."""
    assert x.dim() == 2 and (residual is None or residual.shape == x.shape)
    out = {}
    h = x
    if residual is not None:
        h = out["sum"] = (x.float() + residual.float()).to(residual.dtype)
    y = h.float() * torch.rsqrt((h.float() ** 2).mean(1, keepdim=True) + eps)
    out["y"] = (y if weight is None else y * weight).to(torch.bfloat16 if out_dtype == 1 else torch.float32)
    return out


def plain_norm_backward(g, h, weight=None, eps=EPS, g_sum=None, dx_dtype=None, want_dweight=True,
                        want_dres=True):
    """quads_rmsnorm_backward's binding: dres is dx unless the types differ."""
    assert g.dim() == 2 and h.shape == g.shape and (g_sum is None or g_sum.shape == g.shape)
    v = h.float()
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    n, wg = v * r, g.float() * (1.0 if weight is None else weight.float())
    d = r * (wg - n * (n * wg).mean(1, keepdim=True))
    if g_sum is not None:
        d = d + g_sum.float()
    dx = d.to(dx_dtype or h.dtype)
    dw = (g.float() * n).sum(0).to(weight.dtype) if want_dweight and weight is not None else None
    return dx, (dx if dx.dtype == h.dtype else d.to(h.dtype) if want_dres else None), dw


@pytest.fixture
def norm(monkeypatch):
    monkeypatch.setattr(qat, "quads_rmsnorm", plain_norm)
    monkeypatch.setattr(qat, "quads_rmsnorm_backward", plain_norm_backward)
    return qat.rms_norm


def leaves(shape, residual=torch.float32):
    g = torch.Generator().manual_seed(0)
    x, r, w = (torch.randn(s, generator=g) for s in (shape, shape, shape[-1:]))
    return [x.requires_grad_(True), r.to(residual).requires_grad_(True), w.requires_grad_(True)]


def plain(x, r, w):
    h = x + r
    return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w, h


@pytest.mark.parametrize("of", ["y", "h", "both"])
@pytest.mark.parametrize("shape", [(4, 8), (8,), (1, 8), (2, 2, 8), (2, 1, 3, 8)])
def test_leaves_accumulate_their_own_gradients(norm, shape, of):
    """Two .backward(): twice the gradient in each leaf, in memory of its own."""
    own, ref = leaves(shape), leaves(shape)
    for x, f in ((own, lambda x, r, w: norm(x, w, EPS, r)), (ref, plain)):
        for _ in range(2):
            y, h = f(*x)
            assert y.shape == h.shape == torch.Size(shape)
            ({"y": y.sin(), "h": h * h, "both": y.sin() + h * h}[of]).sum().backward()
    for a, b in zip(own, ref):
        assert (a.grad is None) == (b.grad is None)
        if b.grad is not None:
            assert torch.allclose(a.grad, b.grad, rtol=1e-5, atol=1e-5)
    grads = [v.grad for v in own if v.grad is not None]
    assert len({v.untyped_storage().data_ptr() for v in grads}) == len(grads)
    before = own[1].grad.clone()
    own[0].grad.mul_(0.5)                                        # clipping of one leaf
    assert torch.equal(own[1].grad, before)


def test_one_leaf_as_both_and_gradients_handed_in(norm):
    x, w = leaves((2, 2, 8))[::2]
    ref = x.detach().clone().requires_grad_(True)
    for v, f in ((x, lambda v: norm(v, w, EPS, v)), (ref, lambda v: plain(v, v, w))):
        for _ in range(2):
            y, h = f(v)
            (y.sin() + h * h).sum().backward()
    assert torch.allclose(x.grad, ref.grad, rtol=1e-5, atol=1e-5)
    x, r, w = leaves((2, 2, 8))                                  # h's gradient stays the caller's
    gh = torch.randn(2, 2, 8)
    keep = gh.clone()
    for _ in range(2):
        norm(x, w, EPS, r)[1].backward(gh)
    assert torch.equal(gh, keep)
    assert torch.allclose(x.grad, 2 * gh) and torch.allclose(r.grad, 2 * gh)


@pytest.mark.parametrize("shape", [(4, 8), (2, 2, 8)])
def test_types_and_results_changed_in_place(norm, shape):
    """A bf16 residual under fp32 x; y and h may be changed in place as any operator's results."""
    x, r, w = leaves(shape, torch.bfloat16)
    for _ in range(2):
        y, h = norm(x, w, EPS, r)
        assert y.dtype == h.dtype == torch.bfloat16
        (y.float().sin() + h.float() * 3).sum().backward()
    assert x.grad.dtype == torch.float32 and r.grad.dtype == torch.bfloat16
    assert torch.allclose(r.grad.float(), x.grad, rtol=2 ** -6, atol=2 ** -6)
    x, r, w = leaves(shape)
    y, _ = norm(x, w, EPS, r)
    y.mul_(2.0)
    y.sum().backward()
    ref = leaves(shape)
    (plain(*ref)[0] * 2).sum().backward()
    for a, b in zip((x, r, w), ref):
        assert torch.allclose(a.grad, b.grad, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("of", ["y", "h", "both"])
@pytest.mark.parametrize("xt,rt", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                   (torch.bfloat16, torch.float32)])
def test_only_wanted_gradients_are_formed(norm, monkeypatch, xt, rt, of):
    """For each choice of inputs that need a gradient: those of the call that forms all, and no
    tensor of another's type is asked for."""
    asked = []

    def spy(*args, **kw):
        out = plain_norm_backward(*args, **kw)
        asked.append([v for v in out if v is not None])
        return out
    monkeypatch.setattr(qat, "quads_rmsnorm_backward", spy)
    g = torch.Generator().manual_seed(3)
    values = [torch.randn(2, 3, 8, generator=g).to(xt), torch.randn(2, 3, 8, generator=g).to(rt),
              torch.randn(8, generator=g)]
    gy, gh = (torch.randn(2, 3, 8, generator=g).to(rt) for _ in range(2))

    def grads(which, residual=True):
        v = [t.clone().requires_grad_(n in which) for n, t in zip("xrw", values)]
        out = norm(v[0], v[2], EPS, v[1])
        pick = {"y": ([0], [gy]), "h": ([1], [gh]), "both": ([0, 1], [gy, gh])}[of]
        results = [out[i] for i in pick[0]]
        if not any(t.requires_grad for t in results):
            return {}
        torch.autograd.backward(results, pick[1])
        return {n: t.grad for n, t in zip("xrw", v)}
    want = grads("xrw")
    for which in ("x", "r", "w", "xr", "xw", "rw"):
        asked.clear()
        got = grads(which)
        for n in "xrw":
            if n not in which:
                assert got.get(n) is None
            elif want[n] is None:
                assert got[n] is None
            else:
                assert torch.equal(got[n], want[n])
        if of != "h":
            (made,) = asked
            full = {id(t) for t in made if t.dim() == 2}
            assert len(full) == (2 if {"x", "r"} <= set(which) and xt != rt else 1)
            assert any(t.dim() == 1 for t in made) == ("w" in which)
            if which == "w":
                assert all(t.dtype == torch.bfloat16 for t in made if t.dim() == 2)


def test_without_a_residual(norm):
    x, _, w = leaves((2, 2, 8))
    for _ in range(2):
        norm(x, w, EPS).sin().sum().backward()
    ref = [v.detach().clone().requires_grad_(True) for v in (x, w)]
    for _ in range(2):
        plain(ref[0], torch.zeros(2, 2, 8), ref[1])[0].sin().sum().backward()
    for a, b in zip((x, w), ref):
        assert torch.allclose(a.grad, b.grad, rtol=1e-5, atol=1e-5)
    x = x.detach()
    w.grad = None
    norm(x, w, EPS).sum().backward()
    assert x.grad is None and w.grad is not None
