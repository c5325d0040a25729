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


def plain_norm_backward(g, h, weight=None, eps=EPS, g_sum=None, dx_dtype=None, want_dweight=True):
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
    return dx, (dx if dx.dtype == h.dtype else d.to(h.dtype)), dw


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
