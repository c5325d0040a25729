"""What leaves accumulate by .backward() through the norm's autograd form on the GPU: each
its own gradient, in memory of its own, twice what one backward pass gives after two.

Doubling is exact in any type, so the accumulated gradients have the bits of twice one
torch.autograd.grad; that in turn is held against the oracle: fp32 to 1e-5 of it and of the
largest (a row of 96 terms of order 1, each off by 2^-24, is below 1e-5), bf16 to a rounding."""

import numpy as np
import pytest
import torch

from nvfp4_w4a4_quantized_act_amd import qat
from oracle import block as OB

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("of", ["y", "h", "both"])
@pytest.mark.parametrize("xt,rt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("shape", [(5, 96), (96,), (2, 3, 96), (3, 1, 2, 61)])
def test_leaves_accumulate_their_own_gradients(shape, xt, rt, of):
    x, r = randn(shape, 1, xt).requires_grad_(True), randn(shape, 2, rt).requires_grad_(True)
    w = randn(shape[-1:], 3).requires_grad_(True)
    gy, gh = randn(shape, 4, rt), randn(shape, 5, rt)
    keep = gy.clone(), gh.clone()

    def results():
        y, h = qat.rms_norm(x, w, EPS, r)
        assert y.shape == h.shape == torch.Size(shape)
        return {"y": ([y], [gy]), "h": ([h], [gh]), "both": ([y, h], [gy, gh])}[of]
    one = torch.autograd.grad(*results()[:1], [x, r, w], results()[1], allow_unused=True)
    for _ in range(2):
        torch.autograd.backward(*results())
    torch.cuda.synchronize()
    assert torch.equal(gy, keep[0]) and torch.equal(gh, keep[1])
    for leaf, g in zip((x, r, w), one):
        assert (leaf.grad is None) == (g is None)
        if g is not None:
            assert leaf.grad.dtype == leaf.dtype and torch.equal(leaf.grad, 2 * g)
    grads = [v.grad for v in (x, r, w) if v.grad is not None]
    assert len({v.untyped_storage().data_ptr() for v in grads}) == len(grads)
    n = shape[-1]
    hr = OB.add(f64(x), f64(r), rt == BF16).reshape(-1, n)
    zero = np.zeros_like(hr)
    dh, dw = OB.rmsnorm_grad(zero if of == "h" else f64(gy).reshape(-1, n), hr, f64(w), EPS,
                             zero if of == "y" else f64(gh).reshape(-1, n))
    for leaf, want in ((x, dh), (r, dh), (w, dw)):
        if leaf.grad is not None:
            # of two bf16 roundings here (a bf16 gradient of h goes to fp32 as it is)
            tol = 1e-5 * (np.abs(want) + np.abs(want).max())
            if leaf.dtype == BF16 or (of == "h" and rt == BF16):
                tol = tol + 2 ** -8 * np.abs(want)
            assert np.all(np.abs(f64(leaf.grad) / 2 - want.reshape(leaf.shape)) <= tol.reshape(leaf.shape))


def test_results_changed_in_place():
    x, r = randn((2, 3, 64), 1).requires_grad_(True), randn((2, 3, 64), 2).requires_grad_(True)
    y, h = qat.rms_norm(x, None, EPS, r)
    y.mul_(3.0)
    gx, gr = torch.autograd.grad(y, [x, r], torch.ones_like(y))
    dh, _ = OB.rmsnorm_grad(3 * np.ones((6, 64)), f64(h).reshape(6, 64), None, EPS)
    assert np.allclose(f64(gx).reshape(6, 64), dh, atol=1e-5) and torch.equal(gx, gr)
    y, h = qat.rms_norm(x, None, EPS, r)
    h.add_(1.0)                                                  # the gradient needs it as it was
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_rows_that_are_not_dense():
    """x, the residual and both gradients as slices and transposed views with leading dimensions."""
    full = randn((3, 4, 70), 1)
    x = full[:, 1:, 3:67].detach().requires_grad_(True)
    r = randn((64, 3, 3), 2).permute(1, 2, 0).requires_grad_(True)
    w = randn((64,), 3).requires_grad_(True)
    gy, gh = randn((3, 64, 3), 4).transpose(1, 2), randn((3, 3, 64), 5)[..., ::1].expand(3, 3, 64)
    dense = [v.detach().clone(memory_format=torch.contiguous_format).requires_grad_(True) for v in (x, r, w)]
    got = torch.autograd.grad(list(qat.rms_norm(x, w, EPS, r)), [x, r, w], [gy, gh])
    want = torch.autograd.grad(list(qat.rms_norm(dense[0], dense[2], EPS, dense[1])), dense,
                               [gy.contiguous(), gh.contiguous()])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("of", ["y", "h", "both"])
@pytest.mark.parametrize("xt,rt", [(F32, F32), (F32, BF16), (BF16, F32)])
def test_any_choice_of_inputs_gets_the_same_gradients(xt, rt, of):
    values = [randn((3, 7, 96), 1, xt), randn((3, 7, 96), 2, rt), randn((96,), 3)]
    gy, gh = randn((3, 7, 96), 4, rt), randn((3, 7, 96), 5, rt)

    def grads(which):
        v = [t.clone().requires_grad_(n in which) for n, t in zip("xrw", values)]
        out = qat.rms_norm(v[0], v[2], EPS, v[1])
        pick = {"y": [(out[0], gy)], "h": [(out[1], gh)], "both": [(out[0], gy), (out[1], gh)]}[of]
        pick = [p for p in pick if p[0].requires_grad]
        if pick:
            torch.autograd.backward([p[0] for p in pick], [p[1] for p in pick])
        return {n: t.grad for n, t in zip("xrw", v)}
    want = grads("xrw")
    for which in ("x", "r", "w", "xr", "xw", "rw"):
        for n, got in grads(which).items():
            if n not in which or want[n] is None:
                assert got is None
            else:
                assert torch.equal(got, want[n])


@pytest.mark.parametrize("rows", [None, 40])
@pytest.mark.parametrize("which", ["y", "w", "yw"])
def test_way_back_with_some_inputs_and_twice(which, rows):
    """Only the gradients that are wanted, the same bits for any choice, doubled by a second pass."""
    t, k, h = 11, 3, 77
    n = rows or t * k
    pos = torch.randperm(n, generator=torch.Generator().manual_seed(0))[:t * k].int().to(DEV)
    values = {"y": randn((n, h), 1), "w": randn((t, k), 2)}
    g = randn((t, h), 3)

    def results(needed):
        v = {name: a.clone().requires_grad_(name in needed) for name, a in values.items()}
        return v, qat.unsort_tokens(v["y"], pos, k, v["w"], rows=rows)
    v, o = results("yw")
    want = dict(zip("yw", torch.autograd.grad(o, [v["y"], v["w"]], g)))
    v, o = results(which)
    o.backward(g)
    o = qat.unsort_tokens(v["y"], pos, k, v["w"], rows=rows)
    o.backward(g)
    for name in "yw":
        assert v[name].grad is None if name not in which else torch.equal(v[name].grad, 2 * want[name])
    dy, dw, _ = OB.unsort_grad(f64(g), f64(values["y"]), pos.cpu().numpy(), k, f64(values["w"]))
    assert np.allclose(f64(want["y"]), dy, rtol=1e-6, atol=0) and np.allclose(f64(want["w"]), dw, atol=1e-4)


def test_sort_and_route_twice():
    t, k, h, e = 9, 2, 50, 16
    x, z = randn((t, h), 1).requires_grad_(True), randn((3, 3, e), 2).requires_grad_(True)
    pos = torch.randperm(t * k, generator=torch.Generator().manual_seed(0)).int().to(DEV)
    gx, gw = randn((t * k, h), 3), randn((3, 3, k), 4)
    one = torch.autograd.grad([qat.sort_tokens(x, pos, k), qat.route(z, k, False)[0]], [x, z], [gx, gw])
    for _ in range(2):
        qat.sort_tokens(x, pos, k).backward(gx)
        qat.route(z, k, False)[0].backward(gw)
    assert torch.equal(x.grad, 2 * one[0]) and torch.equal(z.grad, 2 * one[1])


def test_leading_dimensions_captured():
    """Forward, gradients and the combine of rows in a graph, replayed with eager work between."""
    from nvfp4_w4a4_quantized_act_amd import quads_moe_combine
    x, r = randn((2, 5, 96), 1).requires_grad_(True), randn((2, 5, 96), 2, BF16).requires_grad_(True)
    w = randn((96,), 3).requires_grad_(True)
    gy, gh = randn((2, 5, 96), 4, BF16), randn((2, 5, 96), 5, BF16)
    pos, tw = torch.tensor([3, 0, 4, 1, 2, 9, 8, 7, 6, 5], dtype=torch.int32, device=DEV), randn((5, 2), 6)

    def step():
        y, h = qat.rms_norm(x, w, EPS, r)
        out = quads_moe_combine(y.detach().view(10, 96), pos, tw, y_dtype=1)
        return [y.detach(), h.detach(), out, *torch.autograd.grad([y, h], [x, r, w], [gy, gh])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        with torch.no_grad():
            x.copy_(randn((2, 5, 96), 20 + turn))
            r.copy_(randn((2, 5, 96), 30 + turn, BF16))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
