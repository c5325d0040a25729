"""The layer around the experts as a rollout and its learner use it: the norm into
the quantizers and the MX product, routes into the packing, expert order and back
under autograd, in captured graphs, on other streams and in two streams at once."""

import numpy as np
import pytest
import torch

from nvfp4_w4a4_quantized_act_amd import qat
from oracle import block as OB
from oracle import moe as OM

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(*shape, seed=0, by=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * by).to(dtype).to(DEV)


@pytest.mark.parametrize("t,h", [(1, 64), (5, 256), (64, 2048), (700, 512), (4100, 128), (3, 20000), (3, 40000),
                                 (70000, 128), (2500, 2048)])
def test_norm_feeds_the_quantizers(Q, t, h):
    """Partial maxima give the codes of the dynamic quantizers, bit for bit."""
    x, res = randn(t, h, seed=1, dtype=torch.bfloat16), randn(t, h, seed=2, dtype=torch.bfloat16)
    r = Q.quads_rmsnorm(x, randn(h, seed=3), EPS, res, want_amax=True)
    for a, b in zip(Q.quads_nvfp4_quantize_partials(r["y"], r["amax_part"]),
                    Q.quads_nvfp4_quantize(r["y"])):
        assert torch.equal(a, b)
    if h <= 2048:
        a = Q.quads_rac_quantize_partials(r["y"], 16, r["amax_part"])
        b = Q.quads_rac_quantize(r["y"], 16)
        assert all(torch.equal(a[k], b[k]) for k in b)


def test_amax_slots_behind_the_groups_are_cleared(Q):
    lib, t, h = Q.lib(), 5, 64
    x = randn(t, h, dtype=torch.bfloat16)
    y = torch.empty_like(x)
    n = Q.quads_rmsnorm_amax_groups(t, h)
    part = torch.full((n + 700,), 0x7F7F, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    assert lib.quads_rmsnorm(x.data_ptr(), 1, t, h, h, None, 0, 0, None, 0, EPS, None, y.data_ptr(), 1,
                             None, part.data_ptr(), n + 700, None) == 0
    torch.cuda.synchronize()
    assert not part[n:].any()
    assert part.max().item() == (y.view(torch.int16).int() & 0x7FFF).max().item()


def test_rollout_layer(Q):
    """residual + norm -> route -> pack -> FP8 products -> combine -> the next norm, against the
    same steps in fp64 from the codes: products of E4M3 numbers are exact, a sum of 256 of them
    is off by the MX product's 2^-12 of the sum of magnitudes, the bf16 of h by 2^-8."""
    t, h, i, e, k = 40, 256, 128, 8, 2
    x, res = randn(t, h, seed=1), randn(t, h, seed=2, dtype=torch.bfloat16)
    w, wr = randn(h, seed=3), randn(e, h, seed=4, by=0.1)
    w13 = randn(e, 2 * i, h, seed=5, by=0.05, dtype=torch.bfloat16)
    w2 = randn(e, h, i, seed=6, by=0.05, dtype=torch.bfloat16)
    q13, q2 = Q.quads_mx_quantize(w13), Q.quads_mx_quantize(w2)
    n8 = Q.quads_rmsnorm(x, w, EPS, res, Q.OUT_MX_FP8)
    n16 = Q.quads_rmsnorm(x, w, EPS, res)
    assert torch.equal(n8["sum"], n16["sum"])
    z = n16["y"].float() @ wr.t()
    ids, tw = Q.quads_moe_route(z, k)
    offsets, row_token, pos = Q.quads_moe_pack(ids, e)
    g = Q.quads_moe_mx_gemm((n8["codes"], n8["scales"]), q13, 2 * i, offsets=offsets, row_token=row_token,
                            epilogue=Q.EPI_SWIGLU, out_dtype=Q.OUT_BF16)
    y = Q.quads_moe_mx_gemm(Q.quads_mx_quantize(g), q2, h, offsets=offsets)
    out = Q.quads_moe_combine(y, pos, tw)
    # one form or the other of the way back: the same sums
    assert torch.allclose(Q.quads_moe_unsort(y, pos, k, tw), out, rtol=0, atol=0)
    last = Q.quads_rmsnorm(out, w, EPS, n8["sum"])
    torch.cuda.synchronize()

    def decode(codes, scales):
        v = codes.view(torch.float8_e4m3fn).double().cpu().numpy()
        return v * np.repeat(np.exp2(scales.cpu().numpy().astype(np.float64) - 127), 32, axis=-1)
    hs = OB.add(f64(x), f64(res), True)
    codes, scales = OB.rmsnorm_mx(hs, f64(w), EPS)
    assert np.array_equal(n8["codes"].cpu().numpy(), codes)
    assert np.array_equal(n8["scales"].cpu().numpy(), scales)
    eids, ew = OB.route(f64(z), k, True)
    assert np.array_equal(ids.cpu().numpy(), eids)
    eoff, ert, epos = OM.pack_routes(eids, e)
    assert np.array_equal(pos.cpu().numpy(), epos)
    a, v13 = decode(n8["codes"], n8["scales"]), decode(*q13)
    got = f64(g.view(torch.bfloat16))
    for x_e in range(e):
        sl = slice(eoff[x_e], eoff[x_e + 1])
        gu = a[ert[sl]] @ v13[x_e].T
        size = np.abs(a[ert[sl]]) @ np.abs(v13[x_e]).T
        gate, up = gu[:, :i], gu[:, i:]
        sw = gate / (1 + np.exp(-gate)) * up
        tol = 2 ** -12 * (size[:, :i] * np.abs(up) * 1.2 + size[:, i:] * np.abs(gate)) * 1.1
        assert np.all(np.abs(got[sl] - sw) <= tol + 2 ** -7 * np.abs(sw) + 1e-6)
    want, size = OB.unsort(f64(y), epos, k, f64(tw))
    assert np.all(np.abs(f64(out) - want) <= 2 * U * size + 1e-30)
    hl = OB.add(f64(out), f64(n8["sum"]), True)
    assert np.array_equal(f64(last["sum"]), hl)
    yl, _ = OB.rmsnorm(hl, f64(w), EPS)
    assert np.all(np.abs(f64(last["y"]) - yl) <= (2 ** -8 + 4 * U) * np.abs(yl) + 1e-30)


def learner(ops, x, res, wn, wr, w13, w2, k):
    """An MoE layer with its norm in front; `ops`: (norm, route, experts' rows, back)."""
    norm, route, there, back = ops
    y, h = norm(x, wn, res)
    tw, ids = route(y @ wr.t(), k)
    order = there(y, ids)
    rows, off = order[0], order[1]
    parts = []
    for e in range(w13.shape[0]):
        gu = rows[off[e]:off[e + 1]] @ w13[e].t()
        n = gu.shape[1] // 2
        parts.append((torch.nn.functional.silu(gu[:, :n]) * gu[:, n:]) @ w2[e].t())
    return h + back(torch.cat(parts), order, tw), ids


def own_ops(Q, k, e):
    def there(y, ids):
        offsets, _, pos = Q.quads_moe_pack(ids, e)
        return qat.sort_tokens(y, pos, k), offsets.tolist(), pos
    return (lambda x, w, res: qat.rms_norm(x, w, EPS, residual=res),
            lambda z, kk: qat.route(z, kk), there,
            lambda y, order, tw: qat.unsort_tokens(y, order[2], k, tw))


def plain_ops(k, e, fixed_ids):
    def norm(x, w, res):
        h = x + res
        return h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w, h

    def route(z, kk):
        return torch.softmax(z.gather(1, fixed_ids), 1), fixed_ids

    def there(y, ids):
        off, tok, pos = OM.pack_routes(ids.numpy(), e)
        return y[torch.from_numpy(tok.astype(np.int64))], off.tolist(), torch.from_numpy(pos.astype(np.int64))

    def back(y, order, tw):
        t = tw.shape[0]
        return (y[order[2]].view(t, k, -1) * tw[..., None]).sum(1)
    return norm, route, there, back


def test_learner_layer_and_its_gradients(Q):
    """All in fp32, against autograd of the plain layer in 64 bits.  Each output is a sum of some
    hundred products after two others: a relative 1e-4 of the tensor's norm is a thousand of
    their roundings (u = 6e-8), the order of the sums left to torch."""
    t, h, i, e, k = 50, 96, 40, 8, 3
    shapes = [(t, h), (t, h), (h,), (e, h), (e, 2 * i, h), (e, h, i)]
    by = [1.0, 2.0, 1.0, 0.3, 0.1, 0.1]
    own = [randn(*s, seed=n, by=b).requires_grad_(True) for n, (s, b) in enumerate(zip(shapes, by))]
    y, ids = learner(own_ops(Q, k, e), *own, k)
    g = randn(t, h, seed=9)
    grads = torch.autograd.grad(y, own, g)
    plain = [p.detach().double().cpu().requires_grad_(True) for p in own]
    want, _ = learner(plain_ops(k, e, ids.cpu().long()), *plain, k)
    wgrads = torch.autograd.grad(want, plain, g.double().cpu())
    for a, b in zip((y,) + grads, (want,) + wgrads):
        a, b = f64(a), b.detach().numpy()
        assert np.linalg.norm(a - b) <= 1e-4 * np.linalg.norm(b), (a.shape, np.linalg.norm(a - b))


def test_autograd_forms(Q):
    """Shapes with leading dimensions, types, outputs without a gradient, inputs without one."""
    x = randn(2, 3, 64, seed=1).requires_grad_(True)
    res = randn(2, 3, 64, seed=2, dtype=torch.bfloat16).requires_grad_(True)
    w = randn(64, seed=3).requires_grad_(True)
    y, h = qat.rms_norm(x, w, EPS, res)
    assert y.dtype == h.dtype == torch.bfloat16 and y.shape == h.shape == x.shape
    gy, gh = randn(2, 3, 64, seed=4, dtype=torch.bfloat16), randn(2, 3, 64, seed=5, dtype=torch.bfloat16)
    gx, gr, gw = torch.autograd.grad([y, h], [x, res, w], [gy, gh], retain_graph=True)
    hr = OB.add(f64(x).reshape(6, 64), f64(res).reshape(6, 64), True)
    dh, dw = OB.rmsnorm_grad(f64(gy).reshape(6, 64), hr, f64(w), EPS, f64(gh).reshape(6, 64))
    assert gx.dtype == torch.float32 and gr.dtype == torch.bfloat16 and gw.dtype == torch.float32
    assert np.allclose(f64(gx).reshape(6, 64), dh, rtol=1e-5, atol=1e-5)
    assert np.allclose(f64(gr).reshape(6, 64), dh, rtol=2 ** -7, atol=1e-5)
    assert np.allclose(f64(gw), dw, rtol=1e-5, atol=1e-5)
    # only the sum, or only the norm, has a gradient
    a, b = torch.autograd.grad(h, [x, res], gh, retain_graph=True)
    assert torch.equal(a, gh.float()) and torch.equal(b, gh)
    gx, = torch.autograd.grad(y, [x], gy)
    dh, _ = OB.rmsnorm_grad(f64(gy).reshape(6, 64), hr, f64(w), EPS)
    assert np.allclose(f64(gx).reshape(6, 64), dh, rtol=1e-5, atol=1e-5)
    y = qat.rms_norm(x, None, EPS, out_dtype=torch.bfloat16)         # no residual, no weight
    assert y.dtype == torch.bfloat16
    gx, = torch.autograd.grad(y, [x], gy)
    dh, _ = OB.rmsnorm_grad(f64(gy).reshape(6, 64), f64(x).reshape(6, 64), None, EPS)
    assert np.allclose(f64(gx).reshape(6, 64), dh, rtol=1e-5, atol=1e-5)
    z = randn(2, 3, 16, seed=6, dtype=torch.bfloat16).requires_grad_(True)
    tw, ids = qat.route(z, 4, False)
    assert tw.shape == ids.shape == (2, 3, 4) and not ids.requires_grad and tw.dtype == torch.float32
    g = randn(2, 3, 4, seed=7)
    gz, = torch.autograd.grad(tw, [z], g)
    assert gz.dtype == torch.bfloat16 and gz.shape == z.shape
    want = OB.route_grad(f64(z).reshape(6, 16), f64(ids).reshape(6, 4), f64(g).reshape(6, 4), False)
    assert np.allclose(f64(gz).reshape(6, 16), want, rtol=2 ** -7, atol=1e-6)


def test_expanded_and_repeated_inputs(Q):
    """A residual broadcast over tokens, one tensor as x and as the residual, rows of a transposed
    view, a gradient broadcast by sum()."""
    x = randn(6, 64, seed=1).requires_grad_(True)
    one = randn(1, 64, seed=2).requires_grad_(True)
    w = torch.ones(64, device=DEV)
    y, h = qat.rms_norm(x, w, EPS, residual=one.expand(6, 64))
    gx, go = torch.autograd.grad(y.sum() + h.sum(), [x, one])
    hr = f64(x) + f64(one)
    dh, _ = OB.rmsnorm_grad(np.ones((6, 64)), hr.astype(np.float32), None, EPS, np.ones((6, 64)))
    assert np.allclose(f64(gx), dh, atol=1e-5) and np.allclose(f64(go), dh.sum(0, keepdims=True), atol=1e-4)
    y, h = qat.rms_norm(x, w, EPS, residual=x)
    gx, = torch.autograd.grad(y.sum(), [x])
    dh, _ = OB.rmsnorm_grad(np.ones((6, 64)), 2 * f64(x), None, EPS)
    assert np.allclose(f64(gx), 2 * dh, atol=1e-5)
    xt = randn(64, 6, seed=3).t()
    assert torch.equal(Q.quads_rmsnorm(xt)["y"], Q.quads_rmsnorm(xt.contiguous())["y"])
    off = randn(7, 65, seed=4)[:, 1:]                                # rows not 16-byte aligned
    assert torch.equal(Q.quads_rmsnorm(off)["y"], Q.quads_rmsnorm(off.contiguous())["y"])


def test_capacity_rows_get_no_garbage(Q):
    """Rows without a slot are 0 in both directions, whatever the memory held."""
    t, h, k, rows = 9, 32, 2, 24
    pos = torch.full((t * k,), -1, dtype=torch.int32)
    pos[:10] = torch.arange(10, dtype=torch.int32) * 2
    pos = pos.to(DEV)
    torch.full((rows, h), float("nan"), device=DEV)                  # the next allocation's memory
    x = randn(t, h, seed=1).requires_grad_(True)
    xs = qat.sort_tokens(x, pos, k, rows)
    y = (xs * 2).detach().requires_grad_(True)
    tw = torch.rand((t, k), device=DEV, requires_grad=True)
    out = qat.unsort_tokens(y, pos, k, tw, rows=rows)
    gy, gw = torch.autograd.grad(out.sum(), [y, tw])
    gx, = torch.autograd.grad(xs.sum(), [x])
    posn = pos.cpu().numpy()
    assert np.array_equal(f64(xs), OB.sort(f64(x), posn, k, rows))
    dy, dw, _ = OB.unsort_grad(np.ones((t, h)), f64(y), posn, k, f64(tw))
    assert np.allclose(f64(gy), dy) and np.allclose(f64(gw), dw, atol=1e-5)
    assert np.array_equal(f64(gx), OB.unsort(np.ones((rows, h)), posn, k)[0])


def everything(Q, s):
    n = Q.quads_rmsnorm(s["x"], s["w"], EPS, s["res"], want_amax=True)
    f8 = Q.quads_rmsnorm(s["x"], s["w"], EPS, s["res"], Q.OUT_MX_FP8)
    dx = Q.quads_rmsnorm_backward(s["g"], n["sum"], s["w"], EPS, s["gs"], torch.float32)
    ids, tw = Q.quads_moe_route(s["z"], 4, False)
    dz = Q.quads_moe_route_backward(s["z"], ids, tw, s["gw"], False)
    _, _, pos = Q.quads_moe_pack(ids, s["z"].shape[1])
    xs = Q.quads_moe_sort(n["y"], pos, 4)
    # rows without a slot: few, or many of a large output (the two ways of zeroing them)
    rows = xs.shape[0] + (2200 if xs.shape[1] > 10000 else 5)
    xr = Q.quads_moe_sort(n["y"], pos, 4, rows=rows)
    o = Q.quads_moe_unsort(xs, pos, 4, tw)
    dy, dw = Q.quads_moe_unsort_backward(o, xs, pos, 4, tw)
    dr, _ = Q.quads_moe_unsort_backward(o, xr, pos, 4, tw, rows=rows)
    return [*n.values(), f8["codes"], f8["scales"], *dx, ids, tw, dz, pos, xs, xr, o, dy, dw, dr]


def state(t, h, e, seed):
    return dict(x=randn(t, h, seed=seed), res=randn(t, h, seed=seed + 1, dtype=torch.bfloat16),
                w=randn(h, seed=seed + 2), g=randn(t, h, seed=seed + 3, dtype=torch.bfloat16),
                gs=randn(t, h, seed=seed + 4, dtype=torch.bfloat16), z=randn(t, e, seed=seed + 5),
                gw=randn(t, 4, seed=seed + 6))


@pytest.mark.parametrize("t,h", [(33, 256), (300, 2048), (5, 16384)])
def test_captured_and_replayed(Q, t, h):
    """Two graphs of the same calls, replayed in turn with eager work between, on new inputs."""
    made = []
    for n in range(2):
        s = state(t, h, 32, 100 * n)
        everything(Q, s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = everything(Q, s)
        made.append((s, graph, out))
    for turn in range(3):
        for n, (s, graph, out) in enumerate(made):
            for k, v in state(t, h, 32, 1000 + 10 * turn + n).items():
                s[k].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            want = everything(Q, s)
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_backward_captured(Q):
    """autograd.grad of the operators inside a graph, against the eager gradients."""
    t, h, k, e = 40, 128, 4, 16
    x = randn(t, h, seed=1).requires_grad_(True)
    w = randn(h, seed=2).requires_grad_(True)
    z = randn(t, e, seed=3).requires_grad_(True)

    def step():
        y, s = qat.rms_norm(x, w, EPS, residual=x)
        tw, ids = qat.route(z, k)
        _, _, pos = Q.quads_moe_pack(ids, e)
        o = qat.unsort_tokens(qat.sort_tokens(y, pos, k), pos, k, tw * tw)
        return torch.autograd.grad([o, s], [x, w, z], [torch.ones_like(o), torch.ones_like(s)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [a.clone() for a in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        if turn:
            with torch.no_grad():
                x.copy_(randn(t, h, seed=20 + turn))
                z.copy_(randn(t, e, seed=30 + turn))
            want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_streams_at_once(Q):
    """Calls of several streams that overlap keep their results."""
    states = [state(700, 2048, 64, 1), state(900, 1024, 64, 2), state(6, 16000, 64, 3)]
    want = [everything(Q, s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [[] for _ in states]
    for _ in range(3):
        for n, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[n].append(everything(Q, states[n]))
    torch.cuda.synchronize()
    for n in range(len(states)):
        for run in got[n]:
            for a, b in zip(run, want[n]):
                assert torch.equal(a, b)


def test_same_bits_every_time(Q):
    s = state(3000, 768, 128, 5)
    first = everything(Q, s)
    for _ in range(3):
        for a, b in zip(everything(Q, s), first):
            assert torch.equal(a, b)


def test_bf16_bits(Q):
    """bf16 as int16 or uint16 bit patterns: the same results, sums and gradients in that type."""
    t, h, e, k = 12, 72, 16, 2
    s = dict(x=randn(t, h, seed=1, dtype=torch.bfloat16), res=randn(t, h, seed=2, dtype=torch.bfloat16),
             w=randn(h, seed=3, dtype=torch.bfloat16), g=randn(t, h, seed=4, dtype=torch.bfloat16),
             z=randn(t, e, seed=5, dtype=torch.bfloat16), gw=randn(t, k, seed=6))
    want = None
    for dtype in (torch.bfloat16, torch.int16, torch.uint16):
        v = {n: a.view(dtype) if a.dtype == torch.bfloat16 else a for n, a in s.items()}
        n = Q.quads_rmsnorm(v["x"], v["w"], EPS, v["res"])
        assert n["sum"].dtype == dtype and n["y"].dtype == torch.bfloat16
        dx, dres, dw = Q.quads_rmsnorm_backward(v["g"], n["sum"], v["w"], EPS, v["g"])
        assert dx.dtype == dres.dtype == dw.dtype == dtype
        ids, tw = Q.quads_moe_route(v["z"], k)
        dz = Q.quads_moe_route_backward(v["z"], ids, tw, v["gw"])
        assert dz.dtype == dtype
        _, _, pos = Q.quads_moe_pack(ids, e)
        xs, xr = Q.quads_moe_sort(v["x"], pos, k), Q.quads_moe_sort(v["x"], pos, k, rows=t * k + 3)
        o = Q.quads_moe_unsort(xs, pos, k, tw, Q.OUT_BF16)
        dy, dtw = Q.quads_moe_unsort_backward(v["g"], xs, pos, k, tw)
        assert xs.dtype == xr.dtype == dy.dtype == dtype and o.dtype == torch.bfloat16
        got = [n["sum"], n["y"], dx, dw, ids, tw, dz, xs, xr, o, dy, dtw]
        got = [a.view(torch.int16) if a.element_size() == 2 else a for a in got]
        want = want or got
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits(Q):
    """More than 2^31 channels (and more than 2^32 bytes): the last rows as a call on them alone."""
    h, t = 4096, 2 ** 19 + 3
    x = torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
    x[:] = randn(1, h, seed=1, dtype=torch.bfloat16)
    x[-3:] = randn(3, h, seed=2, dtype=torch.bfloat16)
    w = randn(h, seed=3, dtype=torch.bfloat16)
    for out, key in ((Q.OUT_BF16, "y"), (Q.OUT_MX_FP8, "codes")):
        r = Q.quads_rmsnorm(x, w, EPS, out_dtype=out)
        a = Q.quads_rmsnorm(x[-3:].contiguous(), w, EPS, out_dtype=out)
        assert torch.equal(r[key][-3:], a[key])
        if out == Q.OUT_MX_FP8:
            assert torch.equal(r["scales"][-3:], a["scales"])
        del r
    dx, _, _ = Q.quads_rmsnorm_backward(x, x, w, EPS, x)
    b, _, _ = Q.quads_rmsnorm_backward(*[x[-3:].contiguous()] * 2, w, EPS, x[-3:].contiguous())
    assert torch.equal(dx[-3:], b)
    del dx
    pos = torch.arange(t - 1, -1, -1, dtype=torch.int32, device=DEV)
    xs = Q.quads_moe_sort(x, pos, 1)
    assert torch.equal(xs[:3], x[-3:].flip(0)) and torch.equal(xs[-1], x[0])
    o = Q.quads_moe_unsort(xs, pos, 1, out_dtype=Q.OUT_BF16)
    assert torch.equal(o[-3:], x[-3:])
    dy, dw = Q.quads_moe_unsort_backward(o, xs, pos, 1, torch.ones((t, 1), device=DEV))
    assert torch.equal(dy[:3], x[-3:].flip(0))
    n2 = (x[-3:].double() ** 2).sum(1)
    assert ((dw[-3:, 0].double() - n2).abs() <= (h / 64 + 24) * U * n2).all()
    del xs, o, dy
    z = x.view(-1, 128)[: 2 ** 24 - 1]                              # 2^31 logits
    ids, tw = Q.quads_moe_route(z, 8)
    i2, w2 = Q.quads_moe_route(z[-5:].contiguous(), 8)
    assert torch.equal(ids[-5:], i2) and torch.equal(tw[-5:], w2)
    dz = Q.quads_moe_route_backward(z, ids, tw, tw, False)
    d2 = Q.quads_moe_route_backward(z[-5:].contiguous(), i2, w2, w2, False)
    assert torch.equal(dz[-5:], d2)


def test_views_are_taken(Q):
    """Column slices and transposed views of every input give what their copies give."""
    t, h, k, e = 10, 48, 2, 8
    x, g, y = randn(t, h + 5, seed=1)[:, 5:], randn(h, t, seed=2).t(), randn(t * k, 2 * h, seed=3)[:, ::2]
    z = randn(e, t, seed=4).t()
    c = [a.contiguous() for a in (x, g, y, z)]
    ids, tw = Q.quads_moe_route(z, k)
    assert torch.equal(ids, Q.quads_moe_route(c[3], k)[0])
    _, _, pos = Q.quads_moe_pack(ids, e)
    assert torch.equal(Q.quads_moe_sort(x, pos, k), Q.quads_moe_sort(c[0], pos, k))
    assert torch.equal(Q.quads_moe_unsort(y, pos, k, tw), Q.quads_moe_unsort(c[2], pos, k, tw))
    for a, b in zip(Q.quads_moe_unsort_backward(g, y, pos, k, tw),
                    Q.quads_moe_unsort_backward(c[1], c[2], pos, k, tw)):
        assert torch.equal(a, b)
    w = randn(2 * h, seed=5)[::2]
    for a, b in zip(Q.quads_rmsnorm_backward(g, x, w, EPS, g),
                    Q.quads_rmsnorm_backward(c[1], c[0], w.contiguous(), EPS, c[1])):
        assert torch.equal(a, b)
    gz = randn(k, t, seed=6).t()
    assert torch.equal(Q.quads_moe_route_backward(z, ids, tw, gz, False),
                       Q.quads_moe_route_backward(c[3], ids, tw, gz.contiguous(), False))


def test_autograd_of_nothing(Q):
    """No tokens: empty results, a zero gradient of the weight."""
    x = torch.zeros((0, 32), device=DEV, requires_grad=True)
    w = torch.ones(32, device=DEV, requires_grad=True)
    z = torch.zeros((0, 8), device=DEV, requires_grad=True)
    y, h = qat.rms_norm(x, w, EPS, residual=x)
    tw, ids = qat.route(z, 2)
    pos = torch.zeros(0, dtype=torch.int32, device=DEV)
    o = qat.unsort_tokens(qat.sort_tokens(y, pos, 2), pos, 2, tw)
    assert y.shape == h.shape == o.shape == (0, 32) and tw.shape == ids.shape == (0, 2)
    gx, gw, gz = torch.autograd.grad(o.sum() + h.sum(), [x, w, z])
    assert gx.shape == (0, 32) and gz.shape == (0, 8) and not gw.any()
