"""The W4A16 product for few rows per expert on the GPU against oracle/head.py
in fp64.

Tolerance, derived: the operands are exact (an NVFP4 value has at most 6
significant bits, a bf16 activation 8), so an error is a rounding of a partial
sum.  A sum of K products in chains of at most 1024 channels, 8 products per
rounding, is rounded at most 128 + K / 1024 times, sums over the parts of K at
most 16 times more, and the tensor scale once; 16 are left for an activation
far below its row's largest.  Every rounding is at most 2^-24 of sum |x w|:
  |err| <= (176 + K / 1024) 2^-24 sum |x w|, plus half a step of the output.
Chains of 512 channels and one addition per chain stay below that up to K =
114688 (64 + K / 512 + 9 <= 176 + K / 1024).
SwiGLU: |silu'| < 1.1, the hardware exponential and reciprocal to 2^-21."""

import numpy as np
import pytest
import torch

import synth
from oracle import head as OH
from oracle import moe as OM

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


def up(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(DEV)


def bits_f64(b):
    return (np.ascontiguousarray(b).view(np.uint16).astype(np.uint32) << 16).view(
        np.float32).astype(np.float64)


def codes(seed, e, n, k):
    """Random codes, and block scales over the whole range of E4M3 (subnormal ones too)."""
    rng = np.random.default_rng(seed)
    nib = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    sc = rng.integers(30, 90, (e, n, k // 16), dtype=np.uint8)
    sc[rng.random(sc.shape) < 0.05] = 0
    sc[rng.random(sc.shape) < 0.02] = 126
    sc[rng.random(sc.shape) < 0.02] = 3
    ts = rng.uniform(0.5, 2.0, e).astype(np.float32) * np.float32(2.0 ** -9)
    return nib, sc, ts


def acts(seed, t, k):
    ra, ro, _, _ = synth.streams(seed)
    return synth.activations(ra, ro, t, k, "normal", 3.0, max(1, k // 100), 20.0)[0]


def check(Q, x, w, offsets=None, row_token=None, swiglu=False, bf16=False, out=None):
    n, k = w[0].shape[1], x.shape[1]
    rows = int(offsets[-1]) if offsets is not None else x.shape[0]
    print(f"w4a16 rows={rows} K={k} N={n} E={w[0].shape[0]} swiglu={swiglu} bf16={bf16}", flush=True)
    y = Q.quads_moe_w4a16_gemv(
        up(x), tuple(up(a) for a in w), n,
        offsets=None if offsets is None else up(np.asarray(offsets, np.int32)),
        row_token=None if row_token is None else up(row_token),
        epilogue=Q.EPI_SWIGLU if swiglu else Q.EPI_NONE,
        out_dtype=Q.OUT_BF16 if bf16 or swiglu else Q.OUT_F32, out=out)
    torch.cuda.synchronize()
    off = [0, rows] if offsets is None else offsets
    want, bound = OH.w4a16(bits_f64(x), w, off, row_token)
    tol = (176 + k / 1024) * 2.0 ** -24 * bound
    if swiglu:
        g, u, eg, eu = want[:, :n // 2], want[:, n // 2:], tol[:, :n // 2], tol[:, n // 2:]
        with np.errstate(over="ignore"):
            s = g / (1 + np.exp(-g))
        want = s * u
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 2.0 ** -21 * np.abs(want)
    got = (bits_f64(y.view(torch.int16).cpu().numpy()) if bf16 or swiglu
           else y.cpu().numpy().astype(np.float64))
    if bf16 or swiglu:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -126
    err = np.abs(got - want)
    assert got.shape == want.shape and np.isfinite(got).all()
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()),
                                np.argwhere(err > tol)[:4].tolist())
    return y


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,k,n", [(1, 16, 1), (1, 256, 128), (2, 48, 33), (3, 272, 1003),
                                      (5, 1040, 130), (16, 2048, 257), (17, 512, 64),
                                      (33, 1536, 96), (64, 4096, 320), (130, 144, 40),
                                      (1, 8208, 70), (7, 2064, 4099), (16, 8192, 48),
                                      (3, 70000, 20), (40, 2048, 33000), (31, 1040, 60001),
                                      (15, 4096, 600), (700, 64, 24)])
def test_dense(Q, rows, k, n, bf16):
    check(Q, acts(rows + k, rows, k), codes(n, 1, n, k), bf16=bf16)


@pytest.mark.parametrize("k,n", [(256, 128), (272, 258), (2048, 130)])
@pytest.mark.parametrize("rows", [1, 6, 19])
def test_dense_swiglu(Q, rows, k, n):
    w = codes(n, 1, n, k)
    check(Q, acts(rows, rows, k), (w[0], w[1], w[2] * np.float32(0.05)), swiglu=True)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("t,e,topk,k,n", [(1, 4, 2, 256, 128), (9, 5, 2, 48, 62),
                                          (64, 128, 8, 512, 96), (3, 300, 9, 128, 34),
                                          (40, 2, 1, 1040, 100), (2, 4096, 4, 32, 16),
                                          (300, 64, 8, 1024, 1100), (600, 3, 2, 80, 50)])
def test_experts(Q, t, e, topk, k, n, swiglu):
    """Experts without rows, with one, with more than a tile of them; tokens out of order."""
    rng = np.random.default_rng(t + e)
    ids = np.stack([rng.choice(e, topk, replace=False) for _ in range(t)]).astype(np.int32)
    ids[:, 0] = e - 1                                         # one expert takes a share of all
    for r in range(t):
        ids[r, 1:][ids[r, 1:] == e - 1] = 0
    off, rt, _ = OM.pack_routes(ids, e)
    w = codes(t, e, n, k)
    check(Q, acts(t, t, k), (w[0], w[1], w[2] * np.float32(0.05)), off, rt, swiglu=swiglu)


def test_experts_in_packed_order(Q):
    check(Q, acts(3, 20, 256), codes(3, 3, 40, 256), [0, 0, 20, 20])


def test_cancelling_and_tiny_activations(Q):
    """Rows whose entries span the range of bf16, zero rows, exact cancellation."""
    x = acts(5, 6, 512)
    f = bits_f64(x)
    f[0] = 0.0
    f[1, :256] *= 2.0 ** -100
    f[2] *= 2.0 ** 100
    f[3, 1::2] = -f[3, 0::2]
    f[4] *= 2.0 ** -120
    x = synth.f32_to_bf16_bits(f.astype(np.float32))
    w = codes(6, 1, 77, 512)
    w[0][..., :] = (w[0] & 15) | (w[0] << 4)                  # pairs of equal codes
    y = check(Q, x, w)
    assert not bool(y[0].any()) and not bool(y[3].any())


def test_equals_the_learners_product(Q):
    """The weights that quads_nvfp4_weight_qdq writes, at a power-of-two tensor scale, where
    the learner's bf16 weights are the codes' exact values: x Wq^T in fp64 (Eq. (12))."""
    wb = synth.weights(np.random.default_rng(4), 1, 200, 512)
    wf = bits_f64(wb)
    wf[0, 0, 0] = 2688.0 * 2.0 ** -12                          # the largest: s_t = 2^-12
    nib, sc, ts, dq = Q.quads_nvfp4_weight_qdq(up(synth.f32_to_bf16_bits(wf.astype(np.float32))), True)
    x = acts(8, 5, 512)
    y = Q.quads_moe_w4a16_gemv(up(x), (nib, sc, ts), 200)
    torch.cuda.synchronize()
    wq = bits_f64(dq[0].cpu().numpy())
    want, bound = bits_f64(x) @ wq.T, np.abs(bits_f64(x)) @ np.abs(wq).T
    assert ts.item() == 2.0 ** -12
    assert (np.abs(y.cpu().numpy() - want) <= 177 * 2.0 ** -24 * bound).all()


def test_rows_behind_the_last_stay(Q):
    x, w = acts(1, 8, 256), codes(1, 1, 50, 256)
    full = torch.full((8, 50), 9.0, device=DEV)
    got = Q.quads_moe_w4a16_gemv(up(x), tuple(up(a) for a in w), 50, rows=5, out=full[:5])
    torch.cuda.synchronize()
    assert got.data_ptr() == full.data_ptr() and bool((full[5:] == 9.0).all())
    assert torch.equal(full[:5], check(Q, x[:5], w))


def test_empty_and_refusals(Q):
    w = tuple(up(a) for a in codes(1, 2, 40, 64))
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    assert tuple(Q.quads_moe_w4a16_gemv(x[:0], w, 40, offsets=off * 0).shape) == (0, 40)
    for call, error in ((lambda: Q.quads_moe_w4a16_gemv(x.float(), w, 40, offsets=off), TypeError),
                        (lambda: Q.quads_moe_w4a16_gemv(x, w, 41, offsets=off), ValueError),
                        (lambda: Q.quads_moe_w4a16_gemv(x[:, :32].contiguous(), w, 40, offsets=off),
                         ValueError),
                        (lambda: Q.quads_moe_w4a16_gemv(x, w, 40, offsets=off[:2]), ValueError),
                        (lambda: Q.quads_moe_w4a16_gemv(x, w, 40, offsets=off.cpu()), ValueError),
                        (lambda: Q.quads_moe_w4a16_gemv(x, w, 40, rows=4, offsets=off), ValueError),
                        (lambda: Q.quads_moe_w4a16_gemv(x, w, 40), Q.QuadsError),
                        (lambda: Q.quads_moe_w4a16_gemv(x, w, 40, offsets=off,
                                                        epilogue=Q.EPI_SWIGLU), Q.QuadsError)):
        with pytest.raises(error):
            call()


def test_same_bits_streams_and_graph(Q):
    x, w = acts(2, 13, 2048), codes(2, 1, 3001, 2048)
    xt, wt = up(x), tuple(up(a) for a in w)
    want = Q.quads_moe_w4a16_gemv(xt, wt, 3001)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = Q.quads_moe_w4a16_gemv(xt, wt, 3001)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = Q.quads_moe_w4a16_gemv(xt, wt, 3001)
    for seed in (3, 4, 5):
        xt.copy_(up(acts(seed, 13, 2048)))
        graph.replay()
        torch.cuda.synchronize()
        got = held.clone()
        want = Q.quads_moe_w4a16_gemv(xt, wt, 3001)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
