"""Sizes at which the layer's kernels take another path than at small ones, every row against
fp64 torch on the device: the norm's gradient where a work-group has more than one turn of rows,
or two work-groups share a CU, and packed rows beyond the caches at odd widths, whose 16-byte
accesses past the caches start at any element.

Tolerances (u = 2^-24; HALF: half a step of the output's type):
  * dh: r u (|w g| + |n| M + 4 |n c| + |w g - n c|) + 2 u |r (w g - n c)| + u |dh| with
    M = mean |n w g|: the roundings of n, w g, c, their fused sum, r's and the last sum's.
  * dweight: terms g n with n's 2 u, at most 64 + 127 additions in fp32: 194 u sum |g n|.
  * sort: a copy.  back: topk u sum |w y|.  dy: u |dy|.  dw: products in fused sums, at most
    H / 64 + 16 in a thread before at most 19 more additions: (H / 64 + 36) u sum |g y|."""

import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TINY = 2.0 ** -126
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


def randn(shape, seed, dtype, by=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * by).to(TYPES[dtype])


def close(got, want, tol):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,h", [(40000, 64), (40001, 61), (70000, 64), (33000, 5), (20000, 128), (20003, 125),
                                 (10000, 250), (5000, 512), (2600, 1000), (8200, 5000), (8193, 5001), (8200, 6144),
                                 (700, 8192), (600, 12001)])
def test_norm_gradient(t, h, dtype):
    print(f"norm gradient T={t} H={h} {dtype}", flush=True)
    x, g, s = randn((t, h), 1, dtype), randn((t, h), 2, dtype, 0.1), randn((t, h), 3, dtype, 0.1)
    w = (1.0 + 0.3 * randn((h,), 4, "f32")).to(TYPES[dtype])
    dx, _, dw = Q.quads_rmsnorm_backward(g, x, w, EPS, s)
    torch.cuda.synchronize()
    hd, gd, wd = x.double(), g.double(), w.double()
    r = torch.rsqrt((hd * hd).mean(1, keepdim=True) + EPS)
    n, wg = hd * r, gd * wd
    c, m = (n * wg).mean(1, keepdim=True), (n * wg).abs().mean(1, keepdim=True)
    inner = wg - n * c
    dh = s.double() + r * inner
    tol = r * U * (wg.abs() + n.abs() * m + 4 * (n * c).abs() + inner.abs())
    tol = (tol + 2 * U * (r * inner).abs() + U * dh.abs()) * 1.01 + TINY * (1 + r)
    close(dx, dh, tol * (1 + HALF[dtype]) + HALF[dtype] * dh.abs())
    want, size = (gd * n).sum(0), (gd * n).abs().sum(0)
    close(dw, want, 194 * U * size * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + TINY)


@pytest.mark.parametrize("room", [False, True])
@pytest.mark.parametrize("t,h,k", [(1200, 2049, 4), (1300, 2047, 4), (4300, 515, 4), (2100, 4099, 1),
                                   (12600, 2049, 4), (50001, 517, 4), (6200, 4001, 4), (12400, 2048, 4),
                                   (1700, 8193, 8)])
def test_packed_rows_beyond_the_caches(t, h, k, room):
    """16 MB and 192 MB are passed, with and without rows that no slot names."""
    n = t * k + (t * k // 4 if room else 0)
    print(f"sort T={t} H={h} topk={k} rows={n}", flush=True)
    gen = torch.Generator(DEV).manual_seed(h)
    pos = torch.randperm(n, generator=gen, device=DEV, dtype=torch.int32)[:t * k]
    if room:
        pos[torch.rand(t * k, generator=gen, device=DEV) < 0.05] = -1
    given = n if room else None
    have = pos >= 0
    at = pos[have].long()
    token = torch.arange(t, device=DEV).repeat_interleave(k)[have]
    empty = torch.ones(n, dtype=torch.bool, device=DEV)
    empty[at] = False
    x, y, g = randn((t, h), 1, "bf16"), randn((n, h), 2, "bf16"), randn((t, h), 3, "bf16")
    w = torch.rand((t, k), generator=gen, device=DEV)
    torch.full((n, h), float("nan"), dtype=torch.bfloat16, device=DEV)   # the next allocation's memory
    xs = Q.quads_moe_sort(x, pos, k, given)
    torch.cuda.synchronize()
    assert torch.equal(xs[at], x[token]) and not xs[empty].any()
    del xs
    dy, dw = Q.quads_moe_unsort_backward(g, y, pos, k, w, given)
    outs = [Q.quads_moe_unsort(y, pos, k, v, c) for v in (w, None) for c in (Q.OUT_F32, Q.OUT_BF16)]
    torch.cuda.synchronize()
    assert not dy[empty].any()
    wn = torch.where(have.view(t, k), w, 0.0)
    slot = torch.where(have, pos, 0).long().view(t, k)
    for a in range(0, t, 2000):                                  # fp64 of some tokens at a time
        b = min(t, a + 2000)
        yd = torch.where(have.view(t, k)[a:b, :, None], y[slot[a:b]].double(), 0.0)
        gd, wd = g[a:b].double()[:, None], wn[a:b].double()[..., None]
        edy = (gd * wd).view(-1, h)
        mine = have.view(t, k)[a:b].reshape(-1)
        got = dy[slot[a:b].view(-1)][mine]
        close(got, edy[mine], (U + HALF["bf16"]) * 1.01 * edy[mine].abs() + TINY)
        prod = gd * yd
        close(dw[a:b], prod.sum(2), (h / 64 + 36) * U * prod.abs().sum(2) + TINY)
        for i, out in enumerate(outs):
            v = yd * wd if i < 2 else yd
            want = v.sum(1)
            tol = k * U * v.abs().sum(1) * (1 + HALF["bf16"]) + TINY
            close(out[a:b], want, tol + (HALF["bf16"] * want.abs() if i % 2 else 0))
