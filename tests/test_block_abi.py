"""The C ABI of the layer around the experts (include/quads_block.h) and its
binding on the CPU: every declared symbol is exported, and bad arguments are
refused on the host before any launch."""

import ctypes
import os
import re

import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q
from nvfp4_w4a4_quantized_act_amd import qat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced (checks fail first)
MORE = ctypes.c_void_p(0x20000)
MIS = ctypes.c_void_p(0x10004)           # misaligned for rows, aligned for 32-bit words
MIS2 = ctypes.c_void_p(0x10002)          # misaligned for a 32-bit word
INF, NAN = float("inf"), float("nan")


def test_library_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "quads_block.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(quads_[a-z0-9_]+)\s*\(", src))
    assert names == {"quads_rmsnorm", "quads_rmsnorm_amax_groups", "quads_rmsnorm_backward",
                     "quads_rmsnorm_backward_ws", "quads_moe_route", "quads_moe_route_backward",
                     "quads_moe_sort", "quads_moe_sort_ws", "quads_moe_unsort",
                     "quads_moe_unsort_backward"}
    lib = Q.lib()
    assert all(hasattr(lib, n) for n in names)
    assert int(re.search(r"#define QUADS_OUT_MX_FP8 (\d+)", src).group(1)) == Q.OUT_MX_FP8


def test_norm_validation():
    f = Q.lib().quads_rmsnorm

    def call(x=FAKE, xt=1, t=4, h=64, ldx=64, res=FAKE, rt=1, ldr=64, w=FAKE, wt=1, eps=1e-6,
             total=FAKE, y=MORE, yt=1, sc=None, am=None, na=0):
        return f(x, xt, t, h, ldx, res, rt, ldr, w, wt, eps, total, y, yt, sc, am, na, None)
    assert call(t=-1) == -2 and call(t=1 << 31) == -2
    assert call(h=0) == -2 and call(h=1 << 24, ldx=1 << 24) == -2
    assert call(ldx=63) == -2 and call(ldr=63) == -2 and call(ldx=1 << 31) == -2
    assert call(xt=2) == -1 and call(rt=2) == -1 and call(wt=-1) == -1 and call(yt=3) == -1
    for eps in (0.0, -1.0, 9e-71, 2e70, INF, NAN):
        assert call(eps=eps) == -1
    assert call(x=None) == -1 and call(x=MIS) == -1 and call(res=MIS) == -1
    assert call(w=MIS) == -1 and call(total=MIS) == -1 and call(y=None) == -1 and call(y=MIS) == -1
    assert call(res=None) == -1                                  # a sum without a residual
    assert call(yt=2) == -1 and call(yt=2, sc=MIS) == -1         # scales
    assert call(yt=2, h=48, ldx=48, ldr=48, sc=FAKE) == -2       # whole blocks of 32
    n = Q.lib().quads_rmsnorm_amax_groups(4, 64)
    assert n >= 1
    assert call(am=FAKE, na=n - 1) == -3 and call(am=MIS2, na=n) == -1
    assert call(am=FAKE, na=n, yt=0) == -1
    assert call(t=0, x=None, res=None, total=None, y=None) == 0
    assert call(y=FAKE) == -1                                    # y and sum are not one
    assert Q.lib().quads_rmsnorm_amax_groups(0, 64) == 0
    assert Q.lib().quads_rmsnorm_amax_groups(4, 0) == 0


def test_norm_backward_validation():
    lib = Q.lib()
    f = lib.quads_rmsnorm_backward
    ws = lib.quads_rmsnorm_backward_ws(4, 64, 1)

    def call(g=FAKE, gt=1, h=FAKE, ht=1, t=4, hh=64, ldh=64, w=FAKE, wt=0, eps=1e-6, gs=None,
             dx=MORE, dt=1, dres=None, dw=FAKE, wsp=FAKE, wsz=ws):
        return f(g, gt, h, ht, t, hh, ldh, w, wt, eps, gs, dx, dt, dres, dw, wsp, wsz, None)
    assert call(t=-1) == -2 and call(hh=0) == -2 and call(ldh=63) == -2
    assert call(gt=2) == -1 and call(ht=2) == -1 and call(dt=2) == -1 and call(wt=2) == -1
    assert call(eps=0.0) == -1 and call(eps=NAN) == -1 and call(eps=9e-71) == -1
    assert call(g=None) == -1 and call(h=MIS) == -1 and call(gs=MIS) == -1 and call(dx=None) == -1
    assert call(dres=MORE) == -1 and call(dres=MIS) == -1        # dres is not dx
    assert call(dx=FAKE) == -1                                   # dx over h
    assert call(w=None) == -1 and call(dw=MIS) == -1             # dweight without a weight
    assert ws > 0 and call(wsz=ws - 1) == -3 and call(wsp=None) == -3
    assert call(t=0, g=None, h=None, dx=None, dw=None) == 0
    # in place only where the types are the same
    assert call(g=FAKE, gt=0, h=MORE, dx=FAKE) == -1
    assert call(h=MORE, gs=FAKE, dx=FAKE, dt=0, g=ctypes.c_void_p(0x30000)) == -1


def test_route_validation():
    f, b = Q.lib().quads_moe_route, Q.lib().quads_moe_route_backward

    def call(z=FAKE, dt=0, t=4, e=16, ld=16, k=2, rn=1, ids=FAKE, w=FAKE, g=FAKE, dz=MORE,
             only=None):
        r = {f(z, dt, t, e, ld, k, rn, ids, w, None)} if only != "b" else set()
        return r | ({b(z, dt, t, e, ld, ids, w, g, k, rn, dz, None)} if only != "f" else set())
    assert call(t=-1) == {-2} and call(t=1 << 24) == {-2}
    assert call(e=0) == {-2} and call(e=4097, ld=5000) == {-2} and call(ld=15) == {-2}
    assert call(k=0) == {-2} and call(k=17) == {-2} and call(e=100, ld=100, k=65) == {-2}
    assert call(dt=2) == {-1} and call(rn=2) == {-1}
    assert call(z=None, rn=0) == {-1} and call(z=MIS, rn=0) == {-1}
    assert call(ids=None) == {-1} and call(ids=MIS2) == {-1} and call(w=None) == {-1}
    assert call(g=None, only="b") == {-1} and call(dz=MIS, only="b") == {-1}
    assert call(dz=FAKE, ld=17, only="b") == {-1}                # in place: dense logits only
    assert call(t=0, z=None, ids=None, w=None, g=None, dz=None) == {0}


def test_sort_validation():
    lib = Q.lib()

    big = 1 << 25                                                # rows of 8 bf16: 512 MB
    ws = lib.quads_moe_sort_ws(big, 8, 1, 1)
    assert ws >= 4 * big and lib.quads_moe_sort_ws(big, 8, 1, 0) == 0
    assert lib.quads_moe_sort_ws(8, 8, 1, 1) == 0 and lib.quads_moe_sort_ws(0, 8, 1, 1) == 0

    def sort(x=FAKE, dt=1, t=4, h=8, ld=8, pos=FAKE, k=2, rows=8, out=MORE, zr=0, wsp=None, wsz=0):
        return lib.quads_moe_sort(x, dt, t, h, ld, pos, k, rows, zr, out, wsp, wsz, None)

    def unsort(y=FAKE, yt=1, rows=8, pos=FAKE, w=FAKE, t=4, k=2, h=8, out=MORE, ot=0):
        return lib.quads_moe_unsort(y, yt, rows, pos, w, t, k, h, out, ot, None)

    def back(g=FAKE, gt=1, y=MORE, yt=1, rows=8, pos=FAKE, w=FAKE, t=4, k=2, h=8, dy=MORE,
             dw=FAKE, zr=0, wsp=None, wsz=0):
        return lib.quads_moe_unsort_backward(g, gt, y, yt, rows, pos, w, t, k, h, zr, dy, dw, wsp,
                                             wsz, None)
    for call in (sort, unsort, back):
        assert call(t=-1) == -2 and call(t=1 << 24) == -2
        assert call(k=0) == -2 and call(k=65) == -2 and call(rows=-1) == -2
        assert call(rows=1 << 31) == -2 and call(pos=None) == -1 and call(pos=MIS2) == -1
        assert call(t=0) == 0
    assert sort(h=1 << 24, ld=1 << 24) == -2 and unsort(h=1 << 24) == -2
    assert sort(h=0, ld=0) == -2 and unsort(h=0) == -2 and back(h=0) == -2 and sort(ld=7) == -2
    assert sort(dt=2) == -1 and unsort(yt=2) == -1 and unsort(ot=2) == -1
    assert back(gt=2) == -1 and back(yt=-1) == -1
    assert sort(x=None) == -1 and sort(out=None) == -1 and sort(out=FAKE) == -1
    assert unsort(y=MIS) == -1 and unsort(out=MIS) == -1 and unsort(out=FAKE) == -1
    assert unsort(w=MIS2) == -1
    assert back(g=None) == -1 and back(y=None) == -1 and back(dy=FAKE) == -1
    assert back(w=None) == -1                                    # dw of no weights
    assert back(dw=MIS2) == -1 and back(dy=MIS) == -1
    assert back(dy=None, dw=None) == 0 and sort(rows=0) == 0
    for call in (sort, back):
        assert call(zr=2) == -1
        on = dict(zr=1, rows=big)
        if call is back:
            on["y"] = ctypes.c_void_p(0x30000)
        assert call(**on) == -3 and call(**on, wsp=FAKE, wsz=ws - 1) == -3
        assert call(**on, wsp=MIS, wsz=ws) == -3 and call(**on, t=0) == -3
    assert back(zr=1) == -1                                      # zeroing y's rows under itself
    assert back(zr=1, dy=None, dw=None) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 32), torch.zeros(2, 2)
    pos, ids = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: Q.quads_rmsnorm(x), lambda: Q.quads_rmsnorm_backward(x, x),
                 lambda: Q.quads_moe_route(x, 2), lambda: Q.quads_moe_route_backward(x, ids, w, w),
                 lambda: Q.quads_moe_sort(x, pos, 2), lambda: Q.quads_moe_unsort(x, pos, 2),
                 lambda: Q.quads_moe_unsort_backward(x, x, pos, 2, w)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    with pytest.raises(TypeError):
        Q.quads_rmsnorm([1.0])
    with pytest.raises(TypeError):
        Q.quads_moe_unsort(None, pos, 2)


def test_autograd_refusals():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="residual must have the shape"):
        qat.rms_norm(x, residual=torch.zeros(6, 8))
    with pytest.raises(TypeError):
        qat.rms_norm(x.half())
    with pytest.raises(TypeError):
        qat.route(x.double(), 2)
    with pytest.raises(ValueError, match="as many as rows says"):
        qat.unsort_tokens(x[0], torch.zeros(4, dtype=torch.int32), 2)
