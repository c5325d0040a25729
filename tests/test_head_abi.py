"""The output head's C ABI (include/quads_head.h) and binding on the CPU: every
declared symbol is exported, and bad arguments are refused on the host before
any launch."""

import ctypes
import os
import re

import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q
from nvfp4_w4a4_quantized_act_amd import qat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced (checks fail first)
MIS = ctypes.c_void_p(0x10004)           # misaligned for a tensor, aligned for 32-bit words
MIS2 = ctypes.c_void_p(0x10002)          # misaligned for a 32-bit word
INF, NAN = float("inf"), float("nan")


def test_library_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "quads_head.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(quads_[a-z0-9_]+)\s*\(", src))
    assert names == {"quads_moe_w4a16_gemv", "quads_moe_w4a16_gemv_ws", "quads_token_logprob",
                     "quads_token_logprob_ws", "quads_token_logprob_backward",
                     "quads_topk_distill", "quads_topk_distill_ws", "quads_topk_distill_backward",
                     "quads_topk_distill_grad", "quads_topk_distill_grad_ws"}
    lib = Q.lib()
    assert all(hasattr(lib, n) for n in names)
    assert int(re.search(r"#define QUADS_TOP_MAX (\d+)", src).group(1)) == Q.TOP_MAX


def test_gemv_validation():
    lib = Q.lib()
    f = lib.quads_moe_w4a16_gemv
    most = lib.quads_moe_w4a16_gemv_ws(8, 256, 4, 64)

    def call(rows=8, k=256, e=4, n=64, epi=0, odt=0, x=FAKE, ts=FAKE, off=FAKE, out=FAKE,
             rt=None, ws=FAKE, wsz=most):
        return f(x, rt, rows, k, FAKE, FAKE, ts, off, e, n, epi, odt, out, ws, wsz, None)
    assert call(k=250) == -2 and call(k=0) == -2
    assert call(e=0) == -2 and call(e=4097) == -2 and call(n=0) == -2
    assert call(rows=-1) == -2 and call(rows=1 << 24) == -2 and call(k=1 << 26) == -2
    assert call(epi=1, odt=1, n=63) == -2
    assert call(epi=1, odt=0) == -1 and call(epi=2) == -1 and call(odt=3) == -1
    assert call(off=None) == -1
    assert call(x=None) == -1 and call(x=MIS) == -1 and call(out=MIS) == -1
    assert call(ts=None) == -1 and call(rt=MIS2) == -1
    assert call(rows=0, x=None, out=None, ts=None) == 0
    if most:
        assert call(wsz=most - 1) == -3 and call(ws=None) == -3


def test_logprob_validation():
    lib = Q.lib()
    f = lib.quads_token_logprob
    ws = lib.quads_token_logprob_ws(4, 1000, 8)

    def call(z=FAKE, dt=0, t=4, v=1000, ld=1000, ids=FAKE, it=1.0, k=8, lp=FAKE, ent=FAKE,
             st=FAKE, tl=FAKE, ti=FAKE, wsp=FAKE, wsz=ws):
        return f(z, dt, t, v, ld, ids, it, k, lp, ent, st, tl, ti, wsp, wsz, None)
    assert call(t=-1) == -2 and call(t=1 << 24) == -2
    assert call(v=0) == -2 and call(ld=999) == -2 and call(ld=1 << 31) == -2
    assert call(v=1 << 30, ld=1 << 30) == -2
    assert call(k=129) == -2 and call(k=-1) == -2 and call(v=5, k=6) == -2
    assert call(dt=2) == -1
    for it in (0.0, -1.0, 2e30, INF, NAN):
        assert call(it=it) == -1
    assert call(z=None) == -1 and call(z=MIS) == -1 and call(ids=MIS2) == -1
    assert call(ids=None) == -1 and call(lp=None) == -1        # both or neither
    assert call(st=None) == -1 and call(tl=None) == -1 and call(ti=None) == -1
    assert call(t=0, z=None, ids=None, lp=None, st=None, tl=None, ti=None) == 0
    big = lib.quads_token_logprob_ws(1, 1 << 20, 64)
    if big:
        assert call(t=1, v=1 << 20, ld=1 << 20, k=64, wsz=big - 1) == -3
        assert call(t=1, v=1 << 20, ld=1 << 20, k=64, wsp=None, wsz=big) == -3
    g = lib.quads_token_logprob_backward

    def back(z=FAKE, ids=FAKE, it=1.0, st=FAKE, ent=FAKE, gl=FAKE, gh=FAKE, dz=FAKE, t=4, ld=1000):
        return g(z, 1, t, 1000, ld, ids, it, st, ent, gl, gh, dz, None)
    assert back(ld=10) == -2 and back(it=0.0) == -1
    assert back(ids=None) == -1 and back(ent=None) == -1       # their gradients are given
    assert back(st=None) == -1 and back(dz=None) == -1 and back(dz=MIS) == -1
    assert back(t=0, z=None, st=None, dz=None) == 0


def test_distill_validation():
    lib = Q.lib()
    f, b, c = lib.quads_topk_distill, lib.quads_topk_distill_backward, lib.quads_topk_distill_grad
    ws = lib.quads_topk_distill_ws(4, 1000, 8) + lib.quads_topk_distill_grad_ws(4, 1000, 8)

    def every(z=FAKE, dt=0, t=4, v=1000, ld=1000, tv=FAKE, ti=FAKE, k=8, w=FAKE, it=1.0, rn=1,
              out=FAKE, dz=FAKE):
        return {f(z, dt, t, v, ld, tv, ti, k, w, it, rn, out, FAKE, FAKE, ws, None),
                b(z, dt, t, v, ld, tv, ti, k, w, it, rn, FAKE, FAKE, dz if out else None, None),
                c(z, dt, t, v, ld, tv, ti, k, w, it, rn, out, dz, FAKE, ws, None)}
    assert every(k=0) == {-2} and every(k=129) == {-2}
    assert every(v=0) == {-2} and every(ld=1) == {-2} and every(t=-1) == {-2}
    assert every(dt=7) == {-1} and every(rn=2) == {-1} and every(it=NAN) == {-1}
    assert every(tv=None) == {-1} and every(ti=MIS2) == {-1} and every(w=MIS2) == {-1}
    assert every(z=MIS) == {-1} and every(out=None) == {-1}
    assert every(t=0, z=None, tv=None, ti=None, out=None, dz=None) == {0}
    assert c(FAKE, 0, 4, 1000, 1000, FAKE, FAKE, 8, None, 1.0, 1, FAKE, MIS, FAKE, ws, None) == -1
    big = lib.quads_topk_distill_ws(1, 1 << 20, 8)
    if big:
        assert f(FAKE, 0, 1, 1 << 20, 1 << 20, FAKE, FAKE, 8, None, 1.0, 1, FAKE, FAKE, FAKE,
                 big - 1, None) == -3
    big = lib.quads_topk_distill_grad_ws(1, 1 << 20, 8)
    assert lib.quads_topk_distill_grad_ws(1, 1000, 8) == 0
    assert lib.quads_topk_distill_grad_ws(64, 1 << 20, 8) == 0
    if big:
        assert c(FAKE, 0, 1, 1 << 20, 1 << 20, FAKE, FAKE, 8, None, 1.0, 1, FAKE, FAKE, FAKE,
                 big - 1, None) == -3
        assert c(FAKE, 0, 1, 1 << 20, 1 << 20, FAKE, FAKE, 8, None, 1.0, 1, FAKE, FAKE, None,
                 big, None) == -3


def test_binding_refuses_host_tensors():
    z, ids = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    tv, ti = torch.zeros(2, 3), torch.zeros((2, 3), dtype=torch.int32)
    w = (torch.zeros((1, 4, 8), dtype=torch.uint8), torch.zeros((1, 4, 1), dtype=torch.uint8),
         torch.ones(1))
    for call in (lambda: Q.quads_token_logprob(z, ids),
                 lambda: Q.quads_token_logprob_backward(z, ids, tv, None, None),
                 lambda: Q.quads_topk_distill(z, tv, ti),
                 lambda: Q.quads_topk_distill_backward(z, tv, ti, z, z),
                 lambda: Q.quads_topk_distill_grad(z, tv, ti),
                 lambda: Q.quads_moe_w4a16_gemv(torch.zeros((2, 16), dtype=torch.bfloat16), w, 4)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    with pytest.raises(TypeError):
        Q.quads_token_logprob([1.0], ids)


def test_autograd_refusals():
    z = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="ids must have the shape"):
        qat.token_logprobs(z, torch.zeros(6, dtype=torch.int32))
    with pytest.raises(ValueError, match="over the logits' rows"):
        qat.distill_loss(z, torch.zeros(6, 2), torch.zeros((6, 2), dtype=torch.int32))
    tv, ti = torch.zeros(2, 3, 2), torch.zeros((2, 3, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="one entry per row"):
        qat.distill_loss(z, tv, ti, torch.zeros(6))
    with pytest.raises(ValueError, match="no gradient"):
        qat.distill_loss(z, tv.requires_grad_(), ti)
