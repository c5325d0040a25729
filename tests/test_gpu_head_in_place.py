"""Gradients written over the logits where a row is shared by several
work-groups: the same bits as into a tensor of their own."""

import pytest
import torch

from test_gpu_head import DEV, lists, make, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v,ld", [(3, 200001, None), (2, 300007, 300016), (40, 140001, None),
                                    (1, 1000003, None), (9, 20000, None)])
def test_split_rows_in_place(Q, t, v, ld, dtype):
    print(f"in place T={t} V={v} ld={ld} {dtype}", flush=True)
    z, zr = make(t, v, dtype, seed=v, ld=ld)
    ids = torch.from_numpy(tokens(zr, 1)).to(DEV)
    tv, ti = (torch.from_numpy(a).to(DEV) for a in lists(zr, 100, 3, 1.0, True))
    ti[0, ::7] = torch.arange(0, v, v // 15, dtype=torch.int32, device=DEV)[: len(ti[0, ::7])]
    g = torch.linspace(0.5, -1.5, t, device=DEV)
    r = Q.quads_token_logprob(z, ids)
    loss, st = Q.quads_topk_distill(z, tv, ti)

    def calls(x, out):
        return [("logprob", lambda: Q.quads_token_logprob_backward(x, ids, r["stats"], r["entropy"],
                                                                   g, g, out=out)),
                ("distill", lambda: Q.quads_topk_distill_backward(x, tv, ti, st, g, out=out)),
                ("both", lambda: Q.quads_topk_distill_grad(x, tv, ti, out=out)[1])]
    want = {name: call() for name, call in calls(z, None)}
    for i in range(3):
        full = torch.full((t, ld or v), 3.0, dtype=z.dtype, device=DEV)
        x = full[:, :v]
        x.copy_(z)
        name, call = calls(x, x)[i]
        got = call()
        torch.cuda.synchronize()
        assert got.data_ptr() == x.data_ptr() and torch.equal(got, want[name]), name
        assert bool((full[:, v:] == 3.0).all())
