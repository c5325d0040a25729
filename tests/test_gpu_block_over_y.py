"""The gradient of the way back with dy over y (through the C ABI), at widths whose last,
partial eight channels stand in another wave, or in another turn over the row, than the
eight before: the bits of the call that writes dy elsewhere, every time."""

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_act_amd as Q
from oracle import block as OB
from oracle import moe as OM

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("h", [3, 61, 127, 250, 511, 513, 519, 700, 1025, 1031, 2049, 2055, 4097, 4099, 8191,
                               8193, 8199, 8201, 8705, 16385])
def test_dy_over_y(h):
    rng = np.random.default_rng(h)
    for t, k, gt, yt in ((40, 4, "bf16", "bf16"), (3, 9, "f32", "f32"), (300, 1, "f32", "bf16"),
                         (600, 2, "bf16", "f32")):
        print(f"gradient over y T={t} H={h} topk={k} g={gt} y={yt}", flush=True)
        ids = np.argsort(-rng.normal(size=(t, 16)), axis=1)[:, :k]
        pos = OM.pack_routes(ids, 16)[2].astype(np.int32)
        pos[rng.random(pos.shape) < 0.1] = -1
        n = t * k
        posn, pos = pos, torch.from_numpy(pos).to(DEV)
        g = torch.from_numpy(rng.normal(size=(t, h)).astype(np.float32)).to(TYPES[gt]).to(DEV)
        y = torch.from_numpy(rng.normal(size=(n, h)).astype(np.float32)).to(TYPES[yt]).to(DEV)
        w = torch.from_numpy(rng.random((t, k)).astype(np.float32)).to(DEV)
        dy, dw = Q.quads_moe_unsort_backward(g, y, pos, k, w, rows=n)
        want = y.clone()                                         # a row without a slot stays
        named = pos[pos >= 0].long()
        want[named] = dy[named]
        for _ in range(3):
            over, dw2 = y.clone(), torch.empty_like(w)
            torch.cuda.synchronize()
            assert Q.lib().quads_moe_unsort_backward(
                g.data_ptr(), int(gt == "bf16"), over.data_ptr(), int(yt == "bf16"), n, pos.data_ptr(),
                w.data_ptr(), t, k, h, 0, over.data_ptr(), dw2.data_ptr(), None, 0, None) == 0
            torch.cuda.synchronize()
            assert torch.equal(over, want) and torch.equal(dw, dw2)
        _, edw, size = OB.unsort_grad(g.double().cpu().numpy(), y.double().cpu().numpy(), posn, k,
                                      w.double().cpu().numpy())
        # a thread adds up at most H / 64 + 16 products before at most 8 (16 waves: 15) more sums
        assert np.all(np.abs(dw.double().cpu().numpy() - edw) <= (h / 64 + 40) * U * size + 2.0 ** -126)
