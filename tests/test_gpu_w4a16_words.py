"""Operands of the W4A16 product that are arrays of 32-bit words may start at any
word (tolerance: test_gpu_w4a16)."""

import numpy as np
import pytest
import torch

from test_gpu_w4a16 import DEV, acts, check, codes, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


def test_words_at_any_address(Q):
    """Tensor scales, offsets and row indices are read by the word: slices of larger arrays."""
    e, k, n = 4, 256, 66
    w = codes(7, e, n, k)
    x = acts(7, 9, k)
    off = np.array([0, 2, 2, 5, 9], np.int32)
    rt = np.array([3, 1, 8, 0, 0, 2, 5, 7, 6], np.int32)
    want = check(Q, x, w, off, rt)
    one = lambda a: torch.cat([a[:1], a])[1:]
    wt = tuple(up(a) for a in w)
    args = dict(offsets=one(up(off)), row_token=one(up(rt)))
    assert all(a.data_ptr() % 16 == 4 for a in args.values())
    got = Q.quads_moe_w4a16_gemv(up(x), (wt[0], wt[1], one(wt[2])), n, **args)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    # experts 1 .. 3 of a layer, as views
    got = Q.quads_moe_w4a16_gemv(up(x[:3]), tuple(a[1:] for a in wt), n,
                                 offsets=torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(got, check(Q, x[:3], tuple(a[1:] for a in w), [0, 1, 2, 3]))
