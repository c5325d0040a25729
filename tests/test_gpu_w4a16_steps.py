"""More of the W4A16 product on the GPU against oracle/head.py in fp64
(tolerance: test_gpu_w4a16): work-groups that bring their activations in parts
and do so again for every step of features."""

import numpy as np
import pytest

from test_gpu_w4a16 import acts, check, codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    import nvfp4_w4a4_quantized_act_amd as lib
    lib.lib()
    return lib


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows,k,n", [(1024, 5120, 2100), (1000, 4624, 2102)])
def test_activations_in_parts_and_steps(Q, rows, k, n, swiglu):
    """A unit of 16 rows of more than 4608 channels does not fit in LDS, and 63 or 64 units leave
    each slot of 8 work-groups a unit more features than one step takes (64 slots for 2100 or, of
    a SwiGLU's outputs, 1050 features)."""
    w = codes(n, 1, n, k)
    if swiglu:
        w = w[0], w[1], w[2] * np.float32(0.02)
    check(Q, acts(rows, rows, k), w, swiglu=swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_experts_in_parts_and_steps(Q, swiglu):
    """The same for experts, one without rows and one whose last unit has one row."""
    e, k, n = 5, 5136, 4100
    counts = [321, 0, 160, 17, 16]
    off = np.concatenate([[0], np.cumsum(counts)])
    w = codes(3, e, n, k)
    check(Q, acts(4, int(off[-1]), k), (w[0], w[1], w[2] * np.float32(0.02)), off, swiglu=swiglu)
