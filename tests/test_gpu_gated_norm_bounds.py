"""Rows that are not whole 16-byte pieces are held in registers like others: the bounds of test_gpu_gated_norm.py
for such rows, not doubled, up to the lengths where that form ends."""
import numpy as np
import pytest

from test_gpu_gated_norm import DEV, TYPES, call, compare, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 5), (5, 33), (530, 111), (40, 1001), (300, 1111), (7, 2047), (33, 3001), (3, 4100), (5, 7001), (2, 8191)])
def test_odd_rows(T, d, dtype):
    import routing_grouped_expert_gemm_amd as mok
    t = TYPES[dtype]
    for gate in ("row", "all"):
        a = inputs(T, d, dtype, gate, True, True, seed=5)
        D = {k: v.to(DEV) for k, v in a.items()}
        compare(a, call(mok, D, T, d, t, 0.875, -0.7), t, 1, np.float32(0.875), np.float32(-0.7))
