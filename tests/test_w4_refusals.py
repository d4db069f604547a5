"""Counts whose products leave 64 bits are refused by the 4-bit weights' entry points, checked without a GPU
(pointers here are never followed)."""
import ctypes

import pytest

from test_block_refusals import EINVAL, EUNSUPPORTED, I32, I64, P, moe_args


@pytest.fixture(scope="module")
def mok():
    import routing_grouped_expert_gemm_amd as m
    return m


def test_tokens_past_64_bits(mok):
    lib = ctypes.CDLL(mok.LIB_PATH)
    lib.mok_moe_w4_forward.argtypes = [ctypes.POINTER(mok.MoeW4Args), P]
    for T, k in ((1 << 62, 4), (1 << 60, 16), ((1 << 62) + 1, 4), (1 << 31, 1), (1 << 58, 2)):
        a = moe_args(mok, T=T, E=64, k=k)
        assert lib.mok_moe_w4_forward(ctypes.byref(a), None) == EINVAL, (T, k)
        with pytest.raises(mok.MokError) as e:
            mok.mok_moe_w4_workspace_bytes(a)
        assert e.value.status == EINVAL


def test_quantised_rows_past_64_bits(mok):
    lib = ctypes.CDLL(mok.LIB_PATH)
    lib.mok_quantize_int4.argtypes = [P, I64, I32, I32, P, P, P, P]
    for rows in (1 << 62, (1 << 62) + 1, 1 << 61, 1 << 32):
        assert lib.mok_quantize_int4(16, rows, 256, 64, 16, 16, None, None) == EUNSUPPORTED, rows
