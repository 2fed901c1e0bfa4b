"""The flag for weights of one bf16: only beside a bf16 output, only of the operators that know it (no GPU)."""
import ctypes

import pytest

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

P, L3 = ctypes.c_void_p, ctypes.c_longlong * 3
OK = P(16)
BF16, OUT, NARROW, FP32 = api.DA_BF16, api.DA_OUT_BF16, api.DA_BF16_WEIGHTS, api.DA_FP32


@pytest.fixture(scope="module")
def lib():
    build()
    return api.load()


@pytest.mark.parametrize("dtype,want", [(BF16 | NARROW, -3), (FP32 | NARROW, -3), (FP32 | OUT | NARROW, -8),
                                        (api.DA_INT8 | OUT | NARROW, -3), (BF16 | OUT | NARROW | 0x200, -3),
                                        (BF16 | OUT | NARROW, 0)])
def test_attention(lib, dtype, want):
    st, s = ctypes.c_int(0), L3(64, 64, 64)
    assert lib.chunk_attn(None, s, 0, None, OK, OK, OK, 0, 0, None, s, 1, 1, 1, 64, 8, 0.125, dtype, None, 0, None, None) == want
    if want:
        assert lib.decode_attn_shared(OK, OK, OK, 8, 8, OK, OK, OK, OK, 1, 1, 1, 64, 8, 0.125, dtype, None, 0, None, None) == want
        for query, more in ((lib.chunk_attn_workspace_bytes, (1, 1, 1, 1, 64, 8)),
                            (lib.decode_attn_shared_workspace_bytes, (1, 1, 1, 64, 8, 8))):
            assert query(*more, dtype, ctypes.byref(st)) == 0
            assert st.value == want


def test_others(lib):
    """The other entry points refuse it as the unknown type that it is to them."""
    st = ctypes.c_int(0)
    lib.decode_attn_workspace_bytes(1, 1, 1, 64, 64, 8, BF16 | OUT | NARROW, 0, ctypes.byref(st))
    assert st.value == -3
