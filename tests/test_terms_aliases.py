"""Arrays that a call would write while it reads them, or write twice, are refused before any CUDA
call (no GPU)."""
import ctypes

import pytest

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build()
    return api.load()


def test_new_lengths_over_what_is_read(lib):
    B = 4

    def append(lens, lens_out, begin):
        mod = api._CMod(0.0, 0, 0, None, begin)
        return lib.decode_attn_mod_append(P(16), P(16), P(16), P(16), P(16), P(lens), lens_out and P(lens_out),
                                          ctypes.byref(mod), P(16), B, 1, 1, 96, 96, 8, 0.125, 0, 0, None, 0, None, None)
    fine = -8  # (as far as the check of the head dimension, 96)
    assert append(4096, None, None) == fine
    assert append(4096, None, 4096) == fine            # both are read only
    assert append(4096, 8192, 12288) == fine
    assert append(4096, 4096 + 4 * B, None) == fine    # neighbours
    assert append(4096, 4096 - 4 * B, 4096) == fine
    for apart in (0, 4, 4 * B - 4, -4, 4 - 4 * B):
        assert append(4096, 4096 + apart, None) == -2
        assert append(8192, 4096 + apart, 4096) == -2


def test_one_array_for_keys_and_values(lib):
    s = (ctypes.c_longlong * 3)(64, 64, 64)

    def write(K=16, V=32, ks=48, vs=64):
        return lib.kv_append_q8b(P(16), P(16), s, s, api.DA_BF16, 1, None, P(K), P(V), P(ks), P(vs), 32, P(16), 1, 1, 64,
                                 8, api.DA_INT8, None, None)

    def read(k=16, v=32):
        return lib.kv_read_q8b(P(16), P(16), P(16), P(16), 32, P(16), None, P(k), P(v), api.DA_BF16, 1, 1, 1, 64, 8,
                               api.DA_INT8, None, None)
    assert write(V=16) == -2
    assert write(vs=48) == -2
    assert read(v=16) == -2
