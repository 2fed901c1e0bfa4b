"""Refusals of the score-term and block-scale entry points: all before any CUDA call (no GPU)."""
import ctypes

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

P = ctypes.c_void_p
OK = P(16)


@pytest.fixture(scope="module")
def lib():
    build()
    return api.load()


def _cmod(softcap=0.0, window=0, prefix=0, slopes=None, begin=None):
    return api._CMod(softcap, window, prefix, slopes, begin)


def _mod(lib, mod=None, q=OK, K=OK, dtype=0, d_k=64, d_v=64, h_q=1, h_kv=1, n_max=8, scale=0.125):
    m = None if mod is None else ctypes.byref(mod)
    return lib.decode_attn_mod(q, K, OK, OK, m, OK, 1, h_q, h_kv, d_k, d_v, n_max, scale, dtype, 0,
                               None, 0, None, None)


def test_score_terms(lib):
    inf, nan = float("inf"), float("nan")
    assert _mod(lib) == -1                                     # terms are required
    for bad in (-1.0, inf, -inf, nan, 1e-31, 1e31):
        assert _mod(lib, _cmod(softcap=bad)) == -2
    assert _mod(lib, _cmod(window=-1)) == -2
    assert _mod(lib, _cmod(prefix=-1)) == -2
    assert _mod(lib, _cmod(slopes=18)) == -4
    assert _mod(lib, _cmod(begin=17)) == -4
    assert _mod(lib, _cmod(), q=None) == -1
    assert _mod(lib, _cmod(), K=P(8)) == -4
    assert _mod(lib, _cmod(), dtype=api.DA_INT8) == -3         # 8-bit caches have entry points of their own
    assert _mod(lib, _cmod(), dtype=9) == -3
    assert _mod(lib, _cmod(), d_k=96, d_v=96) == -8
    assert _mod(lib, _cmod(), d_k=256, d_v=256) == -8          # bf16 only
    assert _mod(lib, _cmod(), h_q=3, h_kv=2) == -2
    assert _mod(lib, _cmod(), n_max=0) == -2
    assert _mod(lib, _cmod(), scale=nan) == -2
    assert _mod(lib, _cmod(softcap=1e-30), scale=1e10) == -2   # scale / softcap overflows
    assert _mod(lib, _cmod(softcap=1e-30), scale=2e8) == -2    # 2 log2(e) of it does
    m = ctypes.byref(_cmod())

    def app(k_new=OK, lens_out=None, mod=m):
        return lib.decode_attn_mod_append(OK, k_new, OK, OK, OK, OK, lens_out, mod, OK, 1, 1, 1, 64,
                                          64, 8, 0.125, 0, 0, None, 0, None, None)
    assert app(k_new=None) == -1
    assert app(k_new=P(8)) == -4
    assert app(lens_out=OK) == -2                              # seq_lens itself
    assert app(mod=None) == -1
    st = ctypes.c_int(0)
    assert lib.decode_attn_mod_workspace_bytes(None, 1, 1, 1, 64, 64, 8, 0, 0, ctypes.byref(st)) == 0
    assert st.value == -1
    lib.decode_attn_mod_workspace_bytes(m, 1, 1, 1, 64, 64, 8, api.DA_INT8, 0, ctypes.byref(st))
    assert st.value == -3


def test_block_scaled_decode(lib):
    def q8b(dtype=api.DA_INT8, ks=OK, block=64, d=64, K=OK, n_max=7, mod=None):
        return lib.decode_attn_q8b(OK, K, OK, ks, OK, block, OK, mod, OK, 1, 1, 1, d, d, n_max, 0.125,
                                   dtype, 0, None, 0, None, None)
    assert q8b(dtype=api.DA_BF16) == -3
    assert q8b(ks=None) == -1
    assert q8b(ks=P(18)) == -4
    assert q8b(K=P(8)) == -4
    for block in (0, 1, 8, 24, 48, 256, -16):
        assert q8b(block=block) == -2
    assert q8b(d=96) == -8
    assert q8b(d=256) == -8
    assert q8b(n_max=0) == -2
    assert q8b(mod=ctypes.byref(_cmod(window=-2))) == -2
    st = ctypes.c_int(0)
    lib.decode_attn_q8b_workspace_bytes(None, 1, 1, 1, 64, 64, 8, api.DA_FP32, 0, ctypes.byref(st))
    assert st.value == -3


def test_write_and_read(lib):
    L3 = ctypes.c_longlong * 3

    def app(k=OK, strides=(64, 64, 64), x=api.DA_BF16, T=1, K=OK, block=32, pos=OK, B=1, d=64, n_max=8,
            dtype=api.DA_INT8, n_new=None):
        s = L3(*strides)
        return lib.kv_append_q8b(k, OK, s, s, x, T, n_new, K, OK, OK, OK, block, pos, B, 1, d, n_max,
                                 dtype, None, None)
    assert app(k=None) == -1
    assert app(K=None) == -1
    assert app(pos=None) == -1
    assert app(x=api.DA_INT8) == -3
    assert app(dtype=api.DA_BF16) == -3
    assert app(T=-1) == -2
    assert app(T=0) == 0                                       # nothing to do
    assert app(B=0) == -2
    assert app(n_max=0) == -2
    assert app(B=1 << 20, n_max=1 << 20) == -2
    assert app(block=10) == -2
    assert app(d=80) == -8
    assert app(k=P(8)) == -4
    assert app(strides=(64, 64, 65)) == -4                     # rows off the 16-byte grid
    assert app(strides=(-64, 64, 64)) == -2
    assert app(n_new=P(18)) == -4

    def read(K=OK, out=OK, out_dtype=api.DA_BF16, T=1, block=32, d=64, dtype=api.DA_INT8, begin=None):
        return lib.kv_read_q8b(K, OK, OK, OK, block, OK, begin, out, OK, out_dtype, T, 1, 1, d, 8, dtype,
                               None, None)
    assert read(K=None) == -1
    assert read(out=None) == -1
    assert read(out_dtype=api.DA_FP8_E4M3) == -3
    assert read(dtype=api.DA_FP32) == -3
    assert read(T=-1) == -2
    assert read(T=0) == 0
    assert read(T=(1 << 30) + 1) == -2
    assert read(block=100) == -2
    assert read(d=32) == -8
    assert read(out=P(8)) == -4
    assert read(begin=P(18)) == -4


def test_binding_checks_tensors(lib):
    """The binding refuses before it touches a device: CPU tensors, wrong shapes and types."""
    q = torch.zeros(1, 2, 64)
    K = torch.zeros(1, 1, 8, 64)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.decode_attn_mod(q, K, K, lens, api.ScoreMod())
    codes = torch.zeros(1, 1, 8, 64, dtype=torch.int8)
    scale = torch.zeros(1, 1, 1)
    for block in (0, 17, 256):
        with pytest.raises(ValueError, match="block"):
            api.kv_append_q8b(q, q, codes, codes, scale, scale, lens, block=block)
    with pytest.raises(ValueError):
        api.kv_read_q8b(codes, codes, scale, scale, lens, block=16)
    with pytest.raises(ValueError):
        api.decode_attn_q8b(q, codes, codes, scale, scale, lens, block=16)
    with pytest.raises(ValueError, match="slopes"):
        api._c_mod(api.ScoreMod(slopes=torch.zeros(3)), 1, 2, 0)
    with pytest.raises(ValueError, match="doc_begin"):
        api._c_mod(api.ScoreMod(doc_begin=torch.zeros(1)), 1, 2, 0)
    with pytest.raises(ValueError, match="window"):
        api._c_mod(api.ScoreMod(window=-1), 1, 2, -1)
    with pytest.raises(ValueError, match="window"):
        api._c_mod(api.ScoreMod(prefix=1 << 31), 1, 2, -1)
