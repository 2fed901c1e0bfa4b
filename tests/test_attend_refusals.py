"""Refusals of kv_append_rope, chunk_attn and decode_attn_shared: all before any CUDA call (no GPU)."""
import ctypes

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

P = ctypes.c_void_p
OK = P(16)
L3 = ctypes.c_longlong * 3
BF16, FP32 = api.DA_BF16, api.DA_FP32


@pytest.fixture(scope="module")
def lib():
    build()
    return api.load()


def _rope(lib, q=OK, k=OK, s=(64, 64, 64), T=1, n_new=None, q_out=OK, so=(64, 64, 64), K=OK, V=P(32), pos=OK, cos=OK,
          sin=P(32), n_angles=8, rot=64, angle_pos=None, w=None, eps=1e-6, B=1, h_q=1, h_kv=1, d=64, d_v=None, n_max=8,
          dtype=FP32):
    st, so = L3(*s), L3(*so)
    return lib.kv_append_rope(q, k, OK, st, st, st, T, n_new, q_out, so, K, V, pos, cos, sin, n_angles, rot, 0,
                              angle_pos, w, w, eps, B, h_q, h_kv, d, d if d_v is None else d_v, n_max, dtype, None, None)


def test_rope(lib):
    for missing in ("K", "V", "pos", "cos", "sin", "q", "k", "q_out"):
        assert _rope(lib, **{missing: None}) == -1
    for bad in (api.DA_INT8, 7, BF16 | api.DA_OUT_BF16, -1):
        assert _rope(lib, dtype=bad) == -3
    for bad in (dict(B=0), dict(h_q=0), dict(h_kv=0), dict(T=-1), dict(n_max=0), dict(n_max=(1 << 30) + 1),
                dict(n_angles=0), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=80), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(B=1 << 20, n_max=1 << 12), dict(T=(1 << 30) + 1),
                dict(V=OK), dict(sin=OK), dict(s=(-64, 64, 64)), dict(so=(64, 64, 1 << 40)),
                dict(B=1 << 20, h_q=1 << 10, T=1 << 10, n_max=8)):
        assert _rope(lib, **bad) == -2, bad
    for bad in (dict(q=P(8)), dict(k=P(20)), dict(K=P(24)), dict(cos=P(8)), dict(pos=P(18)), dict(n_new=P(17)),
                dict(angle_pos=P(18)), dict(w=P(8)), dict(s=(64, 64, 2)), dict(so=(64, 64, 66))):
        assert _rope(lib, **bad) == -4, bad
    for d, d_v in ((96, 96), (64, 128), (128, 64), (192, 192), (512, 512)):
        assert _rope(lib, d=d, d_v=d_v) == -8
    assert _rope(lib, T=0, q=None, k=None, q_out=None) == 0     # nothing to do


def _chunk(lib, q=OK, K=OK, V=OK, lens=OK, n_new=None, out=OK, s=(64, 64, 64), so=(64, 64, 64), T=1, window=0, prefix=0,
           B=1, h_q=1, h_kv=1, d=64, n_max=8, scale=0.125, dtype=BF16):
    return lib.chunk_attn(q, L3(*s), T, n_new, K, V, lens, window, prefix, out, L3(*so), B, h_q, h_kv, d, n_max, scale,
                          dtype, None, 0, None, None)


def test_chunk(lib):
    for missing in ("q", "K", "V", "lens", "out"):
        assert _chunk(lib, **{missing: None}) == -1
    for bad in (api.DA_INT8, api.DA_FP8_E4M3, 9, BF16 | 0x200):
        assert _chunk(lib, dtype=bad) == -3
    for bad in (dict(dtype=FP32), dict(d=96), dict(d=256), dict(d=192)):
        assert _chunk(lib, **bad) == -8, bad
    for bad in (dict(B=0), dict(h_q=3, h_kv=2), dict(n_max=0), dict(T=-1), dict(window=-1), dict(prefix=-1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3.4e38), dict(s=(64, -64, 64)),
                dict(T=1 << 28, h_q=8), dict(T=(1 << 30) + 1), dict(B=1 << 16, n_max=1 << 16)):
        assert _chunk(lib, **bad) == -2, bad
    for bad in (dict(q=P(8)), dict(K=P(8)), dict(out=P(8)), dict(lens=P(18)), dict(n_new=P(18)), dict(s=(64, 64, 4)),
                dict(so=(64, 64, 2))):
        assert _chunk(lib, **bad) == -4, bad
    assert _chunk(lib, so=(64, 64, 4), dtype=BF16 | api.DA_OUT_BF16) == -4   # 8 bytes
    assert _chunk(lib, T=0, q=None, out=None) == 0
    st = ctypes.c_int(0)
    for dtype, d, want in ((FP32, 64, -8), (api.DA_INT8, 64, -3), (BF16, 256, -8)):
        assert lib.chunk_attn_workspace_bytes(1, 1, 1, 1, d, 8, dtype, ctypes.byref(st)) == 0
        assert st.value == want


def _shared(lib, q=OK, Kp=OK, Vp=OK, n=8, most=8, K=OK, V=OK, lens=OK, out=OK, B=1, h_q=1, h_kv=1, d=64, n_max=8,
            scale=0.125, dtype=BF16):
    return lib.decode_attn_shared(q, Kp, Vp, n, most, K, V, lens, out, B, h_q, h_kv, d, n_max, scale, dtype, None, 0,
                                  None, None)


def test_shared(lib):
    for missing in ("q", "Kp", "Vp", "K", "V", "lens", "out"):
        assert _shared(lib, **{missing: None}) == -1
    for bad in (dict(n=-1), dict(n=9), dict(most=0, n=0), dict(most=(1 << 30) + 1), dict(h_q=3, h_kv=2), dict(B=0),
                dict(h_q=8, h_kv=8, most=1 << 29), dict(scale=float("nan"))):
        assert _shared(lib, **bad) == -2, bad
    for bad in (dict(Kp=P(8)), dict(Vp=P(24)), dict(q=P(8)), dict(lens=P(17))):
        assert _shared(lib, **bad) == -4, bad
    assert _shared(lib, dtype=FP32) == -8
    assert _shared(lib, dtype=api.DA_INT8) == -3
    assert _shared(lib, d=256) == -8
    st = ctypes.c_int(0)
    lib.decode_attn_shared_workspace_bytes(1, 1, 1, 64, 8, -1, BF16, ctypes.byref(st))
    assert st.value == -2


def test_binding_checks():
    """The binding refuses what the C entry points cannot see: shapes, types, devices, overlaps."""
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i = torch.zeros(2, dtype=torch.int32)
    cs = torch.zeros(9, 32)
    with pytest.raises(ValueError):   # not on a GPU
        api.kv_append_rope(z(2, 4, 1, 64), z(2, 2, 1, 64), z(2, 2, 1, 64), z(2, 2, 9, 64), z(2, 2, 9, 64), i, cs, cs)
    with pytest.raises(ValueError):
        api.chunk_attn(z(2, 4, 1, 64), z(2, 2, 9, 64), z(2, 2, 9, 64), i)
    with pytest.raises(ValueError):
        api.decode_attn_shared(z(2, 4, 64), z(2, 9, 64), z(2, 9, 64), z(2, 2, 9, 64), z(2, 2, 9, 64), i)
    rows = lambda t, write: api._row_strides("x", t, t.shape, t.dtype, -1, write)  # noqa: E731
    assert list(rows(z(2, 5, 4, 64).transpose(1, 2), True)) == [1280, 64, 256]
    assert list(rows(z(1, 4, 64).expand(3, 4, 64).unsqueeze(1), False)) == [0, 0, 64]
    for bad in (z(1, 4, 8, 64).expand(3, 4, 8, 64), z(2, 4, 9 * 64).as_strided((2, 4, 9, 64), (2304, 576, 32, 1))):
        with pytest.raises(ValueError, match="overlap"):
            rows(bad, True)
    with pytest.raises(ValueError, match="last dimension"):
        rows(z(2, 4, 8, 128)[..., ::2], False)
