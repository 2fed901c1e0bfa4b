"""Outputs of kv_append_rope and chunk_attn over their inputs are refused, layouts that only lie close are not (no GPU:
what is not refused ends at the missing device; with one the calls' made-up addresses would be used)."""
import ctypes
import random

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
P, L3 = ctypes.c_void_p, ctypes.c_longlong * 3
SHAPE = -2
D, ES = 64, 2       # bf16 heads of 64
FAR = 1 << 40       # where what is not looked at lies


@pytest.fixture(scope="module")
def lib():
    build()
    return api.load()


def rows(at, strides, B, h, T):
    """The 16-byte pieces of a tensor's rows."""
    return {at // 16 + (b * strides[0] + x * strides[1] + i * strides[2]) * ES // 16 + k
            for b in range(B) for x in range(h) for i in range(T) for k in range(D * ES // 16)}


def rope(lib, B, h_q, h_kv, T, n_max, q, k, v, out, K, V, pos=FAR, cos=2 * FAR, w=3 * FAR):
    """q, k, v, out: (address, strides)."""
    return lib.kv_append_rope(P(q[0]), P(k[0]), P(v[0]), L3(*q[1]), L3(*k[1]), L3(*v[1]), T, None, P(out[0]), L3(*out[1]),
                              P(K), P(V), P(pos), P(cos), P(cos + FAR // 2), 8, 64, 0, None, P(w), P(w), 1e-6, B, h_q, h_kv,
                              D, D, n_max, api.DA_BF16, None, None)


def test_projections(lib):
    """The layouts that programs have: one projection's columns, in place or not; token or head first."""
    B, h_q, h_kv, T, n_max = 3, 4, 2, 5, 9
    w = (h_q + 2 * h_kv) * D
    at = 1 << 20
    st = (T * w, D, w)
    q, k, v = (at, st), (at + h_q * D * ES, st), (at + (h_q + h_kv) * D * ES, st)
    K, V = 1 << 30, 1 << 31
    go = lambda **kw: rope(lib, **{**dict(B=B, h_q=h_q, h_kv=h_kv, T=T, n_max=n_max, q=q, k=k, v=v,  # noqa: E731
                                          out=(1 << 33, (T * h_q * D, D, h_q * D)), K=K, V=V), **kw})
    assert go() != SHAPE
    assert go(out=q) != SHAPE                                            # in place
    assert go(out=(at, (h_q * T * D, T * D, D))) == SHAPE                # on q with other strides
    assert go(out=k) == SHAPE and go(out=v) == SHAPE
    assert go(out=(at + 16, st)) == SHAPE                                # 16 bytes on
    assert go(out=(at + w * ES, st)) == SHAPE                            # a token on
    # q and q_out as halves of one buffer's columns
    two = (T * 2 * h_q * D, D, 2 * h_q * D)
    assert go(q=(1 << 35, two), out=((1 << 35) + h_q * D * ES, two)) != SHAPE
    assert go(q=(1 << 35, two), out=((1 << 35) + (h_q - 1) * D * ES, two)) == SHAPE
    # caches
    size = B * h_kv * n_max * D * ES
    assert go(V=K + size) != SHAPE and go(V=K + size - 16) == SHAPE and go(V=K - size + 16) == SHAPE
    for x in (K, V, V + size - 16):
        assert go(out=(x, (T * h_q * D, D, h_q * D))) == SHAPE
        assert go(k=(x, st)) == SHAPE and go(v=(x, st)) == SHAPE and go(q=(x, st)) == SHAPE
        assert go(pos=x) == SHAPE and go(cos=x) == SHAPE and go(w=x) == SHAPE
    assert go(out=(K - T * B * h_q * D * ES, (T * h_q * D, D, h_q * D))) != SHAPE
    # heads of 192 and values of 128 in one projection, in place
    w = h_q * 192 + h_kv * (192 + 128)
    s3, sv = L3(T * w, 192, w), L3(T * w, 128, w)
    big = 1 << 36

    def mixed(out, so):
        return lib.kv_append_rope(P(at), P(at + h_q * 192 * ES), P(at + (h_q + h_kv) * 192 * ES), s3, s3, sv, T, None, P(out),
                                  so, P(big), P(2 * big), P(3 * big), P(4 * big), P(5 * big), 8, 64, 0, None, None, None,
                                  1e-6, B, h_q, h_kv, 192, 128, n_max, api.DA_BF16, None, None)
    assert mixed(at, s3) != SHAPE and mixed(at, s3) != -8
    assert mixed(at + (h_q + h_kv) * 192 * ES, sv) == SHAPE


def layouts(rng, B, h, T, base):
    """Strides of rows in some order of their dimensions, with gaps; an address near the base."""
    order, strides, step = rng.sample(range(3), 3), [0] * 3, D
    for i in order:
        strides[i] = step + 8 * rng.choice([0, 0, 8, 24])
        step = strides[i] * (B, h, T)[i]
    return base + 16 * rng.randrange(0, 3000), tuple(strides)


def test_any_layouts(lib):
    """Against the sets of pieces: refused when q_out meets q, k or v."""
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(1500):
        B, h_q, h_kv, T = (rng.randint(1, 3) for _ in range(4))
        q, out = (layouts(rng, B, h_q, T, 1 << 20) for _ in range(2))
        k, v = (layouts(rng, B, h_kv, T, 1 << 20) for _ in range(2))
        if rng.random() < 0.4:            # of one buffer, some columns on
            B, h_q, T = 2, 2, 3
            w = D * rng.randint(4, 9)
            st = (T * w, D, w)
            q, out = ((1 << 20) + D * ES * rng.randint(0, 6) for _ in range(2))
            q, out = (q, st), (out, st)
            k, v = (1 << 25, st), (1 << 26, st)
        mine = rows(*out, B, h_q, T)
        same = out[0] == q[0] and all(a == b or n == 1 for a, b, n in zip(out[1], q[1], (B, h_q, T)))
        meets = bool(mine & (rows(*k, B, h_kv, T) | rows(*v, B, h_kv, T))) or (not same and bool(mine & rows(*q, B, h_q, T)))
        seen[meets] += 1
        got = rope(lib, B, h_q, h_kv, T, 9, q, k, v, out, 1 << 30, 1 << 31)
        assert (got == SHAPE) == meets, (q, k, v, out, B, h_q, h_kv, T)
    assert min(seen) > 300


def test_chunk(lib):
    B, h_q, h_kv, T, n_max = 2, 4, 2, 5, 9
    st, at, K, V = (T * h_q * D, D, h_q * D), 1 << 20, 1 << 30, 1 << 31
    size = B * h_kv * n_max * D * ES

    def go(out, so=st, dtype=api.DA_BF16 | api.DA_OUT_BF16, lens=FAR, n_new=None):
        return lib.chunk_attn(P(at), L3(*st), T, None if n_new is None else P(n_new), P(K), P(V), P(lens), 0, 0, P(out),
                              L3(*so), B, h_q, h_kv, D, n_max, 0.125, dtype, None, 0, None, None)
    total = B * T * h_q * D
    assert go(1 << 33) != SHAPE and go(1 << 33, dtype=api.DA_BF16) != SHAPE
    assert go(at + total * ES) != SHAPE and go(at + total * ES - 16) == SHAPE
    assert go(at - total * 4, dtype=api.DA_BF16) != SHAPE and go(at - total * 4 + 16, dtype=api.DA_BF16) == SHAPE
    assert go(at) == SHAPE
    for x in (K, V, K + size - 16, V + size - 16):
        assert go(x) == SHAPE
    assert go(K + size) != SHAPE
    assert go(1 << 33, lens=(1 << 33) + 4) == SHAPE and go(1 << 33, n_new=1 << 33) == SHAPE
