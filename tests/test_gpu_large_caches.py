"""Caches whose rows lie more than 2^32 bytes from their start (needs a GB300)."""
import math

import pytest
import torch

import decode_bounds as D
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_block_scaled_cache():
    """Written near its end, read back and attended: as a cache of its last rows alone, and against
    64 bits."""
    B, h_q, h, n, d, block = 3, 16, 8, 1500000, 128, 32
    K, V = (torch.randint(-127, 128, (B, h, n, d), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-8, -4, (B, h, n // block), device="cuda").float()) for _ in range(2))
    base = (n - 4096) // block * block
    tail = [t.contiguous().clone() for t in (K[:, :, base:], V[:, :, base:], ks[:, :, base // block:], vs[:, :, base // block:])]
    x = [4 * torch.randn(B, h, 90, d, device="cuda").to(torch.bfloat16) for _ in range(2)]
    pos = [n - 90, n - 1000, n - 4000]
    api.kv_append_q8b(x[0], x[1], K, V, ks, vs, i32(pos), block)
    api.kv_append_q8b(x[0], x[1], *tail, i32([p - base for p in pos]), block)
    for t, s in zip((K[:, :, base:], V[:, :, base:], ks[:, :, base // block:], vs[:, :, base // block:]), tail):
        assert torch.equal(t, s)
    lens, begin = [p + 90 for p in pos], [p - 60 for p in pos]
    got = api.kv_read_q8b(K, V, ks, vs, i32(lens), block, rows=150, row_begin=i32(begin), out_dtype=torch.float32)
    want = api.kv_read_q8b(*tail, i32([n - base for n in lens]), block, rows=150, row_begin=i32([b - base for b in begin]),
                           out_dtype=torch.float32)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and b.any()
    q = torch.randn(B, h_q, d, device="cuda").to(torch.bfloat16)
    part = D.weight_rounding("q8b")
    at = torch.arange(n - base, device="cuda") // block
    Kv, Vv = (tail[i].double() * tail[i + 2][:, :, at, None].double() for i in range(2))
    for window, splits in ((90, 0), (90, 3), (3000, 0), (3000, 7)):
        lens = [n, n - 5, n - 910]
        out = api.decode_attn_q8b(q, K, V, ks, vs, i32(lens), block, mod=ScoreMod(window=window), num_splits=splits)
        ref, tol = D.attend(q, Kv, Vv, [m - base for m in lens], d ** -0.5, part, window=window, floor=2.0 ** -31)
        D.check(out, ref, tol, f"window {window} splits {splits}")
    del Kv, Vv
    out = api.decode_attn_q8b(q, K, V, ks, vs, i32([0, 0, n]), block)
    assert not out[:2].any()
    at = torch.arange(n, device="cuda") // block
    for k in (0, h - 1):
        heads = slice(2 * k, 2 * k + 2)
        ref, tol = D.attend(q[2:, heads], (K[2, k].double() * ks[2, k][at, None].double())[None, None],
                            (V[2, k].double() * vs[2, k][at, None].double())[None, None], [n], d ** -0.5, part, floor=2.0 ** -31)
        D.check(out[2:, heads], ref, tol)


@pytest.mark.parametrize("h_q,h,d,dtype", [(16, 8, 128, torch.bfloat16), (32, 2, 128, torch.bfloat16),
                                          (16, 8, 64, torch.float32)], ids=["bf16", "tc5", "fp32"])
def test_score_terms(h_q, h, d, dtype):
    """A fused append at the last rows of the last heads, over a window and over everything."""
    B = 3
    n = (13 << 29) // (B * h * d * torch.finfo(dtype).bits // 8)  # 6.5 * 2^30 bytes a tensor
    K, V = (torch.randn(B * h * d, 1, device="cuda").to(dtype).view(B, h, 1, d).repeat(1, 1, n, 1) for _ in range(2))
    K[:, :, -4000:], V[:, :, -4000:] = (torch.randn(B, h, 4000, d, device="cuda").to(dtype) for _ in range(2))
    kn, vn = (torch.randn(B, h, d, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(B, h_q, d, device="cuda").to(dtype)
    part = D.weight_rounding("fp32" if dtype == torch.float32 else "bf16")
    for window, splits in ((500, 0), (500, 3), (3000, 5)):
        lens, base = [n - 1, n - 2, n - 700], n - 4000
        out = api.decode_attn_mod_append(q, kn, vn, K, V, i32(lens), ScoreMod(window=window, softcap=20.0), num_splits=splits)
        for b, m in enumerate(lens):
            assert torch.equal(K[b, :, m], kn[b]) and torch.equal(V[b, :, m], vn[b])
        ref, tol = D.attend(q, K[:, :, base:], V[:, :, base:], [m + 1 - base for m in lens], 1 / math.sqrt(d), part, softcap=20.0,
                            window=window)
        D.check(out, ref, tol, f"window {window} splits {splits}")
    out = api.decode_attn_mod(q, K, V, i32([0, 0, n]), ScoreMod(softcap=20.0))
    assert not out[:2].any()
    g = h_q // h
    for k in (0, h - 1):
        heads = slice(g * k, g * k + 2)
        ref, tol = D.attend(q[2:, heads], K[2:, k:k + 1], V[2:, k:k + 1], [n], 1 / math.sqrt(d), part, softcap=20.0)
        D.check(out[2:, heads], ref, tol)
