"""Prompts in chunks, then decode steps, as they are used together (needs a GB300): rotation and
append, chunk attention, steps over the same cache and behind a shared prefix; against 64 bits."""
import math

import pytest
import torch

import attend_bounds as A
import decode_bounds as D
from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_chunks_then_steps():
    B, h_q, h_kv, d, n_max, rot = 3, 8, 2, 128, 512, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    half = rot // 2
    angle = torch.arange(2000, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    cos, sin = angle.cos().float(), angle.sin().float()
    w = (1 + 0.1 * r(d).float()).bfloat16()
    K, V = (torch.full((B, h_kv, n_max, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    prefix = 700                                              # rows of a shared prefix, computed first
    Kp, Vp = (torch.zeros((1, h_kv, prefix, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = r(1, prefix, h_q + 2 * h_kv, d)
    cut = lambda x: (x[:, :, :h_q].transpose(1, 2), x[:, :, h_q:h_q + h_kv].transpose(1, 2),  # noqa: E731
                     x[:, :, h_q + h_kv:].transpose(1, 2))
    q = api.kv_append_rope(*cut(x), Kp, Vp, i32([0]), cos, sin, q_weight=w, k_weight=w)
    got = api.chunk_attn(q, Kp, Vp, i32([prefix]))
    A.check(got, *A.chunk(q, Kp, Vp, [prefix], [prefix], 1 / math.sqrt(d), torch.float32))

    lens = [0] * B
    for news in ([200, 131, 0], [1, 129, 64], [5, 0, 7]):     # prompts, in ragged chunks
        T = max(news)
        x = r(B, T, h_q + 2 * h_kv, d)
        q = api.kv_append_rope(*cut(x), K, V, i32(lens), cos, sin, q_weight=w, k_weight=w, n_new=i32(news),
                               angle_pos=i32([prefix + n for n in lens]))
        lens = [n + m for n, m in zip(lens, news)]
        out = torch.zeros((B, h_q, T, d), dtype=torch.bfloat16, device="cuda")
        got = api.chunk_attn(q, K, V, i32(lens), n_new=i32(news), window=150, prefix=4, out=out)
        A.check(got, *A.chunk(q, K, V, lens, news, 1 / math.sqrt(d), torch.bfloat16, 150, 4))

    for _ in range(3):                                        # steps of the whole batch behind the prefix
        x = r(B, 1, h_q + 2 * h_kv, d)
        q = api.kv_append_rope(*cut(x), K, V, i32(lens), cos, sin, q_weight=w, k_weight=w,
                               angle_pos=i32([prefix + n for n in lens]))
        lens = [n + 1 for n in lens]
        q1 = q.squeeze(2).contiguous()
        got = api.decode_attn_shared(q1, Kp[0], Vp[0], K, V, i32(lens))
        A.check(got, *A.shared(q1, Kp[0], Vp[0], prefix, K, V, lens, 1 / math.sqrt(d), torch.float32))
        # and the decode over their own rows, from the cache that the chunks have filled
        D.check(api.decode_attn(q1, K, V, i32(lens)), *D.attend(q1, K, V, lens, 1 / math.sqrt(d), D.weight_rounding("bf16")))


def test_steps_into_an_eight_bit_cache():
    """Rows rotated into a buffer of one chunk, quantised from there, read back and attended."""
    B, h_q, h_kv, d, T, n_max = 2, 8, 2, 64, 50, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((B, T, h_q + 2 * h_kv, d), generator=g, device="cuda").bfloat16()
    angle = torch.arange(100, device="cuda")[:, None] * 10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, h_q), (h_q, h_q + h_kv), (h_q + h_kv, h_q + 2 * h_kv)))
    Kc, Vc = (torch.zeros((B, h_kv, T, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    zero = i32([0] * B)
    q = api.kv_append_rope(q, k, v, Kc, Vc, zero, angle.cos().float(), angle.sin().float())
    codes = [torch.zeros((B, h_kv, n_max, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((B, h_kv, n_max // 16), device="cuda") for _ in range(2)]
    api.kv_append_q8b(Kc, Vc, *codes, *scales, zero, 16)
    Kb, Vb = api.kv_read_q8b(*codes, *scales, i32([T] * B), 16)
    got = api.chunk_attn(q, Kb, Vb, i32([T] * B))
    A.check(got, *A.chunk(q, Kb, Vb, [T] * B, [T] * B, 1 / math.sqrt(d), torch.float32))


def test_rows_more_than_two_to_the_32_bytes_away():
    B, h_q, h_kv, d, n_max = 2, 4, 2, 128, 6_000_000            # 1.5 GB a head, 6.1 GB a cache
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    K, V = (torch.empty((B, h_kv, n_max, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n, T, window = n_max - 3, 5, 700
    K[:, :, n - 1000:n], V[:, :, n - 1000:n] = r(B, h_kv, 1000, d), r(B, h_kv, 1000, d)
    x = r(B, T, h_q + 2 * h_kv, d)
    cos, sin = torch.ones((T, d // 2), device="cuda"), torch.zeros((T, d // 2), device="cuda")
    api.kv_append_rope(x[:, :, :h_q].transpose(1, 2), x[:, :, h_q:h_q + h_kv].transpose(1, 2),
                       x[:, :, h_q + h_kv:].transpose(1, 2), K, V, i32([n - T] * B), cos, sin, angle_pos=i32([0] * B))
    assert torch.equal(K[:, :, n - T:n], x[:, :, h_q:h_q + h_kv].transpose(1, 2))
    q = x[:, :, :h_q].transpose(1, 2)
    got = api.chunk_attn(q, K, V, i32([n] * B), window=window)
    near = slice(n - 1000, n)
    A.check(got, *A.chunk(q, K[:, :, near], V[:, :, near], [1000] * B, [T] * B, 1 / math.sqrt(d), torch.float32, window))
