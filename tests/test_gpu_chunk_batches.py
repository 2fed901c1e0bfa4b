"""Chunks of batches that mix prompts and single tokens, of sequences about as many as the schedule lists, and the
largest windows and always-seen rows (needs a GB300)."""
import math

import pytest
import torch

import attend_bounds as A
from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu
MOST = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(B, T, h_q, h_kv, d, n_max, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16()
               for s in ((B, T, h_q, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d)))
    return (2 * q).transpose(1, 2), K, V


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,n_max,h_kv,window", [(300, 5000, 4, 0), (2048, 6000, 8, 0), (600, 9000, 2, 3000)])
def test_a_prompt_among_single_tokens(T, n_max, h_kv, window, out_dtype):
    """One sequence brings T tokens, the others one each behind long contexts, or none."""
    B, g, d = 6, 2, 128
    q, K, V = make(B, T, g * h_kv, h_kv, d, n_max, T)
    lens, news = [T, n_max, n_max - 1, 4000, 1, 700], [T, 1, 1, 1, 1, 0]
    out = torch.full((B, T, g * h_kv, d), 7.0, dtype=out_dtype, device="cuda").transpose(1, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.chunk_attn(q, K, V, i32(lens), n_new=i32(news), window=window, out=out, dev_error=err)
    assert int(err) == 0
    for b in range(B):
        assert (out[b, :, news[b]:] == 7.0).all()
        m = news[b]
        if m == 0:
            continue
        # the prompt's tokens a few at a time
        for at in [*range(0, m, 97), m - 1]:
            n = lens[b] - m + at + 1
            want, tol = A.chunk(q[b:b + 1, :, at:at + 1], K[b:b + 1], V[b:b + 1], [n], [1], 1 / math.sqrt(d), out_dtype,
                                window)
            A.check(out[b:b + 1, :, at:at + 1], want, tol, (b, at))


@pytest.mark.parametrize("B,T,g", [(1023, 1, 2), (1024, 1, 2), (1025, 1, 2), (256, 4, 256), (257, 4, 256)])
def test_as_many_sequences_as_are_listed(B, T, g):
    """1024 entries are cut along the rows, more are not: one long context among short ones, either way."""
    d, n_max = 64, 2600
    gen = torch.Generator(device="cuda").manual_seed(B)
    q, K, V = (torch.randn(s, generator=gen, device="cuda").bfloat16()
               for s in ((B, g, T, d), (B, 1, n_max, d), (B, 1, n_max, d)))
    lens = [T + (b * 5) % 40 for b in range(B)]
    lens[B // 3] = n_max
    before = api.launch_count()
    out = api.chunk_attn(q, K, V, i32(lens), out_dtype=torch.bfloat16)
    assert api.launch_count() - before == (2 if B * -(-T * g // 256) <= 1024 else 1)
    for b in (0, B // 3, B // 2, B - 1):
        at = slice(b, b + 1)
        want, tol = A.chunk(q[at], K[at], V[at], [lens[b]], [T], 1 / math.sqrt(d), torch.bfloat16)
        A.check(out[at], want, tol, b)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("window,prefix", [(MOST, 7), (MOST, MOST), (50, MOST), (1, MOST), ((1 << 30) + 1, 3), (0, MOST)])
def test_largest_windows(window, prefix, out_dtype):
    """All that came before is seen: positions plus a window, and first rows, beyond 32 bits."""
    B, T, n_max = 2, 150, 900
    q, K, V = make(B, T, 4, 2, 64, n_max, 3)
    lens, news = [900, 431], [150, 90]
    out = torch.zeros((B, T, 4, 64), dtype=out_dtype, device="cuda").transpose(1, 2)
    api.chunk_attn(q, K, V, i32(lens), n_new=i32(news), window=window, prefix=prefix, out=out)
    want, tol = A.chunk(q, K, V, lens, news, 0.125, out_dtype)
    A.check(out, want, tol)
