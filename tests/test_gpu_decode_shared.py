"""Decode steps of a batch behind a shared prefix (needs a GB300): each element against 64 bits with a bound of its own."""
import math

import pytest
import torch

import attend_bounds as A
from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu
OUTS = [torch.bfloat16, torch.float32]
OID = ["bf16", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(B, h_q, h_kv, d, P, n_max, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return 2 * r(B, h_q, d), r(h_kv, P, d), r(h_kv, P, d), r(B, h_kv, n_max, d), r(B, h_kv, n_max, d)


def run(B, h_q, h_kv, d, P, cap, lens, n_max, out_dtype, seed=0, scale=None):
    q, Kp, Vp, K, V = make(B, h_q, h_kv, d, cap, n_max, seed)
    Kx, Vx = K.clone(), V.clone()
    for b, n in enumerate(lens):
        Kx[b, :, n:] = Vx[b, :, n:] = float("nan")
    Kpx, Vpx = Kp.clone(), Vp.clone()
    Kpx[:, P:] = Vpx[:, P:] = float("nan")
    scale = 1 / math.sqrt(d) if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.decode_attn_shared(q, Kpx, Vpx, Kx, Vx, i32(lens), prefix_len=P, scale=scale, dev_error=err,
                                 out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert int(err) == 0 and out.dtype == out_dtype
    want, tol = A.shared(q, Kp, Vp, P, K, V, lens, scale, out_dtype)
    A.check(out, want, tol)
    return out


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d", [64, 128])
def test_small(out_dtype, d):
    run(1, 1, 1, d, 1, 1, [0], 4, out_dtype)
    run(1, 1, 1, d, 1, 1, [1], 4, out_dtype)
    run(2, 2, 1, d, 5, 9, [0, 3], 4, out_dtype)
    run(3, 6, 2, d, 130, 200, [128, 129, 1], 200, out_dtype)
    run(2, 4, 2, d, 0, 7, [0, 100], 100, out_dtype)           # no prefix; nothing at all: 0


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("P", [127, 128, 129, 1000, 20000])
def test_prefixes(P, out_dtype):
    run(6, 16, 2, 128, P, P + 3, [0, 1, 500, 128, 300, 77], 500, out_dtype, seed=P)


@pytest.mark.parametrize("B,h_q,h_kv", [(1, 8, 8), (17, 8, 1), (33, 32, 1), (33, 24, 8), (3, 300, 1), (2, 520, 2), (300, 4, 2)])
def test_batches_and_groups(B, h_q, h_kv):
    lens = [(b * 53) % 280 for b in range(B)]
    run(B, h_q, h_kv, 64, 777, 777, lens, 280, torch.bfloat16, seed=B)
    run(B, h_q, h_kv, 128, 300, 300, lens, 280, torch.float32, seed=B)


def test_long_own_rows_and_scales():
    run(2, 8, 1, 128, 300, 300, [9000, 4], 9000, torch.bfloat16)
    for scale in (0.0, -0.25, 2.0):
        run(4, 8, 2, 64, 400, 400, [30, 0, 200, 129], 200, torch.float32, scale=scale)


def test_batch_of_several_launches():
    """More sequences than one launch lists."""
    B = 1100
    q, Kp, Vp, K, V = make(B, 2, 1, 64, 200, 40, seed=2)
    lens = [(b * 7) % 41 for b in range(B)]
    out = api.decode_attn_shared(q, Kp, Vp, K, V, i32(lens))
    for b0 in range(0, B, 100):
        part = slice(b0, b0 + 100)
        want, tol = A.shared(q[part], Kp, Vp, 200, K[part], V[part], lens[part], 0.125, torch.float32)
        A.check(out[part], want, tol)


def test_same_as_one_cache():
    """The prefix copied in front of every sequence's rows and decoded as one cache."""
    q, Kp, Vp, K, V = make(4, 16, 2, 128, 1500, 64, seed=3)
    lens = [64, 0, 1, 33]
    full = [torch.zeros((4, 2, 1564, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for f, x, y in ((full[0], Kp, K), (full[1], Vp, V)):
        f[:, :, :1500] = x
        f[:, :, 1500:] = y
    a = api.decode_attn_shared(q, Kp, Vp, K, V, i32(lens))
    b = api.decode_attn(q, *full, i32([1500 + n for n in lens]))
    torch.testing.assert_close(a, b, rtol=0, atol=4e-4)       # two roundings of weights of 2^-16 |V|, |V| < 6


def test_bad_lengths_graph_and_repeats():
    q, Kp, Vp, K, V = make(3, 8, 2, 64, 300, 50, seed=4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.decode_attn_shared(q, Kp, Vp, K, V, i32([60, -2, 50]), dev_error=err)
    assert int(err) == api.DEVERR_SEQ_LEN
    lens = i32([50, 0, 50])
    assert torch.equal(out, api.decode_attn_shared(q, Kp, Vp, K, V, lens))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = api.decode_attn_shared(q, Kp, Vp, K, V, lens)
    lens.copy_(i32([3, 50, 0]))
    want = api.decode_attn_shared(q, Kp, Vp, K, V, lens)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want)
