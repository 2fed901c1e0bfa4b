"""How exactly chunk_attn and decode_attn_shared multiply their weights (needs a GB300)."""
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


def rand(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").bfloat16() for s in shapes]


CHUNKS = [  # B, T, h_q, h_kv, d, n_max, lens, news, window, prefix: whole units, units cut along the rows, few tokens
    (2, 300, 6, 2, 128, 700, [700, 300], [300, 41], 0, 0), (2, 150, 4, 2, 64, 1900, [1900, 431], [150, 90], 200, 9),
    (2, 7, 16, 2, 128, 9000, [9000, 6], [7, 6], 0, 0), (1, 40, 8, 1, 64, 12000, [11990], [40], 0, 0),
    (3, 1, 16, 2, 128, 5000, [5000, 431, 1], [1, 1, 1], 0, 0)]


def chunk_case(case):
    B, T, h_q, h_kv, d, n_max, lens, news, window, prefix = case
    q, K, V = rand(T, (B, T, h_q, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d))
    q = (2 * q).transpose(1, 2)

    def run(out_dtype, **kw):
        out = torch.zeros((B, T, h_q, d), dtype=out_dtype, device="cuda").transpose(1, 2)
        return api.chunk_attn(q, K, V, i32(lens), n_new=i32(news), window=window, prefix=prefix, out=out, **kw)
    return run, lambda out_dtype: A.chunk(q, K, V, lens, news, 1 / math.sqrt(d), out_dtype, window, prefix)


SHARED = [(3, 8, 2, 64, 1000, [20, 0, 50], 50), (33, 32, 1, 128, 3000, [(b * 31) % 600 for b in range(33)], 600)]


def shared_case(case):
    B, h_q, h_kv, d, P, lens, n_max = case
    q, Kp, Vp, K, V = rand(P, (B, h_q, d), (h_kv, P, d), (h_kv, P, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d))
    q = 2 * q
    return (lambda out_dtype, **kw: api.decode_attn_shared(q, Kp, Vp, K, V, i32(lens), out_dtype=out_dtype, **kw),
            lambda out_dtype: A.shared(q, Kp, Vp, P, K, V, lens, 1 / math.sqrt(d), out_dtype))


CASES = [(chunk_case, c) for c in CHUNKS] + [(shared_case, c) for c in SHARED]
IDS = [f"chunk-T{c[1]}n{c[5]}" for c in CHUNKS] + [f"shared-B{c[0]}" for c in SHARED]


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("make,case", CASES, ids=IDS)
def test_exact_unless_asked(make, case, out_dtype, monkeypatch):
    """Weights carry 2^-16 whatever the output's type, as decode_attn's do: a bf16 and its bf16 remainder."""
    run, reference = make(case)
    monkeypatch.setattr(A, "part", lambda out: 2.0 ** -16)
    A.check(run(out_dtype), *reference(out_dtype))


@pytest.mark.parametrize("make,case", CASES, ids=IDS)
def test_asked_for_as_one_bf16(make, case):
    """2^-8 of a weight, where the caller says so, and other bits than the exact ones."""
    run, reference = make(case)
    out = run(torch.bfloat16, bf16_weights=True)
    assert A.part(torch.bfloat16) == 2.0 ** -8
    A.check(out, *reference(torch.bfloat16))
    assert not torch.equal(out, run(torch.bfloat16))
    with pytest.raises(ValueError):
        run(torch.float32, bf16_weights=True)


def test_as_decode_attn():
    """One token a sequence: the same weights as the decode step's, rounded once to the output's type."""
    q, K, V = rand(9, (3, 16, 128), (3, 2, 9000, 128), (3, 2, 9000, 128))
    lens = i32([9000, 4321, 1])
    exact = api.decode_attn(2 * q, K, V, lens)
    out = api.chunk_attn((2 * q).unsqueeze(2), K, V, lens, out_dtype=torch.bfloat16).squeeze(2).float()
    off = 4e-4   # two roundings of weights of 2^-16 |V|, |V| < 6; then half a step of the output
    half = torch.finfo(torch.bfloat16).eps / 2
    assert ((out - exact).abs() <= off + half * (exact.abs() + off)).all()
