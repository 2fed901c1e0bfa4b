"""A slope that is NaN makes its own head's output NaN and no other's (needs a GB300)."""
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


def check(run, h_q, want, tol, bad):
    """run(slopes) against the bounds of all heads but the bad one."""
    slopes = torch.full((h_q,), 0.125, device="cuda")
    keep = [h for h in range(h_q) if h != bad]
    slopes[bad] = float("nan")
    out = run(slopes)
    D.check(out[:, keep], want[:, keep], tol[:, keep])
    assert torch.isnan(out[:, bad]).all()


@pytest.mark.parametrize("splits", [0, 1, 3, 40, -1])  # (40: the combine of several warps)
@pytest.mark.parametrize("kind", ["fp32", "fp32-8", "bf16", "bf16-32", "tc5"])
def test_decode_mod(kind, splits):
    h_q, h_kv, d, dtype = {"fp32": (2, 2, 64, torch.float32), "fp32-8": (8, 1, 128, torch.float32),
                           "bf16": (8, 2, 128, torch.bfloat16), "bf16-32": (32, 1, 64, torch.bfloat16),
                           "tc5": (32, 1, 128, torch.bfloat16)}[kind]
    n, lens = 6000, [6000, 77]
    q, K, V = (torch.randn(s, device="cuda").to(dtype) for s in ((2, h_q, d), (2, h_kv, n, d), (2, h_kv, n, d)))
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for cap in (0.0, 9.0):
        want, tol = D.attend(q, K, V, lens, d ** -0.5, D.weight_rounding("fp32" if dtype == torch.float32 else "bf16"),
                             softcap=cap, slopes=[0.125] * h_q)
        check(lambda s: api.decode_attn_mod(q, K, V, ld, ScoreMod(slopes=s, softcap=cap), num_splits=splits), h_q, want, tol,
              h_q // 2)


@pytest.mark.parametrize("splits", [0, 1, 40])
@pytest.mark.parametrize("d,h_q", [(64, 4), (128, 8), (128, 32)])
def test_decode_q8b(d, h_q, splits):
    n, lens = 6000, [6000, 77]
    K, V = (torch.randint(-127, 128, (2, 1, n, d), dtype=torch.int8, device="cuda") for _ in range(2))
    s = torch.full((2, 1, -(-n // 32)), 2.0 ** -6, device="cuda")
    q = torch.randn(2, h_q, d, device="cuda").to(torch.bfloat16)
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want, tol = D.attend(q, K.double() / 64, V.double() / 64, lens, d ** -0.5, D.weight_rounding("q8b"),
                         slopes=[0.125] * h_q, floor=2.0 ** -31)
    check(lambda sl: api.decode_attn_q8b(q, K, V, s, s, ld, 32, mod=ScoreMod(slopes=sl), num_splits=splits), h_q, want, tol, 1)
