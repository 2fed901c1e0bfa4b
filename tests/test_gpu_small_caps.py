"""Caps far below the scores: every score saturates, none becomes NaN (needs a GB300)."""
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


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("h_q,h_kv,d,dtype", [(2, 2, 64, torch.float32), (8, 1, 128, torch.float32),
                                             (8, 2, 128, torch.bfloat16), (32, 1, 128, torch.bfloat16)])
def test_scores_far_above_the_cap(h_q, h_kv, d, dtype, splits):
    """q . K / cap is beyond float; the capped scores are +-1e-30, so that all rows weigh the same:
    the mean of V, off by the sums' roundings and the weights' (decode_bounds)."""
    n = 600
    q, K = (1e6 * torch.randn(s, device="cuda").to(dtype) for s in ((2, h_q, d), (2, h_kv, n, d)))
    V = torch.randn(2, h_kv, n, d, device="cuda").to(dtype)
    lens = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    for out_dtype in (torch.float32, torch.bfloat16):
        out = api.decode_attn_mod(q, K, V, lens, ScoreMod(softcap=1e-30), num_splits=splits, out_dtype=out_dtype)
        want = V.double().mean(2).repeat_interleave(h_q // h_kv, 1)
        part = D.weight_rounding("fp32" if dtype == torch.float32 else "bf16")
        tol = V.double().abs().mean(2).repeat_interleave(h_q // h_kv, 1) * (part + 4 * (n / 8 + 64) * D.U)
        tol = tol + (want.abs() + tol) * (torch.finfo(out_dtype).eps / 2)
        D.check(out, want, tol)
