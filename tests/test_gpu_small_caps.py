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


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("splits", [0, 3])
def test_block_scales_far_above_the_cap(splits, out_dtype):
    """The factor of the scores is beyond float; rows of zeros have a score of zero all the same."""
    n, d, h_q = 600, 64, 8
    K, V = (torch.randint(-127, 128, (1, 1, n, d), dtype=torch.int8, device="cuda") for _ in range(2))
    K[:, :, ::3] = 0
    q = torch.randn(1, h_q, d, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    vs = torch.full((1, 1, 38), 2.0 ** -6, device="cuda")
    part = 2.0 ** -11 if out_dtype == torch.bfloat16 else D.weight_rounding("q8b")
    for cap, size in ((1e-30, 1e12), (0.0, 3e38)):
        ks = torch.full((1, 1, 38), size, device="cuda")
        if cap == 0.0:
            K.zero_()  # (every score is zero)
        out = api.decode_attn_q8b(q, K, V, ks, vs, lens, 16, mod=ScoreMod(softcap=cap) if cap else None, scale=1e6,
                                  num_splits=splits, out_dtype=out_dtype)
        want = (V.double() / 64).mean(2).expand(1, h_q, d)
        tol = (V.double() / 64).abs().mean(2) * (part + 4 * (n / 8 + 64) * D.U)
        tol = tol + (want.abs() + tol) * (torch.finfo(out_dtype).eps / 2)
        D.check(out, want, tol)
