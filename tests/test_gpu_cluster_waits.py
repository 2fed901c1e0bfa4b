"""Waits that run out in the cluster form of short caches (needs a GB300).

As test_gpu_bounded_wait.py: in the test build one CTA's last stage is never
filled.  The CTAs of its cluster merge through each other's shared memory: none
of the unit's outputs may be written, every other unit's is right, the error word
says so, and the next call is right."""
import ctypes

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod
from decode_attention_kv_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def chk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    prod = api.load()
    lib = ctypes.CDLL(build(test_hooks=True))
    for name, (res, args) in api.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    lib.decode_attn_test_withhold.argtypes = [ctypes.c_int]
    lib.decode_attn_test_withhold.restype = None
    lib.decode_attn_test_withhold(-1)
    yield lib
    lib.decode_attn_test_withhold(-1)
    api._lib = prod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def decodes():
    """name, query heads of a unit (one KV head, or a part of its heads), run(out, err)."""
    for h_q, h_kv, d_k, d_v, dtype, unit in ((4, 2, 64, 64, torch.float32, 2), (8, 2, 128, 128, torch.bfloat16, 4),
                                             (32, 1, 128, 128, torch.bfloat16, 8), (40, 1, 64, 64, torch.bfloat16, 32),
                                             (4, 1, 256, 256, torch.bfloat16, 4), (6, 2, 192, 128, torch.bfloat16, 3)):
        q, K, V = (torch.randn(s, device="cuda").to(dtype)
                   for s in ((2, h_q, d_k), (2, h_kv, 700, d_k), (2, h_kv, 700, d_v)))
        mod = ScoreMod(softcap=9.0, slopes=torch.ones(h_q, device="cuda") / 16, prefix=3, window=690)
        yield (f"{str(dtype)[6:]}-{d_k}-{h_q}", unit, (2, h_q, d_v),
               lambda out, err, q=q, K=K, V=V, mod=mod: api.decode_attn_mod(q, K, V, i32([700, 650]), mod, out=out,
                                                                           dev_error=err))
        kn, vn = K[:, :, 0].contiguous(), V[:, :, 0].contiguous()
        yield (f"append-{str(dtype)[6:]}-{d_k}-{h_q}", unit, (2, h_q, d_v),
               lambda out, err, q=q, K=K, V=V, kn=kn, vn=vn, mod=mod: api.decode_attn_mod_append(
                   q, kn, vn, K, V, i32([650, 699]), mod, out=out, dev_error=err))
    for d, h_q, unit in ((64, 4, 4), (128, 4, 4), (64, 32, 16), (128, 32, 16)):
        K, V = (torch.randint(-100, 100, (2, 1, 900, d), device="cuda", dtype=torch.int8) for _ in range(2))
        ks, vs = (torch.rand((2, 1, 29), device="cuda") / 100 for _ in range(2))
        q = torch.randn(2, h_q, d, device="cuda").to(torch.bfloat16)
        for mod in (None, ScoreMod(softcap=9.0)):
            yield (f"q8b-{d}-{h_q}-{mod is not None}", unit, (2, h_q, d),
                   lambda out, err, q=q, c=(K, V, ks, vs), mod=mod: api.decode_attn_q8b(
                       q, *c, i32([900, 800]), 32, mod=mod, out=out, dev_error=err))


@pytest.mark.parametrize("cta", [0, 1, 4])
def test_a_unit_whose_wait_ran_out_is_not_written(chk, monkeypatch, cta):
    """CTAs 0 to 4 are in the first unit's cluster (every shape has five shares of rows or more)."""
    for name, unit, shape, run in decodes():
        want = torch.full(shape, 77.0, device="cuda")
        run(want, None)
        monkeypatch.setattr(api, "_lib", chk)
        chk.decode_attn_test_withhold(cta)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = torch.full_like(want, 77.0)
        before = api.launch_count()
        run(got, err)
        torch.cuda.synchronize()
        assert api.launch_count() == before + 1, name  # one launch: the cluster form
        assert int(err) == api.DEVERR_TIMEOUT, name
        assert bool((got[0, :unit] == 77.0).all()), name
        got[0, :unit] = want[0, :unit]
        assert torch.equal(got, want), name
        chk.decode_attn_test_withhold(-1)
        err.zero_()
        got.fill_(77.0)
        run(got, err)
        assert int(err) == 0 and torch.equal(got, want), name
        monkeypatch.undo()
        got.fill_(77.0)
        run(got, None)
        assert torch.equal(got, want), name
