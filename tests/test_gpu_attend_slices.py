"""Shared-prefix batches of more sequences than one launch lists, in the bounds-checked test build (needs a GB300).

Every launch checks its indices against what is left of q and out from its first sequence on."""
import ctypes

import pytest
import torch

import attend_bounds as A
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    prod = api.load()
    chk = ctypes.CDLL(build(test_hooks=True))
    for name, (res, args) in api.SIGNATURES.items():
        fn = getattr(chk, name)
        fn.restype = res
        fn.argtypes = args
    yield prod, chk
    api._lib = prod


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,h_q,h_kv,d,P,n_max", [(1023, 2, 2, 64, 130, 9), (1024, 4, 2, 64, 130, 9), (2100, 2, 1, 128, 40, 5),
                                                  (600, 520, 2, 64, 50, 3)])
def test_launches(libs, monkeypatch, B, h_q, h_kv, d, P, n_max, out_dtype):
    g = torch.Generator(device="cuda").manual_seed(B)
    q, Kp, Vp, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16()
                       for s in ((B, h_q, d), (h_kv, P, d), (h_kv, P, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d)))
    n = [(b * 7) % (n_max + 1) for b in range(B)]
    lens, got = torch.tensor(n, dtype=torch.int32, device="cuda"), []
    for lib in libs:
        monkeypatch.setattr(api, "_lib", lib)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        before = lib.decode_attn_launch_count()
        got.append(api.decode_attn_shared(q, Kp, Vp, K, V, lens, dev_error=err, out_dtype=out_dtype))
        assert lib.decode_attn_launch_count() - before == (2 if B == 1023 else 6 if B == 2100 else 4)
        assert int(err) == 0
    assert torch.equal(got[0], got[1])
    for part in (slice(0, 40), slice(B // 2 - 20, B // 2 + 20), slice(B - 40, B)):
        want, tol = A.shared(q[part], Kp, Vp, P, K[part], V[part], n[part], d ** -0.5, out_dtype)
        A.check(got[0][part], want, tol)
