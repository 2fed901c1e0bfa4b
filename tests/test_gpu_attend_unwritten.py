"""A shared-prefix call one of whose waits runs out, in a workspace that no call has used (needs a GB300).

The CTA that gives up leaves the rest of its units unnoted, so the merge finds what the workspace held there: it
follows no index out of the partials, the call reports DA_DEVERR_TIMEOUT, and the next call is right."""
import ctypes

import pytest
import torch

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
    chk.decode_attn_test_withhold.argtypes = [ctypes.c_int]
    chk.decode_attn_test_withhold.restype = None
    chk.decode_attn_test_withhold(-1)
    yield prod, chk
    chk.decode_attn_test_withhold(-1)
    api._lib = prod


# bytes of the workspace before the call: CTAs of -1, 0x7f7f7f7f, 0x80808080 and 0x01010101
@pytest.mark.parametrize("fill", [0xff, 0x7f, 0x80, 0x01])
@pytest.mark.parametrize("cta", [0, 5, 100])
def test_units_that_nobody_noted(libs, monkeypatch, cta, fill):
    """1040 units, seven to a CTA (the prefix's first): the withheld one gives up at its first."""
    B, h, d, P, n = 64, 16, 64, 100, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q, Kp, Vp, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16()
                       for s in ((B, h, d), (h, P, d), (h, P, d), (B, h, n, d), (B, h, n, d)))
    lens = torch.tensor([1 + (b * 37) % n for b in range(B)], dtype=torch.int32, device="cuda")
    st = ctypes.c_int(0)
    need = libs[1].decode_attn_shared_workspace_bytes(B, h, h, d, n, P, api.DA_BF16, ctypes.byref(st))
    assert st.value == 0 and need > 0
    ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return api.decode_attn_shared(q, Kp, Vp, K, V, lens, workspace=ws, dev_error=err)
    monkeypatch.setattr(api, "_lib", libs[1])
    libs[1].decode_attn_test_withhold(cta)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        libs[1].decode_attn_test_withhold(-1)
    assert int(err) & api.DEVERR_TIMEOUT and not int(err) & api.DEVERR_BOUNDS
    err.zero_()
    ws.fill_(fill)
    have = call()
    assert int(err) == 0
    monkeypatch.setattr(api, "_lib", libs[0])
    ws.fill_(fill)
    want = call()
    assert int(err) == 0 and torch.equal(have, want) and torch.isfinite(want).all()
