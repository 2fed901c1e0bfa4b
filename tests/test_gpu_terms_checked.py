"""Score-term and block-scale entry points in the bounds-checked test build (needs a GB300).

As test_gpu_checked_build.py: each call through the product library and through
the build that checks every global index, on the same inputs: no index out of
range, the same error word, bit-equal outputs and caches.  And as
test_gpu_bounded_wait.py: a stage that is never filled makes a wait run out,
the call returns DA_DEVERR_TIMEOUT and the next one is right."""
import ctypes

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod
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


def both(libs, monkeypatch, run):
    """run(err) -> tensors through each library."""
    got = []
    for lib in libs:
        monkeypatch.setattr(api, "_lib", lib)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = run(err)
        torch.cuda.synchronize()
        got.append(([t.clone() for t in outs], int(err)))
    monkeypatch.setattr(api, "_lib", libs[0])
    (want, err_p), (have, err_c) = got
    assert err_c & api.DEVERR_BOUNDS == 0, f"checked build found an index out of range ({err_c:#x})"
    assert err_c == err_p
    for a, b in zip(want, have):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return err_p


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def terms(h_q, B):
    slopes = torch.exp2(-8.0 * torch.arange(1, h_q + 1, device="cuda") / h_q)
    return [ScoreMod(window=100, prefix=3), ScoreMod(softcap=20.0, doc_begin=i32([150 * b for b in range(B)])),
            ScoreMod(slopes=slopes, prefix=40, doc_begin=i32([9000] * B)),
            ScoreMod(softcap=9.0, slopes=-slopes, window=300)]


SHAPES = [
    (3, 8, 8, 64, 64, 700, [700, 0, 333], torch.float32),
    (2, 16, 2, 128, 128, 600, [600, 77], torch.float32),
    (4, 32, 4, 128, 128, 2000, [2000, 1, 999, 1500], torch.bfloat16),
    (2, 32, 1, 128, 128, 2500, [2500, 1234], torch.bfloat16),
    (2, 32, 2, 256, 256, 260, [260, 65], torch.bfloat16),
    (2, 32, 4, 192, 128, 260, [257, 128], torch.bfloat16),
    (3, 16, 2, 64, 64, 500, [-5, 5000, 100], torch.bfloat16),
]


@pytest.mark.parametrize("splits", [0, 3, -1])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{str(s[7])[6:]}d{s[3]}g{s[1] // s[2]}" for s in SHAPES])
def test_decode_mod(libs, monkeypatch, shape, splits):
    B, h_q, h_kv, dk, dv, n_max, lens, dtype = shape
    r = torch.Generator(device="cuda").manual_seed(1)
    q, K, V, kn, vn = (torch.randn(s, generator=r, device="cuda").to(dtype)
                       for s in ((B, h_q, dk), (B, h_kv, n_max, dk), (B, h_kv, n_max, dv), (B, h_kv, dk),
                                 (B, h_kv, dv)))
    ld = i32(lens)
    for mod in terms(h_q, B):
        for out_dtype in (torch.float32, torch.bfloat16):
            both(libs, monkeypatch, lambda e: [api.decode_attn_mod(q, K, V, ld, mod, num_splits=splits, dev_error=e,
                                                                   out_dtype=out_dtype)])

        def step(e):
            K2, V2, grown = K.clone(), V.clone(), torch.zeros_like(ld)
            out = api.decode_attn_mod_append(q, kn, vn, K2, V2, ld, mod, seq_lens_out=grown, num_splits=splits,
                                             dev_error=e)
            return [out, K2, V2, grown]
        both(libs, monkeypatch, step)


def test_decode_mod_many_items(libs, monkeypatch):
    B = 400
    r = torch.Generator(device="cuda").manual_seed(1)
    q, K, V = (torch.randn(s, generator=r, device="cuda").to(torch.bfloat16)
               for s in ((B, 8, 64), (B, 8, 200, 64), (B, 8, 200, 64)))
    lens = i32([(b * 31) % 201 for b in range(B)])
    mod = ScoreMod(window=64, prefix=10, doc_begin=i32([b % 90 for b in range(B)]))
    for splits in (3, -1):
        both(libs, monkeypatch, lambda e: [api.decode_attn_mod(q, K, V, lens, mod, num_splits=splits, dev_error=e)])


Q8B = [(3, 8, 2, 64, 517, [517, 0, 130], 16), (2, 24, 2, 64, 300, [300, 299], 128), (2, 8, 1, 128, 1000, [999, 5], 32),
       (2, 32, 1, 128, 1500, [1500, 700], 64), (2, 12, 3, 128, 400, [-1, 999], 64)]


def q8b_cache(B, h, n_max, d, block, dtype):
    r = torch.Generator(device="cuda").manual_seed(2)
    codes = [torch.randint(-100, 100, (B, h, n_max, d), generator=r, device="cuda", dtype=torch.int8).view(dtype)
             if dtype == torch.int8 else torch.randn((B, h, n_max, d), generator=r, device="cuda").to(dtype)
             for _ in range(2)]
    scales = [torch.rand((B, h, -(-n_max // block)), generator=r, device="cuda") + 0.01 for _ in range(2)]
    return codes + scales


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "fp8"])
@pytest.mark.parametrize("shape", Q8B, ids=[f"d{s[3]}g{s[1] // s[2]}" for s in Q8B])
def test_decode_q8b(libs, monkeypatch, shape, dtype):
    B, h_q, h_kv, d, n_max, lens, block = shape
    K, V, ks, vs = q8b_cache(B, h_kv, n_max, d, block, dtype)
    q = torch.randn(B, h_q, d, device="cuda").to(torch.bfloat16)
    for mod in [None] + terms(h_q, B):
        for splits, out_dtype in ((0, torch.float32), (5, torch.bfloat16)):
            both(libs, monkeypatch,
                 lambda e: [api.decode_attn_q8b(q, K, V, ks, vs, i32(lens), block, mod=mod, num_splits=splits,
                                                dev_error=e, out_dtype=out_dtype)])


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "fp8"])
@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_write_and_read(libs, monkeypatch, d, x_dtype, dtype):
    B, h, n_max = 5, 3, 333
    for block in (16, 32, 64, 128):
        cache = q8b_cache(B, h, n_max, d, block, dtype)
        for T, pos, n_new in ((1, [0, 332, 17, 333, -2], [1, 1, 1, 1, 1]), (300, [0, 5, 100, 300, 33], [300, 0, 200, 99, 128])):
            x = torch.randn(B, h, T, d, device="cuda").to(x_dtype)

            def step(e):
                K, V, ks, vs = (t.clone() for t in cache)
                api.kv_append_q8b(x, -x, K, V, ks, vs, i32(pos), block, n_new=i32(n_new), dev_error=e)
                out = [K, V, ks, vs]
                for t in (torch.float32, torch.bfloat16):
                    out += api.kv_read_q8b(K, V, ks, vs, i32([333, 1, 50, 400, 200]), block, rows=T + 20,
                                           row_begin=i32([0, 0, 49, 20, 300]), out_dtype=t, dev_error=e)
                return out
            assert both(libs, monkeypatch, step) != 0


def test_waits_that_run_out(libs, monkeypatch):
    """One CTA's last stage is never filled: the call returns, says so, and the next one is right."""
    prod, chk = libs
    cases = []
    for B, h_q, h_kv, d, n, dtype in ((2, 4, 2, 64, 600, torch.float32), (2, 8, 2, 128, 900, torch.bfloat16),
                                      (1, 32, 1, 128, 900, torch.bfloat16)):
        q, K, V = (torch.randn(s, device="cuda").to(dtype) for s in ((B, h_q, d), (B, h_kv, n, d), (B, h_kv, n, d)))
        for mod in (ScoreMod(window=500, softcap=9.0), ScoreMod(slopes=torch.ones(h_q, device="cuda"))):
            cases.append(lambda e, q=q, K=K, V=V, mod=mod, B=B, n=n: api.decode_attn_mod(
                q, K, V, i32([n] * B), mod, num_splits=2, dev_error=e))
    for d, h_q in ((64, 4), (128, 4), (128, 32)):
        K, V, ks, vs = q8b_cache(2, 2, 900, d, 32, torch.int8)
        q = torch.randn(2, h_q, d, device="cuda").to(torch.bfloat16)
        cases.append(lambda e, q=q, c=(K, V, ks, vs): api.decode_attn_q8b(q, *c, i32([900, 800]), 32, num_splits=2,
                                                                          dev_error=e))
    for run in cases:
        want = run(None)
        monkeypatch.setattr(api, "_lib", chk)
        chk.decode_attn_test_withhold(0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        run(err)
        torch.cuda.synchronize()
        assert int(err) & api.DEVERR_TIMEOUT and not int(err) & api.DEVERR_BOUNDS
        chk.decode_attn_test_withhold(-1)
        err.zero_()
        got = run(err)
        assert int(err) == 0 and torch.equal(got, want)
        monkeypatch.setattr(api, "_lib", prod)
        assert torch.equal(run(None), want)
