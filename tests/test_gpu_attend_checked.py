"""The chunk, shared-prefix and rotation entry points in the bounds-checked test build (needs a GB300).

Each call through the product library and through the build that checks every global index: no
index out of range, the same error word, bit-equal results.  And a stage that is never filled makes
a wait run out: the call returns DA_DEVERR_TIMEOUT, the GPU stays usable and the next call is right."""
import ctypes

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

pytestmark = pytest.mark.gpu
OUTS = [torch.bfloat16, torch.float32]


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
        got.append(([t.contiguous().clone() for t in outs], int(err)))
    monkeypatch.setattr(api, "_lib", libs[0])
    (want, err_p), (have, err_c) = got
    assert err_c & api.DEVERR_BOUNDS == 0, f"an index out of range ({err_c:#x})"
    assert err_c == err_p
    for a, b in zip(want, have):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return err_p


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").bfloat16() for s in shapes]


CHUNKS = [  # B, T, h_q, h_kv, d, n_max, lens, news, window, prefix
    (3, 5, 8, 2, 64, 300, [300, 5, 77], [5, 5, 2], 0, 0),
    (2, 300, 6, 2, 128, 700, [700, 300], [300, 41], 0, 0),
    (2, 7, 64, 1, 128, 9000, [9000, 6], [7, 7], 0, 0),
    (4, 33, 20, 4, 64, 3000, [3000, 0, 33, -4], [33, 0, 40, 1], 500, 9),
    (40, 3, 16, 8, 128, 2000, [(b * 97) % 2001 for b in range(40)], [b % 4 for b in range(40)], 0, 0),
    (1, 1, 300, 1, 64, 5000, [5000], [1], 3000, 200),
]


@pytest.mark.parametrize("case", CHUNKS, ids=[f"T{c[1]}d{c[4]}n{c[5]}" for c in CHUNKS])
def test_chunk(libs, monkeypatch, case):
    B, T, h_q, h_kv, d, n_max, lens, news, window, prefix = case
    q, K, V = rand(1, (B, T, h_q, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d))
    for out_dtype in OUTS:
        def run(e):
            out = torch.zeros((B, h_q, T, d), dtype=out_dtype, device="cuda")
            return [api.chunk_attn(q.transpose(1, 2), K, V, i32(lens), n_new=i32(news), window=window, prefix=prefix,
                                   out=out, dev_error=e)]
        both(libs, monkeypatch, run)


SHARED = [(3, 8, 2, 64, 1000, [20, 0, 50], 50), (33, 32, 1, 128, 3000, [(b * 31) % 600 for b in range(33)], 600),
          (5, 24, 8, 128, 0, [0, 300, 1, 7, 128], 300), (2, 300, 1, 64, 500, [-3, 90], 50)]


@pytest.mark.parametrize("case", SHARED, ids=[f"B{c[0]}h{c[1]}P{c[4]}" for c in SHARED])
def test_shared(libs, monkeypatch, case):
    B, h_q, h_kv, d, P, lens, n_max = case
    q, Kp, Vp, K, V = rand(2, (B, h_q, d), (h_kv, P + 5, d), (h_kv, P + 5, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d))
    for out_dtype in OUTS:
        both(libs, monkeypatch, lambda e: [api.decode_attn_shared(q, Kp, Vp, K, V, i32(lens), prefix_len=P, dev_error=e,
                                                                  out_dtype=out_dtype)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128), (256, 256)])
def test_rope(libs, monkeypatch, dtype, d, d_v):
    B, T, h_q, h_kv, n_max = 3, 130, 7, 3, 150
    x, v, K, V, w = (t.to(dtype) for t in rand(3, (B, T, h_q + h_kv, d), (B, T, h_kv, d_v), (B, h_kv, n_max, d),
                                                (B, h_kv, n_max, d_v), (d,)))
    cos, sin = (torch.randn(400, d // 2, device="cuda") for _ in range(2))
    for pos, news, at in (([0, 20, 149], [130, 0, 1], None), ([-1, 150, 21], [5, 1, 140], [0, 390, 5])):
        def run(e):
            K2, V2 = K.clone(), V.clone()
            q_out = torch.zeros((B, h_q, T, d), dtype=dtype, device="cuda")
            api.kv_append_rope(x[:, :, :h_q].transpose(1, 2), x[:, :, h_q:].transpose(1, 2), v.transpose(1, 2), K2, V2,
                               i32(pos), cos, sin, q_weight=w, k_weight=w, n_new=i32(news), q_out=q_out, dev_error=e,
                               angle_pos=None if at is None else i32(at))
            return [q_out, K2, V2]
        both(libs, monkeypatch, run)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["chunk", "cut", "shared"])
def test_withheld_stage(libs, monkeypatch, kind, d):
    q, K, V, Kp, Vp = rand(4, (2, 8, 40, d), (2, 2, 3000, d), (2, 2, 3000, d), (2, 700, d), (2, 700, d))
    lens = i32([200, 90] if kind == "chunk" else [3000, 1234])

    def run(e=None):
        if kind == "shared":
            return api.decode_attn_shared(q[:, :, 0].contiguous(), Kp, Vp, K, V, lens, dev_error=e)
        n = 900 if kind == "chunk" else 3000
        return api.chunk_attn(q, K[:, :, :n].contiguous(), V[:, :, :n].contiguous(), lens, dev_error=e)
    want = run()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setattr(api, "_lib", libs[1])
    libs[1].decode_attn_test_withhold(0)
    try:
        run(err)
        torch.cuda.synchronize()
    finally:
        libs[1].decode_attn_test_withhold(-1)
    assert int(err) & api.DEVERR_TIMEOUT
    err.zero_()
    assert torch.equal(run(err), want) and int(err) == 0
    monkeypatch.setattr(api, "_lib", libs[0])
    assert torch.equal(run(err), want) and int(err) == 0
