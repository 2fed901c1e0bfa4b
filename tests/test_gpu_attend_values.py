"""Infinities and NaN in rows of V that some tokens of a chunk see and others do not (needs a GB300)."""
import ctypes
import math

import pytest
import torch

import attend_bounds as A
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.build import build

pytestmark = pytest.mark.gpu
OUTS = [torch.bfloat16, torch.float32]
OID = ["bf16", "fp32"]
BAD = [float("inf"), float("nan"), -float("inf")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(B, T, h_q, h_kv, d, n_max, lens, news, bad, out_dtype, window=0, prefix=0, seed=0):
    """bad: (sequence, row, column) of V that is not finite.  Tokens that see it are not finite in that column, every
    other output is as if it were not there."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16()
               for s in ((B, T, h_q, d), (B, h_kv, n_max, d), (B, h_kv, n_max, d)))
    q = (2 * q).transpose(1, 2)
    Vx = V.clone()
    hit = torch.zeros((B, T, d), dtype=torch.bool, device="cuda")
    for k, (b, row, col) in enumerate(bad):
        V[b, :, row, col], Vx[b, :, row, col] = 0, BAD[k % 3]
        for i in range(news[b]):
            p = lens[b] - news[b] + i
            if row <= p and (not window or row > p - window or row < prefix):
                hit[b, i, col] = True
    assert hit.any() and not hit.all()
    hit = hit[:, None].expand(B, h_q, T, d)
    out = torch.zeros((B, T, h_q, d), dtype=out_dtype, device="cuda").transpose(1, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.chunk_attn(q, K, Vx, i32(lens), n_new=i32(news), window=window, prefix=prefix, out=out, dev_error=err)
    assert int(err) == 0
    assert not out[hit].isfinite().any()
    want, tol = A.chunk(q, K, V, lens, news, 1 / math.sqrt(d), out_dtype, window, prefix)
    A.check(torch.where(hit, 0, out), torch.where(hit, 0, want), torch.where(hit, 0, tol))


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d", [64, 128])
def test_later_rows(d, out_dtype):
    """A token's own row and those behind it, in whole units of one and of two streams, and cut ones."""
    run(2, 5, 4, 2, d, 200, [200, 5], [5, 5], [(0, 197, 3), (1, 0, 0), (1, 4, d - 1)], out_dtype)
    run(2, 300, 2, 1, d, 700, [700, 300], [300, 299], [(0, 500, 7), (0, 650, 7), (0, 699, 0), (1, 128, 9), (1, 299, 20)],
        out_dtype, seed=1)
    run(1, 290, 1, 1, d, 9000, [9000], [290], [(0, 8800, 1), (0, 8999, 2), (0, 8960, 3)], out_dtype, seed=2)
    run(2, 6, 16, 2, d, 12000, [12000, 400], [6, 6], [(0, 11998, 5), (1, 396, 5)], out_dtype, seed=3)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_behind_the_window(d, out_dtype):
    """Rows that the first tokens' windows still hold and the last ones' do not, and the always-seen ones."""
    run(2, 150, 4, 2, d, 900, [900, 431], [150, 90], [(0, 760, 1), (0, 700, 2), (1, 300, 3), (1, 400, 4)], out_dtype,
        window=64, seed=4)
    run(2, 290, 2, 1, d, 1500, [1500, 290], [290, 290], [(0, 1100, 1), (0, 1010, 6), (0, 1400, 2), (1, 150, 3)], out_dtype,
        window=200, prefix=130, seed=5)
    run(1, 40, 8, 1, d, 9000, [9000], [40], [(0, 5990, 1), (0, 5999, 2), (0, 8990, 3)], out_dtype, window=3000, prefix=200,
        seed=6)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_one_tile_of_queries_does_not_see(d, out_dtype):
    """Rows behind a row tile's last token (a later tile's tokens see them), and every value of a tile."""
    run(1, 600, 2, 1, d, 600, [600], [600], [(0, 64, 1), (0, 127, 2), (0, 128, 3), (0, 255, 4), (0, 256, 5), (0, 599, 6)],
        out_dtype, seed=7)
    run(1, 128, 1, 1, d, 128, [128], [128], [(0, r, c) for r in range(100, 128) for c in range(d)], out_dtype, seed=8)


def test_shared_prefix():
    """Rows of one sequence, and of the prefix, which every sequence sees."""
    g = torch.Generator(device="cuda").manual_seed(9)
    q, Kp, Vp, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16()
                       for s in ((5, 8, 64), (2, 300, 64), (2, 300, 64), (5, 2, 200, 64), (5, 2, 200, 64)))
    n = [200, 0, 33, 128, 129]
    want, tol = A.shared(q, Kp, Vp, 300, K, V, n, 0.125, torch.float32)
    V[0, :, 199, 3] = V[2, :, 0, 4] = float("nan")
    V[3, :, 128:] = K[3, :, 128:] = float("nan")
    Vp[:, 299, 7] = float("inf")
    hit = torch.zeros_like(want, dtype=torch.bool)
    hit[0, :, 3] = hit[2, :, 4] = hit[:, :, 7] = True
    out = api.decode_attn_shared(q, Kp, Vp, K, V, i32(n))
    assert not out[hit].isfinite().any()
    A.check(torch.where(hit, 0, out), torch.where(hit, 0, want), torch.where(hit, 0, tol))


@pytest.fixture(scope="module")
def checked():
    lib = ctypes.CDLL(build(test_hooks=True))
    for name, (res, args) in api.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


@pytest.mark.parametrize("n_max,window,prefix", [(700, 0, 0), (700, 90, 30), (9000, 0, 0), (9000, 2000, 3)])
@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
def test_in_the_checked_build(checked, monkeypatch, out_dtype, n_max, window, prefix):
    """No index out of range, and the product build's bits."""
    g = torch.Generator(device="cuda").manual_seed(10)
    B, T, h_q, h_kv, d = 2, 70, 6, 2, 128
    q, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((B, h_q, T, d), (B, h_kv, n_max, d),
                                                                               (B, h_kv, n_max, d)))
    for row in (0, 1, n_max - 75, n_max - 70, n_max - 30, n_max - 1, 300, 369):
        V[:, :, row, row % d] = float("nan")
    lens, got = i32([n_max, 370]), []
    product = api._lib
    for lib in (product, checked):
        monkeypatch.setattr(api, "_lib", lib)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got.append(api.chunk_attn(q, K, V, lens, window=window, prefix=prefix, out_dtype=out_dtype, dev_error=err))
        assert int(err) == 0
    assert got[0].isnan().any() and torch.equal(got[0].contiguous().view(torch.uint8), got[1].contiguous().view(torch.uint8))


@pytest.mark.parametrize("group", [1, 4])
def test_nothing_finite(group):
    """A sequence all of whose values are NaN: its outputs are, the other's are not, and no wait runs out."""
    B, T, h_kv, d = 2, 2048, 4, 128
    g = torch.Generator(device="cuda").manual_seed(11)
    q, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((B, h_kv * group, T, d), (B, h_kv, T, d),
                                                                               (B, h_kv, T, d)))
    for window in (0, 300):
        want = api.chunk_attn(q, K, V, i32([T, T]), window=window)
        Vx = V.clone()
        Vx[1] = float("nan")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = api.chunk_attn(q, K, Vx, i32([T, T]), window=window, dev_error=err)
        assert int(err) == 0
        assert torch.equal(out[0], want[0]) and out[1].isnan().all()


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("window,prefix", [(0, 0), (20, 0), (20, 35)])
def test_signs(window, prefix, out_dtype):
    """Of rows that not every token sees: an infinity where only one sign is seen, NaN where both are or one is NaN."""
    T, d = 128, 64
    g = torch.Generator(device="cuda").manual_seed(12)
    q, K, V = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((1, 2, T, d), (1, 1, T, d), (1, 1, T, d)))
    inf = float("inf")
    V[0, 0, 50, 3], V[0, 0, 60, 4], V[0, 0, 30, 5], V[0, 0, 45, 5], V[0, 0, 100, 6], V[0, 0, 33, 7] = inf, -inf, inf, -inf, \
        float("nan"), -inf
    out = torch.zeros((1, 2, T, d), dtype=out_dtype, device="cuda")
    api.chunk_attn(q, K, V, i32([T]), window=window, prefix=prefix, out=out)
    for p in range(T):
        for c in range(8):
            seen = V[0, 0, [l for l in range(p + 1) if not window or l > p - window or l < prefix], c]
            bad = seen[~seen.isfinite()]
            for got in out[0, :, p, c]:
                if not bad.numel():
                    assert got.isfinite()
                elif bad.isnan().any() or bad.unique().numel() == 2:
                    assert got.isnan()
                else:
                    assert got == bad[0]
