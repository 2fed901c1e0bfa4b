"""The block-scaled 8-bit cache: written, read back and attended (needs a GB300).

The write is checked code for code against the definition in 64 bits, the read
value for value, the decode against plain 64-bit attention on the values the
codes and scales stand for."""
import math

import numpy as np
import pytest
import torch

import terms_reference as R
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod

pytestmark = pytest.mark.gpu
KINDS = [torch.int8, torch.float8_e4m3fn]
KID = ["int8", "fp8"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def nblk(n, block):
    return -(-n // block)


def random_cache(B, h, n_max, d, block, dtype, seed, pow2=True, spread=3.0):
    """Random codes (no NaN) and positive scales."""
    g = torch.Generator().manual_seed(seed)
    codes = []
    for _ in range(2):
        v = torch.randn(B, h, n_max, d, generator=g) * R.Q[dtype] / 4
        codes.append(R.as_codes(R.round_codes(v.double().numpy(), dtype), dtype))
    scales = []
    for _ in range(2):
        e = torch.randn(B, h, nblk(n_max, block), generator=g) * spread - 5
        scales.append(torch.exp2(e.round() if pow2 else e))
    return codes[0], codes[1], scales[0], scales[1]


# ----------------------------------------------------------------- write
def same_codes(got, want, dtype):
    """Codes equal as values (int8: as bytes; e4m3: +0 and -0 are one value)."""
    return torch.equal(got.cpu().float(), want.float())


def write_case(B, h, d, n_max, block, dtype, x_dtype, pos, m, T, seed=0, strided=False, scale_of=None,
               old_scale=None, use_n_new=True):
    g = torch.Generator().manual_seed(seed)
    K, V, ks, vs = random_cache(B, h, n_max, d, block, dtype, seed + 1)
    if old_scale is not None:
        ks, vs = torch.full_like(ks, old_scale), torch.full_like(vs, old_scale)
    H = h * 3 if strided else h
    x = torch.randn(B, T, H, d, generator=g)
    if scale_of is not None:
        x = x * scale_of(g, x.shape)
    x = x.to(x_dtype)
    kn, vn = x[:, :, :h].transpose(1, 2), x[:, :, -h:].transpose(1, 2)
    xd = x.cuda()
    knd, vnd = xd[:, :, :h].transpose(1, 2), xd[:, :, -h:].transpose(1, 2)
    if not strided:
        knd, vnd = knd.contiguous(), vnd.contiguous()
    for b in range(B):  # rows that are not written are not read
        knd[b, :, m[b]:] = float("nan")
        vnd[b, :, m[b]:] = float("nan")
    Kd, Vd, ksd, vsd = K.cuda(), V.cuda(), ks.cuda(), vs.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_append_q8b(knd, vnd, Kd, Vd, ksd, vsd, i32(pos), block, n_new=i32(m) if use_n_new else None,
                      dev_error=err)
    assert int(err) == 0
    for codes, sc, new, cd, sd in ((K, ks, kn, Kd, ksd), (V, vs, vn, Vd, vsd)):
        wc, ws = R.append(codes.double().numpy(), sc.double().numpy(), new.double().numpy(), pos, m,
                          block, dtype)
        torch.testing.assert_close(sd.cpu().double(), torch.from_numpy(ws), rtol=0, atol=0)
        assert torch.equal(cd.cpu().double(), torch.from_numpy(wc))


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_write(dtype, x_dtype, d, block):
    # one token: into an empty cache, at a block's start, inside and at the end of one, at the cache's end
    write_case(6, 2, d, 300, block, dtype, x_dtype, [0, block, block + 1, 2 * block - 1, 299, 7], [1] * 6, 1,
               use_n_new=False)
    # chunks: ragged counts, none among them, over several blocks, up to the last row
    write_case(5, 3, d, 517, block, dtype, x_dtype, [0, 5, 130, 500, 517], [301, 128, 0, 17, 0], 301, seed=3)
    # rows inside a projection's output
    write_case(2, 2, d, 300, block, dtype, x_dtype, [3, 64], [200, 200], 200, seed=4, strided=True)


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_write_grows_and_keeps(dtype):
    """Held rows are rewritten when a block's scale grows, and untouched when it does not."""
    for old in (2.0 ** -12, 2.0 ** -5, 8.0, 0.0, 0.013, 2.0 ** -126, 1e-40, 1e30):
        write_case(3, 2, 128, 256, 64, dtype, torch.float32, [10, 63, 100], [2, 40, 1], 40, seed=5, old_scale=old)


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_write_of_tiny_huge_and_zero_rows(dtype):
    for f in (0.0, 1e-45, 1e-39, 1e-30, 1e30, 2e37):
        write_case(2, 1, 64, 128, 32, dtype, torch.float32, [5, 0], [50, 3], 50, seed=6,
                   scale_of=lambda g, s: f)
    # rows and channels of very unequal size
    write_case(2, 2, 128, 256, 16, dtype, torch.bfloat16, [1, 30], [100, 99], 100, seed=7,
               scale_of=lambda g, s: torch.exp2(6 * torch.randn(s[0], s[1], 1, s[3], generator=g)))


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_write_at_the_scale_borders(dtype):
    """Maxima on both sides of Q times a power of two: the scale is the smallest that holds them."""
    top = R.Q[dtype]
    for e in (-120, -30, -1, 0, 5, 100):
        for a in (top * 2.0 ** e, np.nextafter(np.float32(top * 2.0 ** e), np.float32(np.inf)),
                  np.nextafter(np.float32(top * 2.0 ** e), np.float32(0)), 2.0 ** e):
            x = torch.zeros(1, 1, 2, 64)
            x[0, 0, 1, 63] = -float(a)
            K = torch.zeros(1, 1, 16, 64, dtype=torch.int8).to(dtype).cuda()
            V = K.clone()
            ks, vs = torch.full((1, 1, 1), 9.0, device="cuda"), torch.full((1, 1, 1), 9.0, device="cuda")
            api.kv_append_q8b(x.cuda(), x.cuda(), K, V, ks, vs, i32([0]), 16)
            assert float(ks) == R.need(float(a), top) and float(vs) == float(ks)


def test_write_out_of_range():
    """Positions and counts out of range: what fits is written, the rest flagged; nothing else changes."""
    B, h, d, n_max, block = 6, 2, 64, 100, 32
    K, V, ks, vs = random_cache(B, h, n_max, d, block, torch.int8, 1)
    x = torch.randn(B, h, 8, d)
    pos, n_new = [-1, 101, 96, 100, 50, 40], [8, 8, 8, 8, 99, -4]
    for p, c, flagged in [([pos[i]], [n_new[i]], True) for i in range(6)] + [([92], [8], False), ([100], [0], False),
                                                                            ([-9], [0], False)]:
        Kd, Vd, ksd, vsd = K[:1].cuda(), V[:1].cuda(), ks[:1].cuda(), vs[:1].cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.kv_append_q8b(x[:1].cuda(), x[:1].cuda(), Kd, Vd, ksd, vsd, i32(p), block, n_new=i32(c), dev_error=err)
        assert int(err) == (api.DEVERR_POS if flagged else 0), (p, c)
        m = min(max(c[0], 0), 8)
        m = 0 if p[0] < 0 or p[0] > n_max else min(m, n_max - p[0])
        wc, ws = R.append(K[:1].double().numpy(), ks[:1].double().numpy(), x[:1].double().numpy(),
                          [max(0, min(p[0], n_max))], [m], block, torch.int8)
        assert torch.equal(Kd.cpu().double(), torch.from_numpy(wc))
        assert torch.equal(ksd.cpu().double(), torch.from_numpy(ws))


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_write_of_values_that_are_none(dtype):
    """NaN and infinities become 0 and are flagged; the other elements are as if they were 0."""
    x = torch.randn(1, 2, 20, 64)
    bad = x.clone()
    bad[0, 0, 3, 5] = float("nan")
    bad[0, 1, 19, 0] = float("-inf")
    x[0, 0, 3, 5] = x[0, 1, 19, 0] = 0
    got = []
    for t in (x, bad):
        K, V, ks, vs = (c.cuda() for c in random_cache(1, 2, 64, 64, 16, dtype, 2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.kv_append_q8b(t.cuda(), x.cuda(), K, V, ks, vs, i32([9]), 16, dev_error=err)
        got.append((K.float(), V.float(), ks, vs, int(err)))
    assert got[0][4] == 0 and got[1][4] == api.DEVERR_VALUE
    for a, b in zip(got[0][:4], got[1][:4]):
        assert torch.equal(a, b)


def test_held_nan_codes_stay():
    """A block from elsewhere that holds NaN codes: its scale grows, the NaN rows still read as NaN."""
    K, V, ks, vs = random_cache(1, 1, 64, 64, 32, torch.float8_e4m3fn, 3)
    K.view(torch.uint8)[0, 0, 3, 7] = 0x7f
    K.view(torch.uint8)[0, 0, 40, 0] = 0xff
    nan = torch.isnan(K.float())
    Kd, Vd, ksd, vsd = K.cuda(), V.cuda(), ks.cuda(), vs.cuda()
    x = torch.full((1, 1, 2, 64), 1e6, device="cuda")
    for pos in (20, 50):
        api.kv_append_q8b(x, x, Kd, Vd, ksd, vsd, i32([pos]), 32)
        nan[0, 0, pos:pos + 2] = False
    assert bool((ksd.cpu() > ks).all())
    assert torch.equal(torch.isnan(Kd.cpu().float()), nan)


def test_write_of_broadcast_and_single_rows():
    """Strides of zero, and [B, h_kv, d] rows."""
    x = torch.randn(1, 1, 1, 64, device="cuda").expand(3, 2, 5, 64)
    y = x.contiguous()
    got = []
    for t in (x, y):
        K, V, ks, vs = (c.cuda() for c in random_cache(3, 2, 64, 64, 16, torch.int8, 2))
        api.kv_append_q8b(t, t, K, V, ks, vs, i32([0, 14, 59]), 16)
        api.kv_append_q8b(t[:, :, 0], y[:, :, 0], K, V, ks, vs, i32([20, 30, 1]), 16)
        got.append((K, V, ks, vs))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    with pytest.raises(api.DecodeAttnError, match="16-byte"):
        api.kv_append_q8b(torch.zeros(3 * 2 * 5 * 65, device="cuda").as_strided((3, 2, 5, 64), (650, 325, 65, 1)),
                          y, *got[0], i32([0, 0, 0]), 16)
    with pytest.raises(ValueError, match="contiguous"):
        api.kv_append_q8b(torch.zeros(3, 2, 64, 5, device="cuda").transpose(2, 3), y, *got[0], i32([0, 0, 0]), 16)


# ----------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_read(dtype, out_dtype, d):
    for block, n_max, pow2 in ((16, 300, True), (128, 517, False), (64, 64, True), (32, 33, False)):
        B, h = 4, 3
        K, V, ks, vs = random_cache(B, h, n_max, d, block, dtype, block, pow2)
        lens, begin = [n_max, 0, n_max // 2, n_max - 1], [0, 0, 5, n_max // 3]
        for rows in (1, 17, n_max, n_max + 40):
            k, v = (torch.full((B, h, rows, d), 77.0, dtype=out_dtype, device="cuda") for _ in range(2))
            api.kv_read_q8b(K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32(lens), block, row_begin=i32(begin),
                            k_out=k, v_out=v)
            for codes, sc, got in ((K, ks, k), (V, vs, v)):
                # the product is rounded to float, then to the output's type
                all_rows = (codes.float() * sc.repeat_interleave(block, 2)[:, :, :n_max, None]).to(out_dtype)
                want = torch.full((B, h, rows, d), 77.0, dtype=out_dtype)
                for b in range(B):
                    n = max(0, min(rows, lens[b] - begin[b]))
                    want[b, :, :n] = all_rows[b, :, begin[b]:begin[b] + n]
                assert torch.equal(got.cpu(), want)
    k, v = api.kv_read_q8b(K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32(lens), block, out_dtype=out_dtype)
    assert k.shape == (B, h, n_max, d) and k.dtype == out_dtype


def test_read_of_many_sequences():
    """More sequences than are counted at a time, most of them without rows to read."""
    B, h, n_max, d, block = 1100, 1, 70, 64, 16
    K, V, ks, vs = random_cache(B, h, n_max, d, block, torch.int8, 5)
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, n_max + 1, (B,), generator=g).tolist()
    begin = [n if b % 3 else max(0, n - 9) for b, n in enumerate(lens)]
    for rows in (5, 200):
        k, v = (torch.full((B, h, rows, d), 77.0, device="cuda") for _ in range(2))
        api.kv_read_q8b(K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32(lens), block, row_begin=i32(begin), k_out=k,
                        v_out=v)
        for codes, sc, got in ((K, ks, k), (V, vs, v)):
            all_rows = codes.float() * sc.repeat_interleave(block, 2)[:, :, :n_max, None]
            want = torch.full((B, h, rows, d), 77.0)
            for b in range(B):
                n = max(0, min(rows, lens[b] - begin[b]))
                want[b, :, :n] = all_rows[b, :, begin[b]:begin[b] + n]
            assert torch.equal(got.cpu(), want)


def test_decode_of_very_unequal_lengths():
    """One long sequence among many short ones: its unit is cut further than the others'."""
    for B, h_q, h_kv, d in ((60, 4, 2, 128), (300, 8, 2, 64), (9, 16, 1, 128), (5, 4, 1, 64)):
        lens = [(b * 7) % 90 for b in range(B)]
        lens[B // 2] = 2500
        decode_case(B, h_q, h_kv, d, 2500, lens, torch.int8, 32)
    decode_case(20, 8, 4, 128, 6000, [(b * 11) % 150 for b in range(20)], torch.float8_e4m3fn, 16)


def test_read_out_of_range():
    K, V, ks, vs = (c.cuda() for c in random_cache(3, 1, 50, 64, 16, torch.int8, 1))
    for lens, begin in (([60, 50, 50], [0, 0, 0]), ([50, -2, 50], [0, 0, 0]), ([50, 50, 50], [0, -1, 0])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = api.kv_read_q8b(K, V, ks, vs, i32(lens), 16, row_begin=i32(begin), out_dtype=torch.float32,
                               dev_error=err)
        assert int(err) == api.DEVERR_SEQ_LEN
        full, _ = api.kv_read_q8b(K, V, ks, vs, i32([50, 50, 50]), 16, out_dtype=torch.float32)
        assert torch.equal(k[0], full[0]) and torch.equal(k[2], full[2])
        assert (not k[1].any()) == (lens[1] < 0 or begin[1] < 0)


# ----------------------------------------------------------------- decode
def decode_case(B, h_q, h_kv, d, n_max, lens, dtype, block, terms=None, seed=0, splits=0, pow2=True, spread=2.0,
                q_scale=1.0, scales=None, out_dtype=torch.float32):
    terms = terms or {}
    K, V, ks, vs = random_cache(B, h_kv, n_max, d, block, dtype, seed, pow2, spread)
    if scales is not None:
        ks, vs = scales(ks, vs)
    q = (q_scale * torch.randn(B, h_q, d, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)
    begin = terms.get("begin")
    Kv = torch.from_numpy(R.values(K.double().numpy(), ks.double().numpy(), block))
    Vv = torch.from_numpy(R.values(V.double().numpy(), vs.double().numpy(), block))
    # what is not seen holds anything: NaN codes (e4m3), NaN scales of blocks without a seen row
    vmax = 0.0
    for b, n in enumerate(lens):
        seen = set(R.seen_rows(n, terms.get("window", 0), terms.get("prefix", 0), begin[b] if begin else 0))
        hidden = [l for l in range(n_max) if l not in seen]
        junk = torch.tensor(float("nan")).to(dtype) if dtype != torch.int8 else torch.tensor(-128, dtype=dtype)
        K.view(torch.uint8)[b, :, hidden] = junk.view(torch.uint8)
        V.view(torch.uint8)[b, :, hidden] = junk.view(torch.uint8)
        for i in range(nblk(n_max, block)):
            if not any(l in seen for l in range(i * block, min((i + 1) * block, n_max))):
                ks[b, :, i] = vs[b, :, i] = float("nan")
        if seen:
            vmax = max(vmax, float(Vv[b][:, sorted(seen)].abs().max()))
    sl, bg = terms.get("slopes"), terms.get("begin")
    mod = None
    if terms:
        mod = ScoreMod(softcap=terms.get("softcap", 0.0),
                       slopes=None if sl is None else torch.tensor(sl, device="cuda"),
                       window=terms.get("window", 0), prefix=terms.get("prefix", 0),
                       doc_begin=None if bg is None else i32(bg))
    sm_scale = 1 / math.sqrt(d)
    out = torch.full((B, h_q, d), float("nan"), dtype=out_dtype, device="cuda")
    api.decode_attn_q8b(q.cuda(), K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32(lens), block, mod=mod, out=out,
                        num_splits=splits)
    sl = None if sl is None else torch.tensor(sl).tolist()
    want, size = R.attend(q, Kv, Vv, lens, sm_scale, terms.get("softcap", 0.0), sl, terms.get("window", 0),
                          terms.get("prefix", 0), bg)
    # weights: fp16 head + fp16 remainder, 2^-22 of them
    eps = torch.finfo(out_dtype).eps if out_dtype == torch.bfloat16 else 0.0
    tol = R.tolerance(d, size, terms.get("softcap", 0.0), vmax, max(max(lens), 1), 21, eps)
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    err = float((got - want).abs().max())
    assert err <= tol, f"max abs error {err:.3e} > {tol:.3e}"


DECODE = [
    # B, h_q, h_kv, d, n_max, lens
    (2, 2, 2, 64, 300, [300, 1]),
    (3, 8, 1, 64, 517, [517, 0, 129]),
    (2, 24, 2, 64, 260, [260, 127]),
    (1, 32, 1, 64, 333, [333]),
    (3, 8, 2, 128, 700, [700, 0, 385]),
    (2, 8, 1, 128, 300, [299, 128]),
    (2, 18, 2, 128, 400, [400, 17]),
    (1, 32, 1, 128, 1000, [999]),
    (1, 80, 2, 128, 200, [200]),
]


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("shape", DECODE, ids=[f"d{s[3]}h{s[1]}kv{s[2]}" for s in DECODE])
def test_decode(shape, dtype):
    for block in (16, 32, 64, 128):
        decode_case(*shape, dtype, block, seed=block)
    decode_case(*shape, dtype, 32, seed=1, pow2=False, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("shape", DECODE, ids=[f"d{s[3]}h{s[1]}kv{s[2]}" for s in DECODE])
def test_decode_with_terms(shape, dtype):
    B, h_q = shape[:2]
    slopes = [2.0 ** (-8 * (h + 1) / h_q) for h in range(h_q)]
    decode_case(*shape, dtype, 16, {"softcap": 20.0}, seed=1)
    decode_case(*shape, dtype, 64, {"slopes": slopes, "window": 130, "prefix": 20}, seed=2)
    decode_case(*shape, dtype, 32, {"softcap": 5.0, "slopes": [-s for s in slopes], "prefix": 3,
                                    "begin": [100 * b + 60 for b in range(B)]}, seed=3)
    decode_case(*shape, dtype, 128, {"window": 1}, seed=4)


@pytest.mark.parametrize("splits", [1, 2, 5, 300, -1])
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_decode_splits(dtype, splits):
    for heads in ((2, 8, 2, 128), (2, 16, 1, 128), (2, 4, 2, 64)):
        decode_case(*heads, 2100, [2099, 700], dtype, 16, seed=splits + 5, splits=splits)
        decode_case(*heads, 2100, [2099, 700], dtype, 64, {"window": 900, "prefix": 130}, seed=splits + 5,
                    splits=splits)


def test_decode_more_than_32_stages_of_scales():
    """A warp's scales are loaded 32 stages at a time: items of 32, 33 and 65 stages."""
    for n in (4096, 4097, 8320):
        decode_case(1, 4, 1, 128, n, [n], torch.int8, 16, splits=1)
        decode_case(1, 4, 1, 64, n, [n], torch.float8_e4m3fn, 128, {"window": n - 100, "prefix": 30}, splits=1)


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_decode_scales_of_any_size(dtype):
    """V scales far below and above what fp16 holds, unequal between blocks, and zero."""
    shape = (2, 8, 2, 128, 600, [600, 333])
    for f in (2.0 ** -126, 1e-30, 1e-6, 1e6, 1e28):
        decode_case(*shape, dtype, 16, scales=lambda ks, vs: (ks, vs * f))
    decode_case(*shape, dtype, 16, spread=8.0, q_scale=0.01)
    decode_case(*shape, dtype, 16, scales=lambda ks, vs: (ks * 0, vs))
    decode_case(*shape, dtype, 16, scales=lambda ks, vs: (ks, vs * 0))

    def some_zero(ks, vs):
        vs = vs.clone()
        vs[:, :, ::3] = 0
        vs[:, :, 1] *= -1
        return ks, vs
    decode_case(*shape, dtype, 16, scales=some_zero)


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_decode_chunks_by_length(dtype):
    """Few sequences of more rows than a cluster takes: chunks from the actual lengths."""
    decode_case(3, 8, 2, 128, 9000, [9000, 0, 4100], dtype, 16)
    decode_case(2, 32, 1, 128, 5003, [1, 5003], dtype, 32, {"softcap": 8.0, "window": 4999, "prefix": 130})


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_decode_clusters(dtype):
    """One to eight CTAs a unit: shares that end with the rows, inside a step and empty ones."""
    for n in (129, 256, 257, 385, 640, 769, 1024, 1025, 2047, 4096):
        decode_case(2, 4, 2, 64, n, [n, n // 3], dtype, 16, seed=n)
    for n in (129, 500, 1024, 3070):
        decode_case(2, 40, 2, 128, n, [0, n], dtype, 64, seed=n, out_dtype=torch.bfloat16)
    # an SM or less to each: clusters of three and two, and one CTA each
    for B in (24, 38, 100):
        decode_case(B, 4, 2, 64, 400, [(b * 61) % 401 for b in range(B)], dtype, 32, seed=B)
    # windows: the rows that are seen are shared
    decode_case(2, 8, 2, 128, 9000, [9000, 700], dtype, 16, {"window": 900, "prefix": 40})
    decode_case(2, 8, 2, 128, 9000, [9000, 700], dtype, 128, {"window": 1, "prefix": 3000})


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("far", [0, 8])
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_decode_behind_a_much_larger_scale(dtype, far, out_dtype):
    """The weight lies on block 1 alone, and block `far`, seen by the same warp with no weight, has
    a V scale 2^k times as large: the output keeps its digits.

    Bound, relative to block 1's largest value: the 16 rows' scores are equal, so their weights
    are off by fp16 alone, 2^-22 in two parts and 2^-12 in one, or by half a step of fp16's
    subnormals, 2^-25, against the 2^(7 - k) that a row's weight counts in units of the large
    scale; 16 products and the merge, under 64 float roundings of 2^-24; the output's own
    rounding."""
    d, n, block = 64, 200, 16
    for k in (0, 8, 12, 16, 20):
        K, V, ks, vs = random_cache(1, 1, n, d, block, dtype, k + 1)
        K = torch.zeros(1, 1, n, d)
        K[..., 0] = -100.0
        K[0, 0, 16:32, 0] = 100.0
        K = K.to(dtype)
        kv = float(K[0, 0, 16, 0].float())
        ks = torch.full_like(ks, 0.1)
        vs = torch.full_like(vs, 2.0 ** -9)
        vs[0, 0, far] = 2.0 ** (k - 9)
        q = torch.zeros(1, 2, d, dtype=torch.bfloat16)
        q[..., 0] = 8.0 * 100.0 / kv
        out = api.decode_attn_q8b(q.cuda(), K.cuda(), V.cuda(), ks.cuda(), vs.cuda(), i32([n]), block, scale=1.0,
                                  out_dtype=out_dtype).cpu().double()
        rows = V[0, 0, 16:32].double() * 2.0 ** -9
        want = rows.mean(0).expand(2, d)
        # (the other rows: weights of e^-160, times 2^20, are nothing)
        part = 2.0 ** -22 if out_dtype == torch.float32 else 2.0 ** -12 + torch.finfo(out_dtype).eps / 2
        tol = float(rows.abs().max()) * (part + 2.0 ** (k - 32) + 64 * 2.0 ** -24)
        err = float((out[0] - want).abs().max())
        assert err <= tol, (k, err, tol)


def test_decode_batch_above_one_launch_and_many_items():
    lens = [(b * 37) % 200 for b in range(600)]
    decode_case(600, 2, 1, 64, 200, lens, torch.int8, 16, {"window": 50})
    decode_case(300, 8, 8, 64, 200, lens[:300], torch.float8_e4m3fn, 32, {"prefix": 4, "window": 60}, splits=3)


# ----------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("terms", [{}, {"softcap": 20.0, "window": 100, "prefix": 4}], ids=["plain", "terms"])
def test_prompt_chunks_then_steps(dtype, terms):
    """A prompt written in ragged chunks, then single tokens, each step attended and read back."""
    B, h_q, h_kv, d, n_max, block = 3, 8, 2, 128, 400, 32
    g = torch.Generator().manual_seed(9)
    codes = [np.zeros((B, h_kv, n_max, d)) for _ in range(2)]
    scales = [np.zeros((B, h_kv, nblk(n_max, block))) for _ in range(2)]
    Kd, Vd = (torch.zeros((B, h_kv, n_max, d), dtype=torch.int8, device="cuda").view(dtype) for _ in range(2))
    ksd, vsd = (torch.zeros(scales[0].shape, device="cuda") for _ in range(2))
    lens = [0, 0, 0]
    mod = ScoreMod(**terms) if terms else None
    for step, T in enumerate([150, 97, 1, 1, 1, 1, 5, 1]):
        m = [T, T // 2, 0 if T > 1 else 1]
        x = [torch.randn(B, h_kv, T, d, generator=g) * (1 + step) for _ in range(2)]
        x = [t.to(torch.bfloat16) for t in x]
        api.kv_append_q8b(x[0].cuda(), x[1].cuda(), Kd, Vd, ksd, vsd, i32(lens), block, n_new=i32(m))
        for i in range(2):
            codes[i], scales[i] = R.append(codes[i], scales[i], x[i].double().numpy(), lens, m, block, dtype)
        lens = [n + k for n, k in zip(lens, m)]
        ld = i32(lens)
        q = torch.randn(B, h_q, d, generator=g).to(torch.bfloat16)
        out = api.decode_attn_q8b(q.cuda(), Kd, Vd, ksd, vsd, ld, block, mod=mod)
        k, v = api.kv_read_q8b(Kd, Vd, ksd, vsd, ld, block, out_dtype=torch.float32)
        want_k, want_v = (torch.from_numpy(R.values(codes[i], scales[i], block)) for i in range(2))
        for b, n in enumerate(lens):
            assert torch.equal(k[b, :, :n].cpu().double(), want_k[b, :, :n])
            assert torch.equal(v[b, :, :n].cpu().double(), want_v[b, :, :n])
            assert not k[b, :, n:].any() and not v[b, :, n:].any()
        want, size = R.attend(q, want_k, want_v, lens, 1 / math.sqrt(d), **terms)
        tol = R.tolerance(d, size, terms.get("softcap", 0.0), float(want_v.abs().max()), max(lens), 21)
        assert float((out.cpu().double() - want).abs().max()) <= tol


def test_step_in_a_graph():
    """A captured write + decode, replayed with new tokens and lengths."""
    B, h_q, h_kv, d, n_max, block = 2, 8, 2, 128, 300, 16
    bufs = random_cache(B, h_kv, n_max, d, block, torch.int8, 3, spread=0.0)
    K, V, ks, vs = (c.cuda() for c in bufs)
    ref = [bufs[0].double().numpy(), bufs[1].double().numpy()]
    sc = [bufs[2].double().numpy(), bufs[3].double().numpy()]
    x = [torch.zeros(B, h_kv, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = torch.zeros(B, h_q, d, dtype=torch.bfloat16, device="cuda")
    pos, lens = i32([20, 200]), i32([21, 201])
    keep = [t.clone() for t in (K, V, ks, vs)]

    def step():
        api.kv_append_q8b(x[0], x[1], K, V, ks, vs, pos, block)
        return api.decode_attn_q8b(q, K, V, ks, vs, lens, block)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t, s in zip((K, V, ks, vs), keep):
        t.copy_(s)
    gen = torch.Generator().manual_seed(1)
    at = [20, 200]
    for i in range(5):
        new = [(torch.randn(B, h_kv, 1, d, generator=gen) * 2.0 ** i).to(torch.bfloat16) for _ in range(2)]
        nq = torch.randn(B, h_q, d, generator=gen).to(torch.bfloat16)
        for t, s in zip((*x, q), (*new, nq)):
            t.copy_(s)
        pos.copy_(torch.tensor(at, dtype=torch.int32))
        lens.copy_(torch.tensor([a + 1 for a in at], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for j in range(2):
            ref[j], sc[j] = R.append(ref[j], sc[j], new[j].double().numpy(), at, [1, 1], block, torch.int8)
        at = [a + 1 for a in at]
        want_k, want_v = (torch.from_numpy(R.values(ref[j], sc[j], block)) for j in range(2))
        want, size = R.attend(nq, want_k, want_v, at, 1 / math.sqrt(d))
        tol = R.tolerance(d, size, 0.0, float(want_v.abs().max()), max(at), 21)
        assert float((out.cpu().double() - want).abs().max()) <= tol
