"""The block-scaled decode with and without score terms, every output element held to a bound of
its own, for float32 and bf16 outputs, by work list and by clusters (needs a GB300)."""
import math

import pytest
import torch

import decode_bounds as D
import terms_reference as R
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod

pytestmark = pytest.mark.gpu
KINDS = [torch.int8, torch.float8_e4m3fn]
KID = ["int8", "fp8"]
OUTS = [torch.float32, torch.bfloat16]
OID = ["fp32", "bf16"]
FLOOR = 2.0 ** -31  # half a step of fp16's subnormals, 2^-25, of a largest product of 2^6 or more


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(shape, n_max, lens, block, dtype, out_dtype, splits=0, seed=0, spread=1.0, softcap=0.0, slopes=None, window=0,
        prefix=0, begin=None, scale=None):
    h_q, h_kv, d = shape
    B, nblk = len(lens), -(-n_max // block)
    g = torch.Generator(device="cuda").manual_seed(seed)
    top = R.Q[dtype]

    def cache():
        v = (torch.randn((B, h_kv, n_max, d), generator=g, device="cuda") * top / 4).clamp(-top, top)
        c = v.round().to(torch.int8) if dtype == torch.int8 else v.to(dtype)
        return c, torch.exp2(torch.randn((B, h_kv, nblk), generator=g, device="cuda") * spread) * (4 / top)
    (K, ks), (V, vs) = cache(), cache()
    q = torch.randn((B, h_q, d), generator=g, device="cuda").to(torch.bfloat16)
    at = torch.arange(n_max, device="cuda") // block
    Kv, Vv = K.double() * ks[:, :, at, None].double(), V.double() * vs[:, :, at, None].double()
    rows = torch.arange(n_max, device="cuda")
    for b, n in enumerate(lens):  # what is not seen holds anything
        first = 0 if begin is None else begin[b]
        first = max(first, n - window) if window else first
        seen = (rows < n) & ((rows < prefix) | (rows >= first))
        junk = torch.tensor(-128, dtype=torch.int8, device="cuda") if dtype == torch.int8 else \
            torch.tensor(float("nan"), device="cuda").to(dtype)
        K.view(torch.uint8)[b, :, ~seen] = junk.view(torch.uint8)
        V.view(torch.uint8)[b, :, ~seen] = junk.view(torch.uint8)
        dead = torch.zeros(nblk * block, dtype=torch.bool, device="cuda")
        dead[:n_max] = seen
        dead = ~dead.view(nblk, block).any(1)
        ks[b, :, dead] = vs[b, :, dead] = float("nan")
    mod = None
    if softcap or slopes is not None or window or prefix or begin is not None:
        mod = ScoreMod(softcap=softcap, window=window, prefix=prefix, doc_begin=None if begin is None else i32(begin),
                       slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.full((B, h_q, d), float("nan"), dtype=out_dtype, device="cuda")
    api.decode_attn_q8b(q, K, V, ks, vs, i32(lens), block, mod=mod, out=out, scale=scale, num_splits=splits)
    want, tol = D.attend(q, Kv, Vv, lens, scale, D.weight_rounding("q8b", out_dtype), out_dtype, softcap, slopes, window,
                         prefix, begin, floor=FLOOR)
    D.check(out, want, tol, f"{shape} {lens} block {block} splits {splits} cap {softcap} window {window} prefix {prefix}")


SHAPES = [(2, 2, 64), (24, 2, 64), (33, 1, 64), (8, 2, 128), (8, 1, 128), (18, 2, 128), (32, 1, 128)]
SID = [f"d{s[2]}h{s[0]}kv{s[1]}" for s in SHAPES]


def falling(h_q, sign=1):
    return [sign * 2.0 ** (-8 * (h + 1) / h_q) for h in range(h_q)]


def all_terms(h_q):
    return [
        {},
        {"softcap": 20.0},
        {"softcap": 50.0, "window": 400, "prefix": 4},
        {"slopes": falling(h_q), "window": 430, "prefix": 20},
        {"slopes": [(-1) ** h * s for h, s in enumerate(falling(h_q))]},
        {"softcap": 5.0, "slopes": falling(h_q, -1), "prefix": 3, "begin": [60, 333]},
        {"begin": [511, 640], "prefix": 130},
        {"window": 1},
    ]


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("which", range(8))
@pytest.mark.parametrize("shape", SHAPES, ids=SID)
def test_terms(shape, which, dtype, out_dtype):
    terms = all_terms(shape[0])[which]
    for splits, block in ((0, 16), (1, 128), (3, 32), (5, 64)):
        run(shape, 901, [901, 640], block, dtype, out_dtype, splits, seed=which, **terms)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[3], SHAPES[6]], ids=[SID[1], SID[3], SID[6]])
def test_caps(shape, dtype, out_dtype):
    for cap in (0.05, 1.0, 30.0, 100.0, 128.0, 129.0, 1e4):
        for scale in (None, 1.0):
            for splits in (0, 2):
                run(shape, 700, [700, 333], 32, dtype, out_dtype, splits, softcap=cap, scale=scale)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("spread", [4.0, 10.0])
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("shape", SHAPES, ids=SID)
def test_unequal_scales(shape, dtype, spread, out_dtype):
    """Blocks whose scales differ by powers of two up to hundreds of thousands."""
    for splits in (0, 1, 4):
        run(shape, 800, [800, 555], 16, dtype, out_dtype, splits, spread=spread, scale=0.01)


@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_scales(d, dtype):
    """A warp's scales are loaded for 16 of its steps at a time: four warps of 32-row steps, 2048 rows."""
    for n in (2047, 2048, 2049, 2048 + 32, 2048 + 128, 4096, 4097):
        for block in (16, 128):
            run((4, 1, d), n, [n, n - 31], block, dtype, torch.float32, 1)
            run((12, 1, d), n, [n, n - 31], block, dtype, torch.bfloat16, 1, window=n - 100, prefix=30)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
def test_long_caches(dtype, out_dtype):
    for shape in (SHAPES[3], SHAPES[6], SHAPES[1]):
        run(shape, 40000, [40000, 31111], 64, dtype, out_dtype)
        run(shape, 40000, [40000, 123], 128, dtype, out_dtype, softcap=30.0, window=30000, prefix=4)
        run(shape, 40000, [39999, 40000], 16, dtype, out_dtype, slopes=falling(shape[0]), begin=[5, 39000])


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("dtype", KINDS, ids=KID)
@pytest.mark.parametrize("shape", SHAPES, ids=SID)
def test_largest_slopes(shape, dtype, splits):
    """One row is all that counts, the last one or the first that is seen: its value, off by its
    weight's rounding and a merge's."""
    h_q, h_kv, d = shape
    K, V = (torch.randn((2, h_kv, 700, d), device="cuda").mul(20).clamp(-100, 100) for _ in range(2))
    K, V = (t.round().to(torch.int8) if dtype == torch.int8 else t.to(dtype) for t in (K, V))
    s = torch.exp2(torch.randint(-9, -3, (2, h_kv, 22), device="cuda").float())
    q = torch.randn((2, h_q, d), device="cuda").to(torch.bfloat16)
    lens = [700, 277]
    for slope in (3.4e38, -3.4e38, float("inf"), float("-inf")):
        for terms in ({}, {"window": 40, "softcap": 9.0}):
            mod = ScoreMod(slopes=torch.full((h_q,), slope, device="cuda"), **terms)
            out = api.decode_attn_q8b(q, K, V, s, s, i32(lens), 32, mod=mod, num_splits=splits).double()
            for b, n in enumerate(lens):
                at = n - 1 if slope > 0 else max(0, n - 40) if terms else 0
                want = (V[b, :, at].double() * s[b, :, at // 32, None].double()).repeat_interleave(h_q // h_kv, 0)
                assert bool(((out[b] - want).abs() <= want.abs() * (D.weight_rounding("q8b") + 64 * D.U)).all())


def test_results_repeat():
    """The same call gives the same bits, whatever ran before it on the same workspace."""
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = (torch.randint(-127, 128, (3, 2, 9000, 128), dtype=torch.int8, device="cuda", generator=g) for _ in range(2))
    s = torch.exp2(torch.randn((3, 2, 282), device="cuda", generator=g) - 6)
    q = torch.randn((3, 32, 128), device="cuda", generator=g).to(torch.bfloat16)
    Kb, Vb = (t.to(torch.bfloat16) / 64 for t in (K, V))
    for lens in ([9000, 100, 4097], [1, 0, 8999]):
        runs = [lambda c=c, n=n, o=o: api.decode_attn_q8b(q, K, V, s, s, i32(lens), 32, mod=ScoreMod(softcap=c) if c else None,
                                                          num_splits=n, out_dtype=o)
                for c in (0.0, 20.0) for n in (0, 7) for o in OUTS]
        runs += [lambda c=c, n=n: api.decode_attn_mod(q, Kb, Vb, i32(lens), ScoreMod(softcap=c, window=5000), num_splits=n)
                 for c in (0.0, 20.0) for n in (0, 7, -1)]
        first = [run().clone() for run in runs]
        for run, want in list(zip(runs, first))[::-1]:
            assert torch.equal(run(), want)
