"""Score terms in the kernels that walk a work list, as long caches run them (needs a GB300).

Calls of a few thousand rows and no split count go to clusters of CTAs; an explicit count goes to
the work list, and for more than 8 heads of 128 to the tcgen05 kernel.  Every output element is
held to a bound of its own (decode_bounds), for float32 and for bf16 outputs.  Rows that are not
seen hold NaN and infinities, outputs start as NaN."""
import math

import pytest
import torch

import decode_bounds as D
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod

pytestmark = pytest.mark.gpu
OUTS = [torch.float32, torch.bfloat16]
OID = ["fp32", "bf16"]

SHAPES = {  # every kernel and head layout: h_q, h_kv, d_k, d_v, type of the cache
    "fp32-64-g1": (2, 2, 64, 64, torch.float32),
    "fp32-128-g2": (4, 2, 128, 128, torch.float32),
    "fp32-128-g4": (12, 3, 128, 128, torch.float32),
    "fp32-128-g17": (17, 1, 128, 128, torch.float32),
    "bf16-64-g1": (8, 8, 64, 64, torch.bfloat16),
    "bf16-64-g16": (32, 2, 64, 64, torch.bfloat16),
    "bf16-64-g40": (40, 1, 64, 64, torch.bfloat16),
    "bf16-128-g4": (8, 2, 128, 128, torch.bfloat16),
    "tc5-g12": (12, 1, 128, 128, torch.bfloat16),
    "tc5-g16": (32, 2, 128, 128, torch.bfloat16),
    "tc5-g32": (32, 1, 128, 128, torch.bfloat16),
    "tc5-g48": (96, 2, 128, 128, torch.bfloat16),
    "bf16-256": (8, 2, 256, 256, torch.bfloat16),
    "bf16-192": (20, 2, 192, 128, torch.bfloat16),
}
FEW = ["fp32-64-g1", "fp32-128-g17", "bf16-64-g40", "bf16-128-g4", "tc5-g16", "tc5-g32", "bf16-192"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(shape, n_max, lens, splits, out_dtype, softcap=0.0, slopes=None, window=0, prefix=0, begin=None, append=False,
        seed=0, scale=None, bad_new=False):
    h_q, h_kv, d_k, d_v, dtype = SHAPES[shape]
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, K, V, kn, vn = (torch.randn(s, generator=g, device="cuda") for s in (
        (B, h_q, d_k), (B, h_kv, n_max, d_k), (B, h_kv, n_max, d_v), (B, h_kv, d_k), (B, h_kv, d_v)))
    q, K, V, kn, vn = (2 * q).to(dtype), K.to(dtype), V.to(dtype), kn.to(dtype), vn.to(dtype)
    rows = torch.arange(n_max, device="cuda")
    after = [n + 1 if append and n < n_max else n for n in lens]
    for b, n in enumerate(after):
        first = 0 if begin is None else begin[b]
        first = max(first, n - window) if window else first
        hidden = rows[~((rows < n) & ((rows < prefix) | (rows >= first)))]
        K[b, :, hidden] = V[b, :, hidden] = float("nan")
        V[b, :, hidden[::2]] = float("inf")
        if bad_new:  # (the appended row is one of them)
            assert n - 1 in hidden.tolist()
            kn[b] = vn[b] = float("nan")
    mod = ScoreMod(softcap=softcap, window=window, prefix=prefix, doc_begin=None if begin is None else i32(begin),
                   slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    scale = 1 / math.sqrt(d_k) if scale is None else scale
    out = torch.full((B, h_q, d_v), float("nan"), dtype=out_dtype, device="cuda")
    before = api.launch_count()
    if append:
        Kd, Vd, grown = K.clone(), V.clone(), torch.full((B,), -7, dtype=torch.int32, device="cuda")
        api.decode_attn_mod_append(q, kn, vn, Kd, Vd, i32(lens), mod, out=out, seq_lens_out=grown, scale=scale,
                                   num_splits=splits)
        assert grown.tolist() == after
        for b, n in enumerate(lens):
            if n < n_max:
                K[b, :, n], V[b, :, n] = kn[b], vn[b]
        assert torch.equal(Kd.view(torch.uint8), K.view(torch.uint8))
        assert torch.equal(Vd.view(torch.uint8), V.view(torch.uint8))
    else:
        api.decode_attn_mod(q, K, V, i32(lens), mod, out=out, scale=scale, num_splits=splits)
    assert splits == 1 or api.launch_count() == before + 2  # a combine: not the cluster form
    part = D.weight_rounding("fp32" if dtype == torch.float32 else "bf16", out_dtype)
    want, tol = D.attend(q, K, V, after, scale, part, out_dtype, softcap, slopes, window, prefix, begin)
    D.check(out, want, tol, f"{shape} {lens} cap {softcap} window {window} prefix {prefix} begin {begin}")


def falling(h_q, sign=1):
    return [sign * 2.0 ** (-8 * (h + 1) / h_q) for h in range(h_q)]


def all_terms(h_q):
    return [
        {},
        {"softcap": 20.0},
        {"slopes": falling(h_q)},
        {"slopes": [(-1) ** h * s for h, s in enumerate(falling(h_q))], "window": 90},
        {"window": 400, "prefix": 3},
        {"begin": [37, 300], "prefix": 5},
        {"softcap": 3.0, "slopes": falling(h_q), "window": 450, "prefix": 170, "begin": [0, 230]},
        {"softcap": 50.0, "window": 500},
        {"softcap": 30.0, "slopes": falling(h_q, -1), "prefix": 140, "begin": [500, 600]},
    ]


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("which", range(9))
@pytest.mark.parametrize("shape", SHAPES)
def test_terms(shape, which, out_dtype):
    terms = all_terms(SHAPES[shape][0])[which]
    for splits in (1, 3):
        run(shape, 900, [900, 641], splits, out_dtype, seed=which, **terms)
    run(shape, 700, [0, 700], 2, out_dtype, seed=which, **terms)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("which", range(9))
@pytest.mark.parametrize("shape", SHAPES)
def test_terms_append(shape, which, out_dtype):
    terms = all_terms(SHAPES[shape][0])[which]
    run(shape, 900, [899, 640], 3, out_dtype, seed=which, append=True, **terms)
    run(shape, 900, [900, 0], 2, out_dtype, seed=which, append=True, **terms)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("shape", FEW)
def test_caps(shape, out_dtype):
    """Caps on both sides of the border between the two forms of tanh, below and above the scores."""
    for cap in (0.05, 1.0, 20.0, 50.0, 100.0, 128.0, 129.0, 1e4, 1e30):
        for scale in (None, 2.0):  # (2: scores of several times the cap)
            run(shape, 700, [700, 333], 2, out_dtype, softcap=cap, scale=scale)


@pytest.mark.parametrize("window,prefix", [(1, 0), (1, 1), (127, 0), (128, 128), (129, 127), (64, 129), (383, 1), (384, 0),
                                           (385, 64), (2 ** 31 - 1, 2 ** 31 - 1), (0, 50), (5, 1000)])
@pytest.mark.parametrize("shape", ["fp32-64-g1", "bf16-128-g4", "tc5-g16", "tc5-g32"])
def test_stage_borders(shape, window, prefix):
    """Prefix ends and window starts on, before and behind the borders of stages and splits."""
    h_q = SHAPES[shape][0]
    for n in (1, 128, 384, 511):
        for splits in (1, 3):
            run(shape, 512, [n, n], splits, torch.float32, window=window, prefix=prefix, seed=n, softcap=9.0)
        run(shape, 512, [n, n], 1, torch.bfloat16, window=window, prefix=prefix, seed=n, slopes=falling(h_q))


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("shape", FEW)
def test_rows_that_nothing_sees(shape, append):
    """Documents that begin at, past or far past the length: only a prefix is left, or nothing; an
    appended row that is not seen may hold anything."""
    for prefix in (0, 3, 200):
        for begin in (299, 300, 301, 302, 5000, 2 ** 31 - 1, -5, -2 ** 31):
            unseen = append and begin > 300
            for splits in (1, 2):
                run(shape, 400, [300, 300], splits, torch.float32, begin=[begin, begin], prefix=prefix, append=append,
                    bad_new=unseen, softcap=20.0 if splits == 1 else 0.0)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("shape", FEW)
def test_largest_slopes(shape, splits):
    """One row is all that counts, the last one or the first that is seen: its value, off by its
    weight's rounding, a merge's and the output's."""
    h_q, h_kv, d_k, d_v, dtype = SHAPES[shape]
    q, K, V = (torch.randn(s, device="cuda").to(dtype) for s in ((2, h_q, d_k), (2, h_kv, 700, d_k), (2, h_kv, 700, d_v)))
    lens = [700, 277]
    for slope in (3.4e38, -3.4e38, float("inf"), float("-inf")):
        for terms in ({}, {"window": 40, "softcap": 9.0}):
            mod = ScoreMod(slopes=torch.full((h_q,), slope, device="cuda"), **terms)
            out = api.decode_attn_mod(q, K, V, i32(lens), mod, num_splits=splits).double()
            for b, n in enumerate(lens):
                at = n - 1 if slope > 0 else max(0, n - 40) if terms else 0
                want = V[b, :, at].double().repeat_interleave(h_q // h_kv, 0)
                part = D.weight_rounding("fp32" if dtype == torch.float32 else "bf16")
                assert bool(((out[b] - want).abs() <= want.abs() * (part + 64 * D.U)).all())


def test_long_caches():
    """The library's own split counts: chunks and balanced pieces over tens of thousands of rows."""
    for shape in ("fp32-128-g4", "fp32-128-g17", "bf16-64-g40", "bf16-128-g4", "tc5-g32", "bf16-256", "bf16-192"):
        h_q = SHAPES[shape][0]
        for out_dtype in OUTS:
            run(shape, 40000, [40000, 31111], 0, out_dtype, softcap=30.0, slopes=falling(h_q), prefix=1000)
            run(shape, 40000, [39999, 123], 0, out_dtype, softcap=50.0, window=30000, prefix=4, append=True)
            run(shape, 40000, [40000, 40000], -1, out_dtype, begin=[100, 39990], prefix=130)
