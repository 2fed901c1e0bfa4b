"""Decode with score terms against a plain 64-bit implementation (needs a GB300).

Rows a query does not see, in the window's gap, before its document and past
the length, hold NaN and infinities; outputs start as NaN.  Tolerances are
terms_reference.tolerance: bf16 weights are two bf16 parts (2^-17 of a weight),
fp32 weights one float (2^-24)."""
import math
import os
import subprocess
import sys

import pytest
import torch

import terms_reference as R
from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod

pytestmark = pytest.mark.gpu
BITS = {torch.float32: 23, torch.bfloat16: 17}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def make(B, h_q, h_kv, d_k, d_v, n_max, lens, dtype, seed, terms, append=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q = (2 * r(B, h_q, d_k)).to(dtype)
    K, V = r(B, h_kv, n_max, d_k).to(dtype), r(B, h_kv, n_max, d_v).to(dtype)
    kn, vn = r(B, h_kv, d_k).to(dtype), r(B, h_kv, d_v).to(dtype)
    begin = terms.get("begin")
    for b, n in enumerate(lens):
        after = n + 1 if append and n < n_max else n
        seen = set(R.seen_rows(after, terms.get("window", 0), terms.get("prefix", 0),
                               0 if begin is None else begin[b]))
        hidden = [l for l in range(n_max) if l not in seen]
        K[b, :, hidden] = float("nan")
        V[b, :, hidden] = float("nan")
        V[b, :, hidden[::2]] = float("inf")
    return q, K, V, kn, vn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def c_terms(terms):
    sl, bg = terms.get("slopes"), terms.get("begin")
    return ScoreMod(softcap=terms.get("softcap", 0.0),
                    slopes=None if sl is None else torch.tensor(sl, dtype=torch.float32, device="cuda"),
                    window=terms.get("window", 0), prefix=terms.get("prefix", 0),
                    doc_begin=None if bg is None else torch.tensor(bg, dtype=torch.int32, device="cuda"))


def check(got, q, K, V, lens, terms, dtype, scale, out_dtype=torch.float32):
    sl = terms.get("slopes")
    # the library takes float slopes: the reference the same values
    sl = None if sl is None else torch.tensor(sl, dtype=torch.float32).tolist()
    want, size = R.attend(q, K, V, lens, scale, terms.get("softcap", 0.0), sl,
                          terms.get("window", 0), terms.get("prefix", 0), terms.get("begin"))
    seen = V[torch.isfinite(V)]
    vmax = float(seen.abs().max()) if seen.numel() else 1.0
    eps = torch.finfo(out_dtype).eps if out_dtype == torch.bfloat16 else 0.0
    tol = R.tolerance(q.shape[2], size, terms.get("softcap", 0.0), vmax, max(max(lens), 1),
                      BITS[dtype], eps)
    got = got.cpu().double()
    assert torch.isfinite(got).all(), "an unseen row reached the output, or an output was not written"
    err = float((got - want).abs().max())
    assert err <= tol, f"max abs error {err:.3e} > {tol:.3e}"


def run(B, h_q, h_kv, d_k, d_v, n_max, lens, dtype, terms, seed=0, splits=0, append=False,
        out_dtype=torch.float32, scale=None):
    q, K, V, kn, vn = make(B, h_q, h_kv, d_k, d_v, n_max, lens, dtype, seed, terms, append)
    scale = 1 / math.sqrt(d_k) if scale is None else scale
    Kd, Vd, ld = K.cuda(), V.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((B, h_q, d_v), float("nan"), dtype=out_dtype, device="cuda")
    mod = c_terms(terms)
    if append:
        grown = torch.full_like(ld, -7)
        api.decode_attn_mod_append(q.cuda(), kn.cuda(), vn.cuda(), Kd, Vd, ld, mod, out=out,
                                   seq_lens_out=grown, scale=scale, num_splits=splits)
        after = [n + 1 if n < n_max else n for n in lens]
        assert grown.tolist() == after
        for b, n in enumerate(lens):
            if n < n_max:
                K[b, :, n], V[b, :, n] = kn[b], vn[b]
        torch.testing.assert_close(Kd.cpu(), K, rtol=0, atol=0, equal_nan=True)
        torch.testing.assert_close(Vd.cpu(), V, rtol=0, atol=0, equal_nan=True)
        lens = after
    else:
        api.decode_attn_mod(q.cuda(), Kd, Vd, ld, mod, out=out, scale=scale, num_splits=splits)
    check(out, q, K, V, lens, terms, dtype, scale, out_dtype)


SHAPES = [
    # B, h_q, h_kv, d_k, d_v, n_max, lens, dtype: every kernel family and head layout
    (3, 2, 2, 64, 64, 500, [500, 0, 129], torch.float32),
    (2, 4, 2, 128, 128, 300, [300, 1], torch.float32),
    (2, 12, 3, 128, 128, 333, [333, 200], torch.float32),
    (2, 16, 2, 64, 64, 400, [399, 65], torch.float32),
    (1, 17, 1, 128, 128, 257, [257], torch.float32),
    (3, 8, 8, 64, 64, 513, [513, 0, 127], torch.bfloat16),
    (2, 32, 2, 64, 64, 300, [300, 128], torch.bfloat16),
    (1, 40, 1, 64, 64, 300, [299], torch.bfloat16),
    (3, 8, 2, 128, 128, 700, [700, 1, 385], torch.bfloat16),
    (2, 16, 2, 128, 128, 640, [640, 130], torch.bfloat16),
    (2, 12, 1, 128, 128, 600, [599, 256], torch.bfloat16),
    (2, 32, 1, 128, 128, 900, [900, 257], torch.bfloat16),
    (1, 96, 2, 128, 128, 400, [400], torch.bfloat16),
    (2, 8, 2, 256, 256, 200, [200, 64], torch.bfloat16),
    (2, 20, 2, 192, 128, 260, [260, 63], torch.bfloat16),
]
IDS = [f"{str(s[7])[6:]}-d{s[3]}v{s[4]}-h{s[1]}kv{s[2]}" for s in SHAPES]


def slopes_of(h_q, sign=1):
    return [sign * 2.0 ** (-8 * (h + 1) / h_q) for h in range(h_q)]


def all_terms(h_q, B):
    return [
        {},
        {"softcap": 20.0},
        {"slopes": slopes_of(h_q)},
        {"slopes": [(-1) ** h * s for h, s in enumerate(slopes_of(h_q))], "window": 90},
        {"window": 100, "prefix": 3},
        {"begin": [37 * (b + 1) for b in range(B)], "prefix": 5},
        {"softcap": 3.0, "slopes": slopes_of(h_q), "window": 150, "prefix": 70,
         "begin": [130 * b for b in range(B)]},
    ]


@pytest.mark.parametrize("which", range(7))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_terms(shape, which):
    B, h_q = shape[:2]
    run(*shape, all_terms(h_q, B)[which], seed=which)


@pytest.mark.parametrize("which", [1, 3, 4, 6])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] <= 128],
                         ids=[i for i, s in zip(IDS, SHAPES) if s[3] <= 128])
def test_terms_append(shape, which):
    B, h_q = shape[:2]
    run(*shape, all_terms(h_q, B)[which], seed=which, append=True)


EDGE = [(2, 8, 2, 128, 128), (1, 32, 1, 128, 128), (2, 2, 2, 64, 64)]


@pytest.mark.parametrize("splits", [0, 1, 2, 5, 300, -1])
@pytest.mark.parametrize("heads", EDGE, ids=["g4", "g32", "mha"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_split_choices(heads, dtype, splits):
    if dtype == torch.float32 and heads[1] == 32:
        heads = (1, 8, 1, 128, 128)
    B, h_q = heads[:2]
    run(*heads, 2100, [2099, 700][:B], dtype, all_terms(h_q, B)[6], seed=splits, splits=splits)


@pytest.mark.parametrize("window,prefix", [(1, 0), (1, 1), (127, 0), (128, 128), (129, 127), (64, 129),
                                           (383, 1), (384, 0), (385, 64), (10 ** 9, 0),
                                           (2 ** 31 - 1, 2 ** 31 - 1), (0, 50), (5, 1000)])
@pytest.mark.parametrize("heads", EDGE, ids=["g4", "g32", "mha"])
def test_tile_borders(heads, window, prefix):
    """Prefix ends and window starts on, before and behind stage borders."""
    B = heads[0]
    dtype = torch.float32 if heads[3] == 64 else torch.bfloat16
    for n in (1, 128, 384, 511):
        run(*heads, 512, [n] * B, dtype, {"window": window, "prefix": prefix}, seed=n)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("heads", EDGE, ids=["g4", "g32", "mha"])
def test_rows_that_nothing_sees(heads, append):
    """Documents that begin at, past or far past the length: only a prefix is left, or nothing."""
    B = heads[0]
    dtype = torch.float32 if heads[3] == 64 else torch.bfloat16
    for prefix in (0, 3, 200):
        for begin in (299, 300, 301, 302, 5000, 2 ** 31 - 1, -5, -2 ** 31):
            run(*heads, 400, [300] * B, dtype, {"begin": [begin] * B, "prefix": prefix}, append=append)


def test_appended_rows_that_nothing_sees_may_hold_anything():
    """A new row before its own document (a slot written ahead): NaN in it stays out of the output."""
    for heads in EDGE:
        B, h_q, h_kv, d, _ = heads
        dtype = torch.float32 if d == 64 else torch.bfloat16
        for prefix in (0, 100):
            q, K, V, *_ = make(*heads, 400, [300] * B, dtype, 3, {"begin": [10 ** 6] * B, "prefix": prefix}, True)
            bad = torch.full((B, h_kv, d), float("nan"), dtype=dtype, device="cuda")
            out = api.decode_attn_mod_append(q.cuda(), bad, bad, K.cuda(), V.cuda(), i32([300] * B),
                                             ScoreMod(prefix=prefix, doc_begin=i32([10 ** 6] * B)))
            check(out, q, K, V, [301] * B, {"begin": [10 ** 6] * B, "prefix": prefix}, dtype, 1 / math.sqrt(d))


def test_empty_sequences():
    for heads in EDGE:
        dtype = torch.float32 if heads[3] == 64 else torch.bfloat16
        run(*heads, 64, [0] * heads[0], dtype, {"softcap": 5.0, "window": 3, "prefix": 2})
        run(*heads, 64, [0] * heads[0], dtype, {"softcap": 5.0, "window": 3}, append=True)


@pytest.mark.parametrize("cap", [1e-3, 0.5, 30.0, 1e4, 1e30])
@pytest.mark.parametrize("heads", EDGE, ids=["g4", "g32", "mha"])
def test_caps(heads, cap):
    B = heads[0]
    dtype = torch.float32 if heads[3] == 64 else torch.bfloat16
    # (far above the scores a cap changes nothing: the bound's cap term is that of the scores)
    q, K, V, *_ = make(*heads, 300, [300] * B, dtype, 1, {})
    out = api.decode_attn_mod(q.cuda(), K.cuda(), V.cuda(),
                              torch.full((B,), 300, dtype=torch.int32, device="cuda"),
                              ScoreMod(softcap=cap))
    scale = 1 / math.sqrt(heads[3])
    want, size = R.attend(q, K, V, [300] * B, scale, cap)
    tol = R.tolerance(heads[3], size, min(cap, size), float(V.abs().max()), 300, BITS[dtype])
    assert float((out.cpu().double() - want).abs().max()) <= tol


def test_bias_where_far_rows_win():
    """Negative slopes make the first seen row the heaviest; positive ones the last."""
    for slope in (-1.0, -0.01, 1.0, 100.0, -100.0):
        for heads in EDGE:
            dtype = torch.float32 if heads[3] == 64 else torch.bfloat16
            run(*heads, 4000, [3999] * heads[0], dtype,
                {"slopes": [slope * (1 + h % 3) for h in range(heads[1])], "prefix": 2,
                 "window": 3000}, splits=3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("heads", EDGE, ids=["g4", "g32", "mha"])
@pytest.mark.parametrize("slope", [3.4e38, -3.4e38])
def test_largest_slopes(heads, dtype, slope):
    """One row is all that counts: the last one, or the first that is seen."""
    lens, h_q = [300, 77][:heads[0]], heads[1]
    run(*heads, 300, lens, dtype, {"slopes": [slope] * h_q})
    run(*heads, 300, lens, dtype, {"slopes": [slope] * h_q, "window": 40, "softcap": 9.0})


CLUSTERS = [  # heads, d_k, d_v, type, the most rows one CTA of a unit's cluster takes
    (2, 2, 64, 64, torch.float32, 384), (6, 1, 128, 128, torch.float32, 96), (8, 2, 128, 128, torch.bfloat16, 512),
    (40, 1, 64, 64, torch.bfloat16, 192), (4, 1, 256, 256, torch.bfloat16, 256), (6, 2, 192, 128, torch.bfloat16, 256),
    (20, 1, 128, 128, torch.bfloat16, 1024),
]


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("heads", CLUSTERS, ids=[f"{str(c[4])[6:]}-d{c[2]}h{c[0]}kv{c[1]}" for c in CLUSTERS])
def test_short_caches(heads, append):
    """Caches that one to eight CTAs a unit share: shares that end inside a tile, on one, empty ones."""
    h_q, h_kv, d_k, d_v, dtype, most = heads
    terms = {"softcap": 9.0, "slopes": slopes_of(h_q), "window": 0, "prefix": 2}
    for n in (1, 2, most // 3, most - 1, most + 1, 2 * most, 5 * most + 7, 8 * most, 8 * most + 1):
        run(2, h_q, h_kv, d_k, d_v, n, [n - append, n // 3], dtype, terms, seed=n, append=append)
        run(3, h_q, h_kv, d_k, d_v, n, [0, n, n // 2], dtype, {"window": max(1, n // 3), "prefix": 5}, seed=n,
            append=append)
    # a window of a long cache: its rows are what the CTAs share
    run(2, h_q, h_kv, d_k, d_v, 6000, [5999, 801], dtype, {"window": 2 * most, "prefix": 3}, append=append)
    # more sequences: fewer CTAs for each, down to one
    for B in (9, 17, 40, 70):
        run(B, h_q, h_kv, d_k, d_v, 300, [(b * 47) % 300 for b in range(B)], dtype, {"prefix": 1, "window": 250},
            seed=B, append=append)


FIRST = """
import torch
from decode_attention_kv_split_gb300 import api
q, K = torch.randn(2, 8, 128, device="cuda"), torch.randn(2, 2, 600, 128, device="cuda")
l = torch.tensor([600, 9], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = api.decode_attn_mod(q, K, K, l, api.ScoreMod(softcap=5.0))
g.replay()
again = api.decode_attn_mod(q, K, K, l, api.ScoreMod(softcap=5.0))
torch.cuda.synchronize()
assert torch.equal(out, again)
"""


def test_first_call_of_a_process_in_a_capture():
    """What the library asks the driver once, it asks then."""
    subprocess.run([sys.executable, "-c", FIRST], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_output_allocated_for_a_stream():
    q, K, V, *_ = make(2, 8, 2, 128, 128, 300, [300, 9], torch.bfloat16, 3, {}, False)
    q, K, V, l = q.cuda(), K.cuda(), V.cuda(), torch.tensor([300, 9], dtype=torch.int32, device="cuda")
    want = api.decode_attn_mod(q, K, V, l, ScoreMod(window=90))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.decode_attn_mod(q, K, V, l, ScoreMod(window=90), stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_bf16_output_and_scales():
    for shape in (SHAPES[8], SHAPES[11]):
        run(*shape, {"softcap": 10.0, "window": 300}, out_dtype=torch.bfloat16)
        run(*shape, {"softcap": 10.0, "window": 300}, scale=0.0)
        run(*shape, {"slopes": slopes_of(shape[1])}, scale=-0.05)


def test_more_items_than_the_cache_of_items():
    """More than 32 work items for a CTA: later ones are decoded on the fly, their rows too."""
    for heads, dtype in (((300, 8, 8, 64, 64), torch.bfloat16), ((300, 8, 8, 64, 64), torch.float32),
                         ((260, 80, 5, 128, 128), torch.bfloat16)):
        B, h_q = heads[:2]
        n_max = 300
        lens = [(b * 53) % 301 for b in range(B)]
        terms = {"window": 40, "prefix": 2, "begin": [(b * 31) % 200 for b in range(B)]}
        run(*heads, n_max, lens, dtype, terms, splits=4)
        run(*heads, n_max, lens, dtype, terms, splits=-1)


def test_plain_terms_equal_decode_attn():
    """No terms at all: the values of decode_attn (the work list and the order of sums are its)."""
    for shape in SHAPES:
        B, h_q, h_kv, d_k, d_v, n_max, lens, dtype = shape
        q, K, V, *_ = make(*shape, 3, {})
        args = (q.cuda(), K.cuda(), V.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        for splits in (1, 4):
            a = api.decode_attn(*args, num_splits=splits)
            b = api.decode_attn_mod(*args, ScoreMod(), num_splits=splits)
            torch.testing.assert_close(a, b, rtol=0, atol=2.0 ** -20)


def test_batch_above_one_launch():
    B = 600
    terms = {"window": 20, "begin": [b % 60 for b in range(B)], "softcap": 8.0}
    run(B, 2, 1, 64, 64, 80, [b % 81 for b in range(B)], torch.bfloat16, terms)
    run(B, 2, 1, 64, 64, 80, [b % 80 for b in range(B)], torch.bfloat16, terms, append=True)


def test_graph_replay_with_new_lengths_and_documents():
    """A captured step replayed: lengths, documents and inputs may change between replays, and two
    graphs captured on one stream do not share scratch."""
    B, h_q, h_kv, d, n_max = 2, 8, 2, 128, 2000
    q, K, V, *_ = make(B, h_q, h_kv, d, d, n_max, [n_max, n_max], torch.bfloat16, 5, {})
    qd, Kd, Vd = q.cuda(), K.cuda(), V.cuda()
    lens = torch.tensor([5, 5], dtype=torch.int32, device="cuda")
    begin = torch.zeros(2, dtype=torch.int32, device="cuda")
    outs = [torch.empty((B, h_q, d), device="cuda") for _ in range(2)]
    mods = [ScoreMod(softcap=9.0, prefix=3, doc_begin=begin), ScoreMod(window=700, doc_begin=begin)]
    graphs = []
    side = torch.cuda.Stream()
    for out, mod in zip(outs, mods):
        api.decode_attn_mod(qd, Kd, Vd, lens, mod, out=out, num_splits=7)
    torch.cuda.synchronize()
    for out, mod in zip(outs, mods):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for _ in range(2):
                api.decode_attn_mod(qd, Kd, Vd, lens, mod, out=out, num_splits=7)
        graphs.append(g)
    for n, at in ((2000, 1500), (1, 0), (1300, 1299), (0, 0)):
        lens.copy_(torch.tensor([n, n // 2], dtype=torch.int32))
        begin.copy_(torch.tensor([at, at // 3], dtype=torch.int32))
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        check(outs[0], q, K, V, [n, n // 2], {"softcap": 9.0, "prefix": 3, "begin": [at, at // 3]},
              torch.bfloat16, 1 / math.sqrt(d))
        check(outs[1], q, K, V, [n, n // 2], {"window": 700, "begin": [at, at // 3]},
              torch.bfloat16, 1 / math.sqrt(d))


def test_calls_on_two_streams():
    """Calls on two streams at once have scratch of their own."""
    shape = (2, 8, 2, 128, 128, 3000, [3000, 2777], torch.bfloat16)
    q, K, V, *_ = make(*shape, 4, {})
    args = (q.cuda(), K.cuda(), V.cuda(), torch.tensor(shape[6], dtype=torch.int32, device="cuda"))
    mods = [ScoreMod(softcap=9.0), ScoreMod(window=2500)]
    want = [api.decode_attn_mod(*args, m, num_splits=9).clone() for m in mods]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in mods]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, s, o in zip(mods, streams, outs):
            api.decode_attn_mod(*args, m, num_splits=9, out=o, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


def test_out_of_range_lengths_are_flagged():
    q, K, V, *_ = make(2, 4, 2, 64, 64, 100, [100, 0], torch.float32, 2, {"window": 30})
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([500, -3], dtype=torch.int32, device="cuda")
    out = api.decode_attn_mod(q.cuda(), K.cuda(), V.cuda(), lens, ScoreMod(window=30), dev_error=err)
    assert int(err) == api.DEVERR_SEQ_LEN
    check(out, q, K, V, [100, 0], {"window": 30}, torch.float32, 0.125)
