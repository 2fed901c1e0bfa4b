"""Attention of chunks of tokens (needs a GB300): each output element against 64 bits with a bound of its own."""
import math

import pytest
import torch

import attend_bounds as A
from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu
OUTS = [torch.bfloat16, torch.float32]
OID = ["bf16", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(B, T, h_q, h_kv, d, n_max, seed=0, peak=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q = (peak * r(B, T, h_q, d)).bfloat16().transpose(1, 2)
    return q, r(B, h_kv, n_max, d).bfloat16(), r(B, h_kv, n_max, d).bfloat16()


def run(q, K, V, lens, news, out_dtype, window=0, prefix=0, scale=None, use_new=True, poison=True, **kw):
    """One call, checked against the definition; rows that no token sees hold NaN."""
    B, h_q, T, d = q.shape
    Kp, Vp = K.clone(), V.clone()
    if poison:
        for b, (n, m) in enumerate(zip(lens, news)):
            Kp[b, :, n:] = Vp[b, :, n:] = float("nan")
            if window:
                first = max(0, n - m + 1 - window)
                if first > prefix:
                    Kp[b, :, prefix:first] = Vp[b, :, prefix:first] = float("nan")
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.full((B, T, h_q, d), 7.0, dtype=out_dtype, device="cuda").transpose(1, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.chunk_attn(q, Kp, Vp, i32(lens), n_new=i32(news) if use_new else None, window=window, prefix=prefix,
                         out=out, scale=scale, dev_error=err, **kw)
    torch.cuda.synchronize()
    assert got is out and int(err) == 0
    want, tol = A.chunk(q, K, V, lens, news, scale, out_dtype, window, prefix)
    for b, m in enumerate(news):
        assert (out[b, :, m:] == 7.0).all()           # tokens that are not there are left alone
        out[b, :, m:] = 0
    A.check(out, want, tol)
    return out


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d", [64, 128])
def test_one_tile(out_dtype, d):
    """A few rows, one unit: the smallest case there is first."""
    q, K, V = make(1, 1, 1, 1, d, 128)
    run(q, K, V, [1], [1], out_dtype)
    run(q, K, V, [2], [1], out_dtype)
    run(q, K, V, [128], [1], out_dtype)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 5, 127, 128, 129, 256, 300])
def test_tokens(out_dtype, d, T):
    """Counts of tokens around the tiles' edges, alone and behind cached rows."""
    q, K, V = make(2, T, 2, 1, d, 700, seed=T)
    run(q, K, V, [T, T + 33], [T, T], out_dtype, use_new=False)
    run(q, K, V, [T + 384, T + 129], [T, T // 2], out_dtype)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 12, 16, 128, 200, 300])
def test_groups(group):
    T = 3 if group >= 100 else 70
    q, K, V = make(2, T, 2 * group, 2, 64, 300, seed=group)
    run(q, K, V, [T + 150, T], [T, T - 1], torch.bfloat16)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
@pytest.mark.parametrize("window,prefix", [(1, 0), (1, 1), (2, 5), (64, 0), (128, 4), (129, 127), (130, 128), (200, 129),
                                           (400, 300), (5000, 3), (1 << 31 - 1, 7)])
def test_window(window, prefix, out_dtype):
    q, K, V = make(2, 150, 4, 2, 64, 900, seed=window)
    run(q, K, V, [900, 431], [150, 90], out_dtype, window=window, prefix=prefix)
    q, K, V = make(2, 290, 1, 1, 128, 700, seed=window)
    run(q, K, V, [700, 290], [290, 290], out_dtype, window=window, prefix=prefix)
    q, K, V = make(2, 1, 8, 1, 128, 1500, seed=window)
    run(q, K, V, [1500, 600], [1, 1], out_dtype, window=window, prefix=prefix)


@pytest.mark.parametrize("out_dtype", OUTS, ids=OID)
def test_cut_along_the_rows(out_dtype):
    """Few units over long caches: cut into items and merged."""
    q, K, V = make(2, 4, 16, 2, 128, 20000, seed=3)
    run(q, K, V, [20000, 13], [4, 4], out_dtype)
    run(q, K, V, [4, 9999], [4, 2], out_dtype)
    run(q, K, V, [19999, 12345], [1, 3], out_dtype, window=6000, prefix=500)
    q, K, V = make(1, 40, 8, 1, 64, 30000, seed=4)      # units of two streams
    run(q, K, V, [29990], [40], out_dtype)


def test_many_units():
    """More units than the grid is cut for: one item each."""
    q, K, V = make(5, 150, 32, 32, 64, 400, seed=5)
    run(q, K, V, [400, 150, 333, 200, 7], [150, 150, 1, 0, 7], torch.bfloat16)
    q, K, V = make(90, 2, 16, 8, 64, 300, seed=6)
    run(q, K, V, [(b * 37) % 300 + 1 for b in range(90)], [min(1 + b % 2, (b * 37) % 300 + 1) for b in range(90)],
        torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
def test_units_of_all_sizes(d):
    """Several units a CTA, of one or two streams and any number of rows, one behind the other."""
    B, T = 24, 70
    q, K, V = make(B, T, 40, 10, d, 420, seed=13)
    news = [(b * 29) % (T + 1) for b in range(B)]
    lens = [min(420, m + (b * 47) % 300) for b, m in enumerate(news)]
    run(q, K, V, lens, news, torch.bfloat16)                              # one item a unit
    run(q, K, V, lens, news, torch.bfloat16, window=150, prefix=5)
    q, K, V = make(B, T, 40, 10, d, 1500, seed=14)                        # the line: cut into equal pieces
    lens = [min(1500, m + (b * 497) % 1400) for b, m in enumerate(news)]
    run(q, K, V, lens, news, torch.float32)
    run(q, K, V, lens, news, torch.bfloat16, window=900, prefix=3)


def test_scales():
    q, K, V = make(1, 30, 2, 1, 64, 200, seed=7)
    for scale in (0.0, -0.125, 1e-30, 3.0, -2.0):
        run(q, K, V, [180], [30], torch.float32, scale=scale)
        run(q, K, V, [180], [30], torch.bfloat16, scale=scale)


def test_peaked_scores():
    """Scores that grow along the rows: the running maximum is exceeded again and again."""
    q, K, V = make(1, 20, 2, 1, 128, 2000, seed=8)
    K = (K.float() + q[:, :1, :1].float() * torch.linspace(0, 0.6, 2000, device="cuda")[:, None]).bfloat16()
    for out in OUTS:
        run(q, K, V, [2000], [20], out)
        run(q, K.flip(2), V, [2000], [20], out)


def test_strides():
    """Queries and outputs head by head, token by token, and as columns of a wider projection."""
    B, T, h_q, h_kv, d, n_max = 2, 40, 8, 2, 128, 100
    q, K, V = make(B, T, h_q, h_kv, d, n_max, seed=9)
    lens = i32([100, 77])
    base = api.chunk_attn(q, K, V, lens, out_dtype=torch.bfloat16)
    assert base.transpose(1, 2).is_contiguous()
    wide = torch.zeros((B, T, 3 * h_q, d), dtype=torch.bfloat16, device="cuda")
    wide[:, :, h_q:2 * h_q] = q.transpose(1, 2)
    for qs in (q.contiguous(), wide[:, :, h_q:2 * h_q].transpose(1, 2)):
        for out in (torch.empty((B, h_q, T, d), dtype=torch.bfloat16, device="cuda"),
                    torch.zeros((B, T, 2 * h_q, d), dtype=torch.bfloat16, device="cuda")[:, :, h_q:].transpose(1, 2)):
            api.chunk_attn(qs, K, V, lens, out=out)
            assert torch.equal(out, base)
    # one query tensor for the whole batch
    one = q[:1].expand(B, -1, -1, -1)
    assert torch.equal(api.chunk_attn(one, K, V, lens), api.chunk_attn(one.contiguous(), K, V, lens))


def test_bad_lengths():
    """Lengths outside their ranges are clamped and reported; tokens without rows get zero."""
    q, K, V = make(4, 6, 4, 2, 64, 50, seed=10)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.chunk_attn(q, K, V, i32([60, -3, 2, 50]), n_new=i32([6, 6, 6, 9]), dev_error=err)
    assert int(err) == api.DEVERR_SEQ_LEN
    want, tol = A.chunk(q, K, V, [50, 0, 2, 50], [6, 6, 6, 6], 0.125, torch.float32)
    A.check(out, want, tol)
    for bad in ((i32([50] * 4), i32([6, 6, 6, -1])), (i32([50, 50, 50, 51]), None), (i32([5, 50, 50, 50]), None)):
        err.zero_()
        api.chunk_attn(q, K, V, bad[0], n_new=bad[1], dev_error=err)
        assert int(err) == api.DEVERR_SEQ_LEN


def test_same_bits_and_decode():
    """The same call gives the same bits, and one token a sequence is a decode step."""
    q, K, V = make(3, 1, 16, 2, 128, 9000, seed=11)
    lens = i32([9000, 4321, 1])
    a = api.chunk_attn(q, K, V, lens)
    for _ in range(3):
        assert torch.equal(a, api.chunk_attn(q, K, V, lens))
    d = api.decode_attn(q.squeeze(2).contiguous(), K, V, lens)
    torch.testing.assert_close(a.squeeze(2), d, rtol=0, atol=4e-4)  # two roundings of weights of 2^-16 |V|, |V| < 6


def test_graph_streams_and_threads():
    """Captured and replayed with new contents; on a stream of its own."""
    q, K, V = make(2, 3, 8, 2, 128, 5000, seed=12)
    lens = i32([5000, 100])
    want = api.chunk_attn(q, K, V, lens).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    api.chunk_attn(q, K, V, lens, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.chunk_attn(q, K, V, lens))
        graphs.append(g)
    lens.copy_(i32([4000, 5000]))
    want = api.chunk_attn(q, K, V, lens).clone()
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("d", [64, 128])
def test_units_cut_between(d):
    """Units of one and two streams, cut wherever a piece ends, in a cache of 2500 rows."""
    B, T = 12, 70
    q, K, V = make(B, T, 20, 5, d, 2500, seed=15)
    news = [(b * 29) % (T + 1) for b in range(B)]
    lens = [min(2500, m + (b * 997) % 2450) for b, m in enumerate(news)]
    run(q, K, V, lens, news, torch.bfloat16)
    run(q, K, V, lens, news, torch.float32, window=900, prefix=3)


@pytest.mark.parametrize("d", [64, 128])
def test_units_taken_over(d):
    """Several times as many units as SMs, whole, many of them without tokens."""
    B, T = 20, 70
    q, K, V = make(B, T, 24, 12, d, 900, seed=16)
    news = [(b * 223) % (T + 1) if b % 3 else 0 for b in range(B)]
    lens = [min(900, m + (b * 497) % 750) for b, m in enumerate(news)]
    run(q, K, V, lens, news, torch.bfloat16)
    run(q, K, V, [T] * B, [T] * B, torch.float32)
    run(q, K, V, [900] + [1] * (B - 1), [T] + [1] * (B - 1), torch.bfloat16, window=300, prefix=2)
    run(q, K, V, [0] * B, [0] * B, torch.bfloat16)
    # lengths out of range are reported whoever takes the sequence's units
    for b in (0, 7, B - 1):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.chunk_attn(q, K, V, i32([901 if x == b else 700 for x in range(B)]), dev_error=err)
        assert int(err) == api.DEVERR_SEQ_LEN


def test_units_taken_over_at_once():
    """Two streams and two graphs at a time, whole units: the same bits as alone."""
    q, K, V = make(12, 500, 16, 8, 128, 1000, seed=17)
    lens = i32([500 + (b * 101) % 501 for b in range(12)])
    want = api.chunk_attn(q, K, V, lens, out_dtype=torch.bfloat16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in streams]
    graphs = []
    for s, o in zip(streams, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                api.chunk_attn(q, K, V, lens, out=o)
        graphs.append(g)
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, o, g in zip(streams, outs, graphs):
            api.chunk_attn(q, K, V, lens, out=o, stream=s)
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
