"""Norms, rotation and the write into the cache (needs a GB300), against 64 bits with a bound on every element."""
import pytest
import torch

from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]
TID = ["bf16", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tables(n, rot):
    half = rot // 2
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return a.cos().float(), a.sin().float()


def turned(x, w, cos, sin, rot, interleaved, eps, dtype):
    """x [h, d] at one angle row -> (want, tol).  With u half a float step: the squares' sum takes at most 21
    roundings a term (16 products and sums in a lane, 5 exchanges), the mean, eps and the root 4 more, half of which
    reach the factor; two products: 15 u + 2 u of the normed value.  A rotation: two products and a sum, 2 u of their
    magnitudes.  20 u in all, and the output's half step."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    c, s = cos.double(), sin.double()
    want, size = y.clone(), y.abs()
    want[:, a], want[:, b] = y[:, a] * c - y[:, b] * s, y[:, b] * c + y[:, a] * s
    size[:, a] = y[:, a].abs() * c.abs() + y[:, b].abs() * s.abs()
    size[:, b] = y[:, b].abs() * c.abs() + y[:, a].abs() * s.abs()
    tol = 20 * U * size
    return want, tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + 1e-44


def run(B, T, h_q, h_kv, d, d_v, n_max, dtype, pos, news, rot, interleaved=False, norm=True, shift=None, seed=0,
        strided=True, in_place=False, eps=1e-6, size=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    H = h_q + h_kv
    qk = (size * r(B, T, H, d)).to(dtype)
    v = r(B, T, h_kv, d_v).to(dtype).transpose(1, 2)
    q, k = qk[:, :, :h_q].transpose(1, 2), qk[:, :, h_q:].transpose(1, 2)
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    for b, m in enumerate(news):            # tokens that are not there are not read
        q[b, :, m:] = k[b, :, m:] = v[b, :, m:] = float("nan")
    q0 = q.clone()
    K, V = r(B, h_kv, n_max, d).to(dtype), r(B, h_kv, n_max, d_v).to(dtype)
    K0, V0 = K.clone(), V.clone()
    w = [(1 + 0.3 * r(d)).to(dtype) if norm else None for _ in range(2)]
    at = pos if shift is None else [p + s for p, s in zip(pos, shift)]
    cos, sin = tables(max(a + m for a, m in zip(at, news)) + 1, rot)
    out = q if in_place else torch.full((B, T, h_q, d), 7.0, device="cuda").to(dtype).transpose(1, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.kv_append_rope(q, k, v, K, V, i32(pos), cos, sin, q_weight=w[0], k_weight=w[1], eps=eps,
                             n_new=None if all(m == T for m in news) else i32(news),
                             angle_pos=None if shift is None else i32(at), interleaved=interleaved, q_out=out,
                             dev_error=err)
    torch.cuda.synchronize()
    assert got is out and int(err) == 0
    for b, m in enumerate(news):
        for i in range(m):
            row = pos[b] + i
            for name, x, res, weight in (("q", q0[b, :, i], out[b, :, i], w[0]), ("k", k[b, :, i], K[b, :, row], w[1])):
                want, tol = turned(x, weight, cos[at[b] + i], sin[at[b] + i], rot, interleaved, eps, dtype)
                assert ((res.double() - want).abs() <= tol).all(), (name, b, i)
        assert torch.equal(V[b, :, pos[b]:pos[b] + m], v[b, :, :m])
        K0[b, :, pos[b]:pos[b] + m] = K[b, :, pos[b]:pos[b] + m]
        V0[b, :, pos[b]:pos[b] + m] = V[b, :, pos[b]:pos[b] + m]
        if not in_place:
            assert (out[b, :, m:] == 7.0).all()
    assert torch.equal(K, K0) and torch.equal(V, V0)       # every other row as it was


@pytest.mark.parametrize("dtype", TYPES, ids=TID)
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128), (256, 256)])
def test_one_token(dtype, interleaved, d, d_v):
    run(1, 1, 1, 1, d, d_v, 4, dtype, [0], [1], d, interleaved)
    run(3, 1, 6, 2, d, d_v, 40, dtype, [0, 39, 17], [1, 1, 1], d, interleaved)
    run(2, 1, 3, 1, d, d_v, 40, dtype, [7, 1], [1, 0], 16, interleaved, norm=False)


@pytest.mark.parametrize("dtype", TYPES, ids=TID)
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
def test_rotated_parts(dtype, interleaved):
    for rot in (16, 32, 48, 64, 96, 112, 128):
        run(2, 3, 4, 2, 128, 128, 20, dtype, [5, 0], [3, 2], rot, interleaved, norm=rot % 32 == 0, seed=rot)
    run(1, 2, 2, 1, 192, 128, 20, dtype, [5], [2], 160, interleaved)


@pytest.mark.parametrize("dtype", TYPES, ids=TID)
def test_chunks(dtype):
    """Many tokens (several heads a group of lanes), ragged counts, up to the last row, behind a prefix."""
    run(3, 700, 9, 3, 128, 128, 800, dtype, [0, 100, 799], [700, 641, 1], 128, seed=1)
    run(2, 900, 7, 1, 64, 64, 1000, dtype, [3, 0], [900, 0], 32, True, shift=[5000, 70000], seed=2)
    run(2, 450, 5, 5, 256, 256, 500, dtype, [50, 1], [450, 450], 64, seed=3, strided=False)
    run(2, 300, 16, 2, 128, 128, 400, dtype, [50, 1], [300, 299], 128, seed=4, in_place=True)


@pytest.mark.parametrize("dtype", TYPES, ids=TID)
def test_sizes_of_values(dtype):
    """Zero, tiny and large vectors: eps decides, nothing overflows."""
    for size in (0.0, 1e-6, 1e-3, 1e15):
        run(2, 2, 2, 1, 128, 128, 8, dtype, [0, 3], [2, 2], 128, size=size)
    run(2, 2, 2, 1, 128, 128, 8, dtype, [0, 3], [2, 2], 128, eps=0.5)


def test_tokens_without_a_row():
    """Rows and angles that do not exist: those tokens are written nowhere, the others are."""
    B, T, d = 6, 3, 64
    q, k, v = (torch.randn(B, 2, T, d, device="cuda") for _ in range(3))
    K, V = (torch.zeros(B, 2, 10, d, device="cuda") for _ in range(2))
    cos, sin = tables(20, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((B, 2, T, d), 7.0, device="cuda")
    api.kv_append_rope(q, k, v, K, V, i32([8, -1, 10, 0, 2147483647, 4]), cos, sin, q_out=out,
                       angle_pos=i32([0, 0, 0, 18, 0, -1]), dev_error=err)
    assert int(err) == api.DEVERR_POS
    there = torch.tensor([[1, 1, 0], [0] * 3, [0] * 3, [1, 1, 0], [0] * 3, [0, 1, 1]], dtype=torch.bool, device="cuda")
    assert torch.equal((out != 7.0).any(3).any(1), there)
    rows = torch.zeros(B, 10, dtype=torch.bool, device="cuda")
    rows[0, 8:] = rows[3, :2] = True
    # a negative angle row: the first token has none, the two behind it do
    rows[5, 5:7] = True
    assert torch.equal((K != 0).any(3).any(1), rows) and torch.equal((V != 0).any(3).any(1), rows)
    # tables that end before the cache does
    err.zero_()
    K.zero_()
    api.kv_append_rope(q, k, v, K, V, i32([0] * B), cos[:2].contiguous(), sin[:2].contiguous(), q_out=out, dev_error=err)
    assert int(err) == api.DEVERR_POS
    assert (K[:, :, :2] != 0).any(3).all() and (K[:, :, 2:] == 0).all()
    # counts outside their range are clamped
    for bad, kept in ((-1, 0), (4, 3)):
        err.zero_()
        K.zero_()
        api.kv_append_rope(q, k, v, K, V, i32([0] * B), cos, sin, n_new=i32([bad] + [1] * (B - 1)), dev_error=err)
        assert int(err) == api.DEVERR_POS
        assert int((K[0] != 0).any(2).all(0).sum()) == kept


def test_streams_and_graphs():
    B, d = 2, 128
    q, k, v = (torch.randn(B, 4, d, device="cuda").bfloat16() for _ in range(3))
    K, V = (torch.zeros(B, 4, 10, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cos, sin = tables(10, d)
    pos = i32([0, 3])
    out = api.kv_append_rope(q, k, v, K, V, pos, cos, sin)
    assert out.shape == q.shape
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = api.kv_append_rope(q, k, v, K, V, pos, cos, sin)
    K.zero_()
    q.mul_(0.5)
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    out = api.kv_append_rope(q, k, v, K2, V2, pos, cos, sin, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, held) and torch.equal(K, K2) and torch.equal(V, V2)
