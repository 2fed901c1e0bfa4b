"""Elements of a head that are not rotated pass through as they are, whatever they hold (needs a GB300)."""
import pytest
import torch

from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d,d_v,rot", [(64, 64, 16), (64, 64, 48), (128, 128, 64), (192, 128, 160), (256, 256, 32)])
@pytest.mark.parametrize("T", [1, 600])
def test_passed_through(T, d, d_v, rot, interleaved, dtype):
    """Infinities, NaN and negative zeros past rot stay where they are, bit for bit but for a NaN's payload."""
    g = torch.Generator(device="cuda").manual_seed(rot)
    B, h_q, h_kv, n_max = 2, 6, 2, T + 3
    x = torch.randn((B, h_q + h_kv, T, d), generator=g, device="cuda").to(dtype)
    kinds = torch.tensor([INF, -INF, NAN, -0.0, 0.0, 1.5], device="cuda", dtype=dtype)
    pick = torch.randint(0, 6, (B, h_q + h_kv, T, d - rot), generator=g, device="cuda")
    x[..., rot:] = kinds[pick]
    v = torch.randn((B, h_kv, T, d_v), generator=g, device="cuda").to(dtype)
    K, V = (torch.zeros((B, h_kv, n_max, w), dtype=dtype, device="cuda") for w in (d, d_v))
    angle = torch.randn((n_max, rot // 2), generator=g, device="cuda")
    pos = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    q_out = api.kv_append_rope(x[:, :h_q], x[:, h_q:], v, K, V, pos, angle.cos(), angle.sin(), interleaved=interleaved)
    got = torch.cat([q_out, torch.stack([K[b, :, p:p + T] for b, p in enumerate((0, 3))])], dim=1)
    want, have = x[..., rot:], got[..., rot:]
    assert torch.equal(have.isnan(), want.isnan())
    same = torch.where(want.isnan(), 0, want)
    have = torch.where(want.isnan(), 0, have)
    assert torch.equal(have, same) and torch.equal(have.signbit(), same.signbit())
    # the rotated ones: two products and a sum in float, rounded once
    at = torch.stack([angle[p:p + T] for p in (0, 3)])[:, None].double()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, z = x.double(), got.double()
    c, s = at.float().cos().double(), at.float().sin().double()
    for have, want, size in ((z[..., a], y[..., a] * c - y[..., b] * s, (y[..., a] * c).abs() + (y[..., b] * s).abs()),
                             (z[..., b], y[..., b] * c + y[..., a] * s, (y[..., b] * c).abs() + (y[..., a] * s).abs())):
        tol = 2 * 2.0 ** -24 * size
        assert ((have - want).abs() <= tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + 1e-44).all()
