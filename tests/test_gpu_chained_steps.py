"""Calls whose inputs the kernel just before them writes, which lets its dependents start early
(needs a GB300)."""
import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def int8(*shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda")


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("kind", ["q8b", "bf16", "tc5"])
def test_q_and_slopes_of_the_kernel_before(kind, splits):
    """q and the slopes are read back from 8-bit caches by the two kernels before the decode, in one
    captured graph; their codes change from replay to replay."""
    h_q, d, n = 64, 128, 700
    h_kv = {"q8b": 8, "bf16": 8, "tc5": 2}[kind]
    src, lens_src = int8(1, 1, h_q, d), i32([h_q])           # q's values
    steep, one = int8(1, 1, 1, h_q), i32([1])                # the slopes'
    s_q, s_steep = torch.full((1, 1, 4), 2.0 ** -5, device="cuda"), torch.full((1, 1, 1), 2.0 ** -10, device="cuda")
    q, slopes = torch.zeros(1, 1, h_q, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, 1, h_q, device="cuda")
    spare = torch.zeros_like(q), torch.zeros_like(slopes)
    lens = i32([n])
    if kind == "q8b":
        K, V = int8(1, h_kv, n, d), int8(1, h_kv, n, d)
        s = torch.full((1, h_kv, 22), 2.0 ** -6, device="cuda")
    else:
        K, V = (torch.randn(1, h_kv, n, d, device="cuda").to(torch.bfloat16) for _ in range(2))

    def read():
        api.kv_read_q8b(steep, steep, s_steep, s_steep, one, 16, k_out=slopes, v_out=spare[1])
        api.kv_read_q8b(src, src, s_q, s_q, lens_src, 16, k_out=q, v_out=spare[0])

    def decode(q, slopes):
        mod = ScoreMod(slopes=slopes.view(-1), window=650)
        if kind == "q8b":
            return api.decode_attn_q8b(q.view(1, h_q, d), K, V, s, s, lens, 32, mod=mod, num_splits=splits)
        return api.decode_attn_mod(q.view(1, h_q, d), K, V, lens, mod, num_splits=splits)

    read()
    decode(q, slopes)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = []
        for _ in range(3):
            read()
            outs.append(decode(q, slopes))
    for _ in range(10):
        src.copy_(int8(*src.shape))
        steep.copy_(int8(*steep.shape))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.float().view(h_q, d), src.view(h_q, d).float() * 2.0 ** -5)
        want = decode(q.clone(), slopes.clone())
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out, want)
