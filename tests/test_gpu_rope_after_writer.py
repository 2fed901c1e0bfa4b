"""kv_append_rope right behind a call that writes what it reads (needs a GB300): its grid may start under that call's."""
import pytest
import torch

from decode_attention_kv_split_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def test_tables_weights_and_tokens_of_the_call_before():
    """Angles, weights and tokens come out of decode steps whose outputs change from round to round."""
    B, h, d, n, rounds = 64, 8, 128, 512, 20
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    K, V = r(B, h, n, d), r(B, h, n, d)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    qs = [r(B, h, d) for _ in range(rounds)]
    pos = torch.arange(B, dtype=torch.int32, device="cuda")
    caches = [torch.zeros(B, h, B + 2, d, device="cuda") for _ in range(2)]
    made = torch.zeros(B, h, d, device="cuda")

    def tables():
        flat = made.view(-1)
        return flat[:256 * 64].view(256, 64), flat[256 * 64:512 * 64].view(256, 64), flat[-d:], made.view(B, h, 1, d)

    def step(q, wait):
        api.decode_attn(q, K, V, lens, out=made)
        if wait:
            torch.cuda.synchronize()
        cos, sin, w, tokens = tables()
        return api.kv_append_rope(tokens, tokens, tokens, *caches, pos, cos, sin, q_weight=w, k_weight=w)
    got, want = ([step(q, wait).clone() for q in qs] for wait in (False, True))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
