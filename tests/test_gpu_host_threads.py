"""Host threads that call on one stream at the same time (needs a GB300)."""
import threading

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


@pytest.mark.parametrize("kind", ["plain", "mod", "q8b", "mixed"])
def test_threads_on_the_default_stream(kind):
    """Every thread's results are those of its calls by themselves."""
    runs = []
    for k in range(4):
        h_q, h_kv, d, n = 8, 2, 128, 3000 + 500 * k
        lens = torch.tensor([n, n // 3], dtype=torch.int32, device="cuda")
        q, K, V = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in ((2, h_q, d), (2, h_kv, n, d), (2, h_kv, n, d)))
        K8, V8 = (torch.randint(-127, 128, (2, h_kv, n, d), dtype=torch.int8, device="cuda") for _ in range(2))
        s = torch.full((2, h_kv, -(-n // 64)), 2.0 ** -6, device="cuda")
        what = ["plain", "mod", "q8b"][k % 3] if kind == "mixed" else kind
        run = {"plain": lambda o, a=(q, K, V, lens), k=k: api.decode_attn(*a, out=o, num_splits=5 + k),
               "mod": lambda o, a=(q, K, V, lens), k=k: api.decode_attn_mod(*a, ScoreMod(softcap=9.0), out=o, num_splits=5 + k),
               "q8b": lambda o, a=(q, K8, V8, s, s, lens), k=k: api.decode_attn_q8b(*a, 64, out=o, num_splits=5 + k)}[what]
        runs.append((run, torch.zeros(2, h_q, d, device="cuda")))
        run(runs[-1][1])
    outs = [[torch.zeros_like(want) for _ in range(50)] for _, want in runs]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(runs)), []

    def body(run, mine):
        try:
            start.wait()
            for out in mine:
                run(out)
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=body, args=(run, mine)) for (run, _), mine in zip(runs, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, want), mine in zip(runs, outs):
        for out in mine:
            assert torch.equal(out, want)
