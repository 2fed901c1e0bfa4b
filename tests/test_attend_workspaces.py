"""Which workspace a chunk or shared-prefix call gets (no GPU: the library and the streams are stand-ins)."""
import contextlib

import pytest
import torch

from decode_attention_kv_split_gb300 import api


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def calls(monkeypatch):
    seen, capturing = [], []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_bytes"):
                    return 4096
                seen.append((args[-4], args[-1]))   # workspace, stream
                return 0
            return call
    lib = Library()
    monkeypatch.setattr(api, "_lib", lib)
    monkeypatch.setattr(api, "load", lambda: lib)
    monkeypatch.setattr(api, "_ws_cache", {})
    monkeypatch.setattr(api, "_mod_bytes_cache", {})
    monkeypatch.setattr(api, "_enter", lambda device: -1)
    monkeypatch.setattr(api, "_on_stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: bool(capturing), raising=False)
    empty = torch.empty
    held = []   # (tensors of captured calls belong to their graphs, which keep them)

    def on_cpu(*a, **kw):
        held.append(empty(*a, dtype=kw["dtype"]))
        return held[-1]
    monkeypatch.setattr(torch, "empty", on_cpu)
    return seen, capturing


def run(kind, stream, workspace=None):
    q, K, lens = torch.zeros(2, 4, 1, 64).bfloat16(), torch.zeros(2, 2, 9, 64).bfloat16(), torch.zeros(2, dtype=torch.int32)
    if kind == "chunk":
        return api.chunk_attn(q, K, K, lens, stream=stream, workspace=workspace)
    return api.decode_attn_shared(q[:, :, 0].contiguous(), K[0], K[0], K, K, lens, stream=stream, workspace=workspace)


@pytest.mark.parametrize("kind", ["chunk", "shared"])
def test_by_stream_and_graph(calls, kind):
    seen, capturing = calls
    a, b = Stream(7), Stream(8)
    for s in (a, b, a):
        run(kind, s)
    assert [x[1] for x in seen] == [7, 8, 7]
    assert seen[0][0] == seen[2][0] != seen[1][0]      # one for each stream, kept
    capturing.append(1)
    run(kind, a)
    run(kind, a)
    assert len({x[0] for x in seen}) == 4              # captured calls share none
    given = torch.zeros(8192, dtype=torch.uint8)
    run(kind, a, given)
    assert seen[-1][0] == given.data_ptr()


def test_two_threads_take_turns(calls):
    assert api._kept_workspace((0, 7, "attend"), 100, None)[2] is api._kept_workspace((0, 7, "attend"), 100, None)[2]
