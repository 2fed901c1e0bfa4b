"""Counts beyond 32 bits are refused, not cut to 32 (no GPU: the library and the streams are stand-ins)."""
import contextlib

import pytest
import torch

from decode_attention_kv_split_gb300 import api

WIDE = [torch.zeros(shape, device="meta") for shape in (((1 << 32) + 5, 32), (1 << 31, 8), (9, (1 << 31) + 32))]


@pytest.fixture
def called(monkeypatch):
    seen = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_bytes"):
                    return 4096
                seen.append(args)
                return 0
            return call
    lib = Library()
    monkeypatch.setattr(api, "_lib", lib)
    monkeypatch.setattr(api, "load", lambda: lib)
    monkeypatch.setattr(api, "_ws_cache", {})
    monkeypatch.setattr(api, "_mod_bytes_cache", {})
    monkeypatch.setattr(api, "_enter", lambda device: -1)
    monkeypatch.setattr(api, "_raw", lambda stream, device: 0)
    monkeypatch.setattr(api, "_on_stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, dtype=kw["dtype"]))
    return seen


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_prefix_len(called):
    q, Kp, K, lens = bf16(2, 4, 64), bf16(2, 9, 64), bf16(2, 2, 9, 64), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(8192, dtype=torch.uint8)
    for bad in ((1 << 32) + 5, 1 << 32, -(1 << 32) + 5, 1 << 31):
        with pytest.raises(ValueError):
            api.decode_attn_shared(q, Kp, Kp, K, K, lens, prefix_len=bad, workspace=ws)
    assert not called
    for n in (0, 5, 9):
        api.decode_attn_shared(q, Kp, Kp, K, K, lens, prefix_len=n, workspace=ws)
    assert [c[3] for c in called] == [0, 5, 9]


def test_tables(called):
    K, x, pos = bf16(2, 2, 9, 64), bf16(2, 2, 1, 64), torch.zeros(2, dtype=torch.int32)
    V = bf16(2, 2, 9, 64)
    for t in WIDE:
        with pytest.raises(ValueError):
            api.kv_append_rope(x, x, x, K, V, pos, t, t)
    assert not called
    t = torch.zeros(9, 32)
    api.kv_append_rope(x, x, x, K, V, pos, t, t)
    assert len(called) == 1
