"""Which workspace a call gets, and who else may be using it (no GPU: the library, the tensors and
the streams are stand-ins)."""
import contextlib
import threading
import time

import pytest
import torch

from decode_attention_kv_split_gb300 import api
from decode_attention_kv_split_gb300.api import ScoreMod


class Tensor:
    at = 1 << 20

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device, self.is_cuda = torch.device("cuda", 0), True
        Tensor.at += 1 << 20
        self.ptr = Tensor.at

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1

    def data_ptr(self):
        return self.ptr

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class Library:
    """Notes the workspace and the stream of every decode call, and which workspaces were in use by
    two calls at once."""

    def __init__(self, wait=0.0):
        self.wait, self.calls, self.inside, self.shared = wait, [], [], []
        self.most = 0

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_bytes"):
                return 4096
            ws, raw = (getattr(args[i], "value", args[i]) for i in (-4, -1))
            if ws in self.inside:
                self.shared.append(ws)
            self.inside.append(ws)
            self.most = max(self.most, len(self.inside))
            time.sleep(self.wait)
            self.inside.remove(ws)
            self.calls.append((ws, raw))
            return 0
        return call


@pytest.fixture
def capturing():
    return []


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch, capturing):
    monkeypatch.setattr(api, "_ws_cache", {})
    monkeypatch.setattr(api, "_mod_bytes_cache", {})
    monkeypatch.setattr(api, "workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(api, "_enter", lambda device: -1)
    monkeypatch.setattr(api, "_on_device", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(api, "_on_stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(1))
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: bool(capturing), raising=False)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(
        shape if isinstance(shape, tuple) else (shape,), dtype))


def use(monkeypatch, lib):
    monkeypatch.setattr(api, "_lib", lib)
    monkeypatch.setattr(api, "load", lambda: lib)
    return lib


def calls():
    """name -> call(stream): every entry point that takes a workspace."""
    f, h, i, c = torch.float32, torch.bfloat16, torch.int32, torch.int8
    q, K, one, out = Tensor((2, 4, 64), f), Tensor((2, 2, 99, 64), f), Tensor((2, 2, 64), f), Tensor((2, 4, 64), f)
    lens, q8, K8, new8 = Tensor((2,), i), Tensor((2, 4, 64), h), Tensor((2, 2, 99, 64), c), Tensor((2, 2, 64), c)
    rows, row, blocks, lse = Tensor((2, 2, 99), f), Tensor((2, 2), f), Tensor((2, 2, 7), f), Tensor((2, 4), f)
    return {
        "decode_attn": lambda s: api.decode_attn(q, K, K, lens, out, stream=s),
        "decode_attn_append": lambda s: api.decode_attn_append(q, one, one, K, K, lens, out, stream=s),
        "decode_attn_partial": lambda s: api.decode_attn_partial(q, K, K, lens, o=out, lse=lse, stream=s),
        "decode_attn_q8": lambda s: api.decode_attn_q8(q8, K8, K8, rows, rows, lens, out, stream=s),
        "decode_attn_q8_append": lambda s: api.decode_attn_q8_append(q8, new8, new8, row, row, K8, K8, rows, rows, lens,
                                                                     out, stream=s),
        "decode_attn_mod": lambda s: api.decode_attn_mod(q, K, K, lens, ScoreMod(window=9), out, stream=s),
        "decode_attn_mod_append": lambda s: api.decode_attn_mod_append(q, one, one, K, K, lens, ScoreMod(window=9), out,
                                                                       stream=s),
        "decode_attn_q8b": lambda s: api.decode_attn_q8b(q8, K8, K8, blocks, blocks, lens, 16, out=out, stream=s),
    }


NAMES = ["decode_attn", "decode_attn_append", "decode_attn_partial", "decode_attn_q8", "decode_attn_q8_append",
         "decode_attn_mod", "decode_attn_mod_append", "decode_attn_q8b"]


def in_threads(*runs):
    start, errors = threading.Barrier(len(runs)), []

    def body(run):
        try:
            start.wait()
            for _ in range(3):
                run()
        except Exception as e:  # (an assertion of a thread has to reach the test)
            errors.append(e)
    threads = [threading.Thread(target=body, args=(r,)) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("name", NAMES)
def test_two_host_threads_on_one_stream(monkeypatch, name):
    """The launches of one call come one after the other: no second call is in the library on the
    same workspace meanwhile."""
    lib = use(monkeypatch, Library(0.01))
    run = calls()[name]
    in_threads(lambda: run(Stream(1)), lambda: run(Stream(1)))
    assert len(lib.calls) == 6 and not lib.shared


def test_two_entry_points_on_one_stream(monkeypatch):
    lib = use(monkeypatch, Library(0.01))
    every = calls()
    in_threads(*(lambda n=n: every[n](Stream(1)) for n in NAMES))
    assert len(lib.calls) == 3 * len(NAMES) and not lib.shared


@pytest.mark.parametrize("name", ["decode_attn_mod", "decode_attn_q8b"])
def test_two_streams_do_not_wait_for_each_other(monkeypatch, name):
    lib = use(monkeypatch, Library(0.05))
    run = calls()[name]
    in_threads(lambda: run(Stream(1)), lambda: run(Stream(2)))
    assert lib.most == 2 and not lib.shared


@pytest.mark.parametrize("name", NAMES)
def test_a_call_that_fails_leaves_the_workspace_free(monkeypatch, name):
    class Failing(Library):
        def __getattr__(self, n):
            call = Library.__getattr__(self, n)

            def fail(*args):
                call(*args)
                raise RuntimeError("no")
            return call if n.endswith("workspace_bytes") else fail
    use(monkeypatch, Failing())
    with pytest.raises(RuntimeError, match="no"):
        calls()[name](Stream(1))
    lib = use(monkeypatch, Library())
    calls()[name](Stream(1))
    assert len(lib.calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_the_workspace_goes_by_the_stream_of_the_call(monkeypatch, name):
    """Not by the current one: calls on two given streams may run at the same time."""
    lib = use(monkeypatch, Library())
    for raw in (7, 8, 7, 8):
        calls()[name](Stream(raw))
    by = {raw: {ws for ws, r in lib.calls if r == raw} for raw in (7, 8)}
    assert len(by[7]) == len(by[8]) == 1 and by[7] != by[8]


@pytest.mark.parametrize("name", NAMES)
def test_captured_calls_have_workspaces_of_their_graph(monkeypatch, capturing, name):
    lib = use(monkeypatch, Library())
    run = calls()[name]
    run(Stream(7))
    capturing.append(1)
    run(Stream(7))
    run(Stream(7))
    capturing.clear()
    run(Stream(7))
    ws = [w for w, _ in lib.calls]
    assert ws[0] == ws[3] and len(set(ws)) == 3


def test_outputs_are_allocated_in_the_stream_of_the_call(monkeypatch):
    on = []

    @contextlib.contextmanager
    def stream_of(s):
        on.append(s)
        yield
        on.pop()
    empty, where = torch.empty, []
    monkeypatch.setattr(api, "_on_stream", stream_of)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: where.append(on[-1] if on else None) or empty(*a, **k))
    use(monkeypatch, Library())
    f, h, i, c = torch.float32, torch.bfloat16, torch.int32, torch.int8
    q, K, one, lens = Tensor((2, 4, 64), f), Tensor((2, 2, 99, 64), f), Tensor((2, 2, 64), f), Tensor((2,), i)
    q8, K8, new8 = Tensor((2, 4, 64), h), Tensor((2, 2, 99, 64), c), Tensor((2, 2, 64), c)
    rows, row, parts, lses = Tensor((2, 2, 99), f), Tensor((2, 2), f), Tensor((3, 2, 4, 64), f), Tensor((3, 2, 4), f)
    for run in (lambda s: api.decode_attn(q, K, K, lens, stream=s),
                lambda s: api.decode_attn_append(q, one, one, K, K, lens, stream=s),
                lambda s: api.decode_attn_owned(q, K, K, lens, stream=s),
                lambda s: api.decode_attn_noalloc(q, K, K, lens, stream=s),
                lambda s: api.decode_attn_partial(q, K, K, lens, stream=s),
                lambda s: api.decode_attn_combine(parts, lses, stream=s),
                lambda s: api.decode_attn_q8(q8, K8, K8, rows, rows, lens, stream=s),
                lambda s: api.decode_attn_q8_append(q8, new8, new8, row, row, K8, K8, rows, rows, lens, stream=s),
                lambda s: api.decode_attn_mod(q, K, K, lens, ScoreMod(), stream=s),
                lambda s: api.kv_quantize(q, c, stream=s)):
        where.clear()
        side = Stream(9)
        run(side)
        assert where and all(s is side for s in where)
