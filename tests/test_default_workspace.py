"""Which workspace an attention call without one gets, and when another call may
use it (no GPU is used here: the library and the streams are stand-ins)."""
import contextlib
import threading
import types

import pytest
import torch

from speculative_decoding_draft_head_gb300 import binding


class _Library:
    """Takes the calls' workspaces; `inside` runs within each call."""

    def __init__(self):
        self.workspaces = []
        self.inside = lambda workspace: None

    def dspark_block_attention(self, *args):
        workspace = args[-3]
        self.workspaces.append(workspace)
        self.inside(workspace)
        return 0


@pytest.fixture
def setting(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(binding, "_lib", lib)
    monkeypatch.setattr(binding, "_default_ws", binding.WorkspaceCache())
    monkeypatch.setattr(binding, "attention_workspace_bytes", lambda B, n, *sizes: 1024 * n)
    # streams as the binding sees them: which one is current, and which ones are being captured
    seen = types.SimpleNamespace(current=[], capturing=set())

    @contextlib.contextmanager
    def on(stream):
        seen.current.append(stream)
        yield
        seen.current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                        lambda: bool(seen.current) and seen.current[-1].cuda_stream in seen.capturing)
    cache = object.__new__(binding.KVCache)
    cache._index, cache.device, cache._ref = -1, torch.device("cpu"), None
    cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim = 4, 2, 16, 64

    def call(stream, rows=3):
        q = torch.zeros((rows, 4, 64), dtype=torch.bfloat16)
        binding.block_attention(q, cache, torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32),
                                torch.tensor([0, rows]), stream=types.SimpleNamespace(device_index=-1, cuda_stream=stream))
        return lib.workspaces[-1]

    return lib, seen, call


def test_one_a_stream(setting):
    _, _, call = setting
    a, b = call(5), call(6)
    assert a != b and call(5) == a and call(6) == b and call(5, rows=2) == a


def test_a_capture_on_a_stream_that_is_not_current_gets_its_own(setting):
    """The stream that counts is the call's: a buffer that a later, larger call replaces must not be in a graph."""
    _, seen, call = setting
    kept = call(5)
    seen.capturing.add(5)
    held = dict(binding._default_ws._attention)
    captured = call(5)
    assert captured != kept and binding._default_ws._attention == held
    seen.capturing.clear()
    assert call(5) == kept


def test_calls_of_two_threads_are_enqueued_one_after_the_other(setting):
    """The call's two launches meet in the workspace: while one thread enqueues them, no other may use it."""
    lib, _, call = setting
    first_inside, second_inside = threading.Event(), threading.Event()
    together = []

    def inside(workspace):
        if not first_inside.is_set():
            first_inside.set()
            # (a second caller would come in here, with the same buffer)
            together.append(second_inside.wait(0.5))
        else:
            second_inside.set()

    lib.inside = inside
    one = threading.Thread(target=call, args=(5,))
    one.start()
    assert first_inside.wait(10)
    two = threading.Thread(target=call, args=(5,))
    two.start()
    one.join(10)
    two.join(10)
    assert together == [False] and second_inside.is_set() and len(lib.workspaces) == 2


def test_a_failing_call_lets_the_next_one_in(setting):
    lib, _, call = setting

    def fail(workspace):
        raise RuntimeError("no")

    lib.inside = fail
    with pytest.raises(RuntimeError):
        call(5)
    lib.inside = lambda workspace: None
    call(5)
