"""The torch side of the paged key/value operators (paged.py) without a GPU:
tensors in host memory that say they are on device 0, with the library's entry
point replaced where a call would go on to the device."""
import ctypes
import gc
import threading
import weakref

import pytest

from dual_ar_tts_frame_gb300 import _lib as L
from dual_ar_tts_frame_gb300.build import build

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A host tensor that names device 0 as its own."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(OnDevice)


def i32(*v):
    return on(torch.tensor(v, dtype=torch.int32))


@pytest.fixture
def paged(monkeypatch):
    build()
    from dual_ar_tts_frame_gb300 import paged as P
    import contextlib
    monkeypatch.setattr(P, "_on", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(P, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return P


def attention_call(P, **over):
    kv = on(P.kv_pool(2, 2, 64, device="cpu"))[:, 0]
    a = dict(q=on(torch.zeros(3, 4, 64)), kv=kv, table=i32(0, 1)[None], row_start=i32(0, 3), kv_len=i32(70))
    a.update(over)
    return P.paged_attention(**a)


class Library:
    """The library with dualar_paged_attention replaced."""

    def __init__(self, lib, attention):
        self.lib, self.dualar_paged_attention = lib, attention

    def __getattr__(self, name):
        return getattr(self.lib, name)


# ---------------------------------------------------------------- workspaces --

def test_calls_of_two_threads_have_their_own_workspaces(paged, monkeypatch):
    """A call queues two kernels, and the interpreter runs other threads
    meanwhile: two calls that are inside the library at once hold two buffers,
    also on one stream (which all threads share by default)."""
    both = threading.Barrier(2, timeout=30)
    spans = []
    monkeypatch.setattr(paged.L, "lib", lambda lib=Library(L.load(), lambda *a: 0): lib)
    attention_call(paged)                # (an earlier call, which may leave a buffer behind)

    def attention(*a):
        both.wait()                      # both calls are in the library
        spans.append((a[16], a[17]))     # workspace, its bytes
        both.wait()
        return 0

    monkeypatch.setattr(paged.L, "lib", lambda lib=Library(L.load(), attention): lib)
    threads = [threading.Thread(target=attention_call, args=(paged,)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (a, n), (b, m) = sorted(spans)
    assert n > 0 and a + n <= b and m == n


def test_a_workspace_is_given_back(paged, monkeypatch):
    """Nothing stays allocated behind a call but its output."""
    seen = []
    make = torch.empty

    def empty(*a, **k):
        t = make(*a, **k)
        if k.get("dtype") is torch.uint8:
            seen.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(paged.L, "lib", lambda lib=Library(L.load(), lambda *a: 0): lib)
    out = attention_call(paged)
    gc.collect()
    assert out.shape == (3, 4, 64) and len(seen) == 1 and seen[0]() is None
