"""The torch side of the paged key/value operators (paged.py) without a GPU:
tensors in host memory that say they are on device 0, with the library's entry
point replaced where a call would go on to the device."""
import gc
import os
import re
import threading
import weakref

import pytest

from dual_ar_tts_frame_gb300 import _lib as L
from dual_ar_tts_frame_gb300.build import build

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# ------------------------------------------------------------------- strides --

def rope_call(P, **over):
    kv = on(P.kv_pool(2, 2, 64, device="cpu"))[:, 0]
    cos, sin = (on(t) for t in P.rope_tables(8, 64, device="cpu"))
    a = dict(qkv=on(torch.zeros(3, 8 * 64)), kv=kv, pos=i32(0, 1, 2), slot=i32(0, 1, 2), q_norm=None, k_norm=None, cos=cos,
             sin=sin)
    a.update(over)
    return P.qk_norm_rope(**a)


def refused(call, *a, **k):
    """Refused as an argument, before anything is queued."""
    with pytest.raises(L.DualARError) as e:
        call(*a, **k)
    assert e.value.code == -1, e.value


@pytest.mark.parametrize("rows", [3, 2])
def test_rows_that_overlap_are_refused(paged, rows):
    """Expanded and overlapping rows hold fewer elements than rows * width: read
    or written as whole rows they would go past the tensor."""
    d, start, pos = 64, i32(0, rows), i32(*range(rows))
    q = on(torch.zeros(rows, 4, d))
    refused(attention_call, paged, q=q[:1].expand(rows, 4, d), row_start=start)
    refused(attention_call, paged, q=on(torch.zeros(4 * d + 64 * rows)).as_strided((rows, 4, d), (64, d, 1)), row_start=start)
    refused(attention_call, paged, q=q, out=q[:1].expand(rows, 4, d), row_start=start)
    qkv = on(torch.zeros(rows, 8 * d))
    refused(rope_call, paged, qkv=qkv[:1].expand(rows, 8 * d), pos=pos, slot=pos)
    refused(rope_call, paged, qkv=qkv, pos=pos, slot=pos, out=q[:1].expand(rows, 4, d))


def test_a_row_that_is_not_contiguous_is_refused(paged):
    """Also where it is the only one."""
    wide = on(torch.zeros(1, 2 * 8 * 64))
    refused(rope_call, paged, qkv=wide[:, ::2], pos=i32(0), slot=i32(0))
    refused(rope_call, paged, qkv=on(torch.zeros(8 * 64, 3)).t())
    heads = on(torch.zeros(1, 4, 128))
    refused(attention_call, paged, q=heads[:, :, ::2], row_start=i32(0, 1))


@pytest.mark.parametrize("stride", [0, 1, 7, 1001, 10 ** 6])
def test_the_stride_of_a_single_row_says_nothing(paged, monkeypatch, stride):
    """A row stride is only used between rows: torch gives a single row any."""
    got = []
    lib = Library(L.load(), lambda *a: got.append((a[2], a[15])) or 0)
    lib.dualar_qk_norm_rope = lambda *a: got.append((a[2], a[15])) or 0
    monkeypatch.setattr(paged.L, "lib", lambda: lib)
    base = on(torch.zeros(8 * 64))
    q = base.as_strided((1, 4, 64), (stride, 64, 1))
    attention_call(paged, q=q, out=q, row_start=i32(0, 1))
    rope_call(paged, qkv=base.as_strided((1, 8 * 64), (stride, 1)), pos=i32(0), slot=i32(0), out=q)
    for ld, ldo in got:
        assert ld >= 256 and ldo >= 256 and ld % 8 == 0 and ldo % 8 == 0
    assert len(got) == 2


# -------------------------------------------------------------- error reports --

@pytest.mark.parametrize("word,says", [(1, "wait"), (4, "slot"), (8, "page"), (5, "wait.* and .*slot")])
def test_every_bit_of_the_error_word_is_named(paged, word, says):
    header = open(os.path.join(ROOT, "include", "dualar_paged.h")).read()
    bits = dict(re.findall(r"(DUALAR_PAGED_ERR_\w+) = 1 << (\d)", header))
    assert sorted(bits.values()) == ["0", "2", "3"]
    err = torch.tensor([word], dtype=torch.int32)
    with pytest.raises(L.DualARError, match=says) as e:
        paged.check_errors(err)
    assert e.value.code == -7 and err.item() == 0


# ------------------------------------------------------------------- integers --

@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63, -2 ** 32 + 5, -1])
def test_integers_that_no_int32_holds_are_refused(paged, big):
    """ctypes keeps an integer's low bits: a window of 2^32 + 5 would be one of 5."""
    refused(attention_call, paged, window=big)
    refused(attention_call, paged, window=7, sinks=big)
    refused(paged.kv_plan, i32(3), i32(1), i32(0), i32(0)[None], big)
    for shape in ((big, 64, 16), (8, big, 16), (8, 64, big)):
        refused(paged.kv_page_bytes, *shape)
        refused(paged.kv_pool, 1, *shape, device="cpu")
    refused(paged.kv_plan, i32(3), i32(1), i32(0), i32(0)[None], 2 ** 24 + 1)
