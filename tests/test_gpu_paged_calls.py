"""Paged key/value operators on the GPU as a program calls them: from several
threads, from other streams, in mixed and padded steps; and the weights' and
queries' precision by inputs that show it."""
import ctypes
import os
import subprocess
import threading

import numpy as np
import pytest

import paged_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
PAGE = R.PAGE


@pytest.fixture(scope="module", autouse=True)
def lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dual_ar_tts_frame_gb300 import build
    build()


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    return g


def i32(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


@pytest.mark.parametrize("bits,new", [(16, [1, 1]), (4, [1, 1]), (16, [300, 200])])
def test_two_threads_on_one_stream(gen, bits, new):
    """Two threads call on the default stream at once, many times, each with its
    own queries: every output is the one its queries give alone."""
    from dual_ar_tts_frame_gb300 import paged_attention
    kv = R.random_layer(150, 8, 128, bits, gen)[:, 0]
    table, start, lens = R.layout(new, [4000, 5000], 150)
    qs = [torch.randn((sum(new), 32, 128), generator=gen, device="cuda") for _ in range(2)]
    want = [paged_attention(q, kv, table, start, lens) for q in qs]
    torch.cuda.synchronize()
    got, go = [[], []], threading.Barrier(2)

    def work(i):
        go.wait()
        for _ in range(50):
            got[i].append(paged_attention(qs[i], kv, table, start, lens))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 50 and all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("h,hk,d", [(4, 2, 64), (2, 1, 64), (5, 3, 64), (3, 1, 128), (7, 7, 128), (8, 2, 128)])
@pytest.mark.parametrize("size", [1e-17, 1e17])
def test_4_bit_keys_that_need_64_bits_beside_values(gen, h, hk, d, size):
    """Sums of squares outside the fp32 rule's range: every key is computed again
    in 64 bits, in warps that hold queries and values too."""
    from dual_ar_tts_frame_gb300 import kv_read, qk_norm_rope, rope_tables
    rows = 40
    pool = R.random_layer(2, hk, d, 4, gen)
    qkv = torch.randn((rows, (h + 2 * hk) * d), generator=gen, device="cuda") * size
    g = [(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    pos, slot = i32(np.arange(rows) * 3), i32(np.arange(rows) + 50)
    cos, sin = rope_tables(200, d)
    qk_norm_rope(qkv, pool[:, 0], pos, slot, *g, cos, sin)
    x = qkv.double().reshape(rows, -1, d)
    k = R.norm_rope(x[:, h:h + hk], g[1].double(), cos[pos.long()].double(), sin[pos.long()].double(),
                    float(np.float32(1e-6)))
    for got, y in zip(kv_read(pool[:, 0], slot), (k, x[:, h + hk:])):
        assert torch.equal(got.double(), torch.mul(*R.quantize(y)))


@pytest.mark.parametrize("n", [2, 1500])
@pytest.mark.parametrize("page", [-1, 9000, 1 << 25, 1 << 30, -(1 << 31)])
def test_a_plan_into_a_page_out_of_range_is_refused(n, page):
    """The page of a request's last tokens is the caller's table entry: where it is
    out of range (times 64 it may even wrap to another page's slots) nothing is
    planned.  An entry that gets no token is not looked at."""
    from dual_ar_tts_frame_gb300 import kv_plan
    refs, table = i32(np.zeros(9000)), i32(np.arange(3 * n).reshape(n, 3))
    refs[:3 * n] = 1
    lens, new = np.full(n, 70), np.full(n, 3)
    bad = n - 1
    table[bad, 1] = page
    keep = refs.clone(), table.clone()
    p = kv_plan(i32(lens), i32(new), refs, table, 3 * n + 5)
    assert p.status.tolist() == [5, 3 * n, 0] and (p.slot == -1).all() and (p.pos == 0).all()
    assert (p.row_start == 0).all() and p.new_len.tolist() == lens.tolist()
    assert torch.equal(refs, keep[0]) and torch.equal(table, keep[1])
    new[bad] = 0                                 # no token for it
    assert kv_plan(i32(lens), i32(new), refs, table, 3 * n + 5).status.tolist() == [0, 3 * n - 3, 0]
    new[bad], lens[bad] = 3, 64                  # its next token goes to a new page
    table[bad, 1:] = page
    p = kv_plan(i32(lens), i32(new), refs, table, 3 * n + 5)
    assert p.status.tolist() == [0, 3 * n, 1] and p.slot[3 * n - 3:3 * n].tolist() == [3 * n * 64 + i for i in range(3)]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("act", [torch.float32, torch.bfloat16])
def test_a_mixed_step_in_one_call_and_in_two(gen, bits, act):
    """Many single tokens beside a chunk of a prompt: in one call (whichever kernel
    that takes), and the single tokens in one, the chunk in another over the same
    tensors, which leaves the first one's rows alone."""
    from dual_ar_tts_frame_gb300 import paged_attention
    singles, h, hk, d = 70, 8, 2, 128
    new, ctx = [1] * singles + [400, 33], [1 + 9 * i for i in range(singles)] + [900, 33]
    n_pages = sum(-(-c // PAGE) for c in ctx) + 1
    kv = R.random_layer(n_pages, hk, d, bits, gen)[:, 0]
    table, start, lens = R.layout(new, ctx, n_pages)
    q = torch.randn((sum(new), h, d), generator=gen, device="cuda").to(act)
    for window, sinks in ((0, 0), (100, 3)):
        R.assert_attention(paged_attention(q, kv, table, start, lens, window, sinks), q, kv, table, start, lens, window, sinks)
        out = torch.full_like(q, 7.0)
        paged_attention(q, kv, table[singles:], start[singles:], lens[singles:], window, sinks, out=out)
        assert (out[:singles] == 7).all()
        paged_attention(q[:singles], kv, table[:singles], start[:singles + 1], lens[:singles], window, sinks, out=out[:singles])
        R.assert_attention(out, q, kv, table, start, lens, window, sinks)


SHIM = r"""
#include "paged.h"
// The prompt kernel and its join; no_waiting: its waits run out at once.
extern "C" int prompt_call(const void* q, int rows, int n_head, void* kv, long long stride, int n_pages, int hk,
                                 int hd, int bits, const int* table, int width, const int* row_start, const int* kv_len,
                                 int n_seq, void* out, void* ws, unsigned* err, int bf16, int no_waiting, void* stream) {
  dualar::AttnArgs a{};
  a.q = q;
  a.ldq = a.ldo = static_cast<long long>(n_head) * hd;
  a.rows = rows;
  a.n_head = n_head;
  a.kv = dualar::KvView{static_cast<unsigned char*>(kv), stride, n_pages, hk, hd, bits};
  a.table = table;
  a.width = width;
  a.row_start = row_start;
  a.kv_len = kv_len;
  a.n_seq = n_seq;
  a.scale = 0.1f;
  a.out = out;
  a.ws = static_cast<float*>(ws);
  a.err = err;
  a.no_waiting = no_waiting;
  return dualar::launch_attn_prompt(a, bf16 != 0, dualar::kAttnSms, static_cast<cudaStream_t>(stream));
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    from dual_ar_tts_frame_gb300 import _lib as L
    L.load()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc, include = os.path.join(root, "dual_ar_tts_frame_gb300", "csrc"), os.path.join(root, "include")
    out = tmp_path_factory.mktemp("shim")
    (out / "shim.cpp").write_text(SHIM)
    so = str(out / "shim.so")
    subprocess.check_call(["g++", "-std=c++17", "-shared", "-fPIC", "-I", csrc, "-I", include, "-I", "/usr/local/cuda/include",
                           str(out / "shim.cpp"), "-o", so, L.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(L.LIB_PATH)}"])
    f = ctypes.CDLL(so).prompt_call
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong] + [ctypes.c_int] * 4 + [
        ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 3 + [
        ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("act", [torch.float32, torch.bfloat16])
def test_a_wait_that_runs_out_leaves_no_wrong_rows(gen, shim, bits, act):
    """Where the kernel's waits run out (here: at once) all rows are NaN
    (not those of the units that ended in time only), rows behind the last request
    stay as they were, and the error word says so.  With the usual limit the same
    call is right behind it."""
    from dual_ar_tts_frame_gb300 import paged_attention
    h, hk, d, new, ctx = 8, 2, 128, [300, 500], [900, 700]
    kv = R.random_layer(30, hk, d, bits, gen)[:, 0]
    table, start, lens = R.layout(new, ctx, 30)
    q = torch.randn((sum(new) + 4, h, d), generator=gen, device="cuda").to(act)
    want = paged_attention(q, kv, table, start, lens, scale=0.1)
    ws = torch.zeros(50 << 20, dtype=torch.uint8, device="cuda")
    for no_waiting in (0, 1, 0):
        out, err = torch.full_like(q, 3.0), i32([0])
        rc = shim(q.data_ptr(), sum(new) + 4, h, kv.data_ptr(), kv.stride(0) * kv.element_size(), 30, hk, d, bits,
                  table.data_ptr(), table.shape[1], start.data_ptr(), lens.data_ptr(), 2, out.data_ptr(), ws.data_ptr(),
                  err.data_ptr(), act == torch.bfloat16, no_waiting, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert (out[sum(new):] == 3).all()
        if no_waiting:
            assert int(err.item()) == 1 and torch.isnan(out[:sum(new)]).all()
        else:
            assert int(err.item()) == 0 and torch.equal(out[:sum(new)], want[:sum(new)])


def test_errors_of_another_stream_are_waited_for(gen):
    """check_errors on the default stream, while the call that reports is still
    queued behind other work on a stream of its own."""
    from dual_ar_tts_frame_gb300 import check_errors, kv_read
    from dual_ar_tts_frame_gb300._lib import DualARError
    kv = R.random_layer(2, 2, 64, 16, gen)[:, 0]
    slot, err, side = i32([128]), i32([0]), torch.cuda.Stream()
    kv_read(kv, i32([0]))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10 ** 8)
        kv_read(kv, slot, err=err)
    with pytest.raises(DualARError, match="slot"):
        check_errors(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
