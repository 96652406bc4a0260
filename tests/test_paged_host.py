"""Host-only checks of the paged key/value operators: symbols, struct layout,
block sizes, refusals before any GPU work, and the plain 64-bit forms the GPU
tests compare with."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from dual_ar_tts_frame_gb300 import _lib as L
from dual_ar_tts_frame_gb300.build import build

torch = pytest.importorskip("torch")
import paged_ref as R  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dualar_paged.h")


@pytest.fixture(scope="module")
def lib():
    build()
    return L.load()


def message(lib):
    buf = ctypes.create_string_buffer(256)
    assert lib.dualar_paged_error(buf, 256) == 0
    return buf.value.decode()


def test_header_and_binding_agree(lib, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(dualar_[a-z0-9_]+)\s*\(", text))) == sorted(L.EXPORTED_PAGED)
    for n in L.EXPORTED_PAGED:
        assert hasattr(lib, n)
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dualar_paged.h"\n'
                   'int main(void){printf("%zu %zu %zu\\n", sizeof(dualar_kv), offsetof(dualar_kv, page_stride),'
                   ' offsetof(dualar_kv, bits));return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    assert list(map(int, subprocess.check_output([str(exe)]).split())) == [
        ctypes.sizeof(L.dualar_kv), L.dualar_kv.page_stride.offset, L.dualar_kv.bits.offset]


def test_page_bytes(lib):
    f = lib.dualar_kv_page_bytes
    assert f(8, 128, 16) == 2 * 8 * 64 * 128 * 2 and f(8, 128, 4) == 2 * 8 * (64 * 64 + 128)
    assert f(2, 64, 4) == 2 * 2 * (64 * 32 + 128)
    for a in ((0, 128, 16), (8, 96, 16), (8, 128, 8), (-1, 64, 4), (2000, 64, 4)):
        assert f(*a) == -1


GOOD_KV = dict(data=1 << 20, page_stride=2 * 2 * 64 * 64 * 2, n_pages=4, n_kv_head=2, head_dim=64, bits=16)


def kv(**over):
    k = L.dualar_kv(**{**GOOD_KV, **over})
    return k


BAD_KV = [dict(data=None), dict(data=(1 << 20) + 8), dict(page_stride=100), dict(page_stride=2 * 2 * 64 * 64 * 2 + 8),
          dict(n_pages=0), dict(n_pages=1 << 25), dict(head_dim=80), dict(bits=8), dict(n_kv_head=0)]
P = 1 << 21     # an aligned address that is never read


def attention_args(**over):
    a = dict(q=P, act=0, ldq=256, rows=3, n_head=4, kv=kv(), table=P, width=5, row_start=P, kv_len=P, n_seq=2, window=0,
             sinks=0, scale=0.1, out=P, ldo=256, workspace=P, nbytes=1 << 40, err=None, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over", [dict(q=None), dict(q=P + 4), dict(act=2), dict(ldq=255), dict(ldq=258), dict(rows=-1), dict(rows=(1 << 24) + 1),
                                  dict(n_head=3), dict(n_head=0), dict(n_head=66), dict(table=None), dict(width=-1),
                                  dict(width=(1 << 20) + 1), dict(row_start=None), dict(kv_len=None), dict(n_seq=-1),
                                  dict(n_seq=8193), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
                                  dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(out=P + 8),
                                  dict(ldo=200), dict(act=1, ldq=260)] + [dict(kv=kv(**b)) for b in BAD_KV])
def test_attention_refusals(lib, over):
    assert lib.dualar_paged_attention(*attention_args(**over)) == -1
    assert message(lib)


def test_attention_of_nothing_is_fine(lib):
    assert lib.dualar_paged_attention(*attention_args(rows=0, q=None, out=None)) == 0
    assert lib.dualar_paged_attention(*attention_args(n_seq=0)) == 0


def test_attention_workspace(lib):
    f = lib.dualar_paged_attention_workspace
    need = f(0, 3, 4, kv(), 2)
    assert need >= 0
    if need:
        assert lib.dualar_paged_attention(*attention_args(nbytes=need - 1)) == -1 and "workspace" in message(lib)
        assert lib.dualar_paged_attention(*attention_args(workspace=None)) == -1
        assert lib.dualar_paged_attention(*attention_args(workspace=P + 8)) == -1
    for bad in ((2, 3, 4, kv(), 2), (0, -1, 4, kv(), 2), (0, 3, 5, kv(), 2), (0, 3, 66, kv(), 2), (0, 3, 4, None, 2),
                (0, 3, 4, kv(bits=5), 2), (0, 3, 4, kv(), 9000)):
        assert f(*bad) == -1


def rope_args(**over):
    a = dict(qkv=P, act=1, ld=512, rows=3, n_head=4, kv=kv(), pos=P, slot=P, qn=P, kn=P, eps=1e-6, cos=P, sin=P,
             n_pos=10, out=P, ldq=256, err=None, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over", [dict(qkv=None), dict(qkv=P + 2), dict(act=-1), dict(ld=500), dict(ld=516), dict(rows=-1), dict(rows=(1 << 24) + 1),
                                  dict(n_head=0), dict(n_head=5000), dict(pos=None), dict(slot=None), dict(qn=None),
                                  dict(kn=None), dict(kn=P + 2), dict(eps=0.0), dict(cos=None), dict(sin=P + 2),
                                  dict(n_pos=0), dict(out=None), dict(ldq=255)] + [dict(kv=kv(**b)) for b in BAD_KV])
def test_norm_rope_refusals(lib, over):
    assert lib.dualar_qk_norm_rope(*rope_args(**over)) == -1
    assert message(lib)


def test_norm_rope_and_read_of_nothing_are_fine(lib):
    assert lib.dualar_qk_norm_rope(*rope_args(rows=0)) == 0
    assert lib.dualar_kv_read(kv(), None, 0, None, None, None, None) == 0
    for bad in ((None, P, 1, P, P), (kv(), None, 1, P, P), (kv(), P, -1, P, P), (kv(), P, 1, None, P), (kv(), P, 1, P, P + 4)):
        assert lib.dualar_kv_read(*bad, None, None) == -1


def plan_args(**over):
    a = dict(kv_len=P, n_new=P, n_seq=2, refs=P, n_pages=4, table=P, width=3, max_rows=8, row_start=P, pos=P, slot=P,
             new_len=P, status=P, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over", [dict(kv_len=None), dict(n_new=None), dict(n_seq=-1), dict(n_seq=8193), dict(refs=None),
                                  dict(n_pages=-1), dict(n_pages=1 << 25), dict(table=None), dict(width=-1),
                                  dict(width=(1 << 20) + 1), dict(max_rows=-1), dict(max_rows=(1 << 24) + 1),
                                  dict(row_start=None), dict(pos=None), dict(slot=None), dict(new_len=None),
                                  dict(status=None)])
def test_plan_refusals(lib, over):
    assert lib.dualar_kv_plan(*plan_args(**over)) == -1
    assert message(lib)


def test_python_refusals_on_the_cpu(lib):
    """Tensors that are no device tensors of the right kind never reach the library."""
    import dual_ar_tts_frame_gb300 as D
    i = torch.zeros(4, dtype=torch.int32)
    pool = D.kv_pool(3, 2, 64, device="cpu")
    assert pool.shape == (3, 1, 2, 2, 64, 64) and D.kv_pool(3, 2, 64, 4, 5, "cpu").shape == (3, 5, 2, 2, 2176)
    for call in (lambda: D.kv_plan(i, i, i, i[None], 4), lambda: D.kv_read(pool[:, 0], i),
                 lambda: D.paged_attention(torch.zeros(1, 4, 64), pool[:, 0], i[None], i[:2], i[:1]),
                 lambda: D.qk_norm_rope(torch.zeros(4, 512), pool[:, 0], i, i, None, None, pool, pool),
                 lambda: D.kv_page_bytes(2, 80), lambda: D.kv_pool(3, 2, 64, bits=8, device="cpu")):
        with pytest.raises(L.DualARError):
            call()


def test_rope_tables_are_the_oracles():
    import dual_ar_tts_frame_gb300 as D
    from oracle.model import rope_table
    c, s = D.rope_tables(50, 64, device="cpu")
    oc, os_ = rope_table(50, 64, 1e6)
    assert np.array_equal(c.float().numpy(), np.asarray(oc, np.float32)[:50])
    assert np.array_equal(s.float().numpy(), np.asarray(os_, np.float32)[:50])


# ---- the plain forms themselves ------------------------------------------------

def test_plain_quantize_is_the_packed_weights_rule():
    """On vectors of 128 the cache's rule is the 4-bit weights' rule."""
    from dualar_inputs.generators import bf16_bits_to_f32, f32_to_bf16_bits
    from oracle import w4a16
    rng = np.random.default_rng(3)
    bits = f32_to_bf16_bits((rng.standard_normal((300, 128)) * 3).astype(np.float32))
    q, s = R.quantize(torch.from_numpy(bf16_bits_to_f32(bits).astype(np.float64)))
    oq, os_ = w4a16.quantize(bits)
    assert np.array_equal(q.numpy().astype(np.int8), oq)
    assert np.array_equal(s.numpy()[:, 0], bf16_bits_to_f32(os_)[:, 0].astype(np.float64))


def test_plain_plan_by_hand():
    out, refs, table = R.plan([63, 0, 128], [2, 1, 0], np.array([1, 0, 1, 0, 1, 1]),
                              np.array([[0, -1], [-1, -1], [4, 5]]), 5)
    assert out["status"] == [0, 3, 2] and out["slot"] == [63, 64, 3 * 64, -1, -1] and out["pos"] == [63, 64, 0, 0, 0]
    assert table.tolist() == [[0, 1], [3, -1], [4, 5]] and refs.tolist() == [1, 1, 1, 1, 1, 1]
    assert out["row_start"] == [0, 2, 3, 3] and out["new_len"] == [65, 1, 128]


def test_plain_attention_by_hand():
    """One visible token returns its value; a window of two with one sink
    averages three equal scores."""
    kv = torch.zeros((1, 2, 1, 64, 64), dtype=torch.bfloat16)
    kv[0, 1, 0, :, 0] = torch.arange(64)
    table, start = torch.zeros((1, 1), dtype=torch.int32), torch.tensor([0, 2])
    q = torch.zeros((2, 1, 64))
    out, _ = R.attention(q, kv, table, start, torch.tensor([2]), 1, 0)
    assert out[:, 0, 0].tolist() == [0.0, 1.0]
    out, _ = R.attention(q, kv, table, start, torch.tensor([10]), 2, 1)
    assert out[0, 0, 0].item() == pytest.approx((0 + 7 + 8) / 3) and out[1, 0, 0].item() == pytest.approx((0 + 8 + 9) / 3)


def test_window_needs_a_handle(lib):
    assert lib.dualar_set_attn_window(None, 4, 0) == -1


@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (2 ** 32 + 4, 0), (4, 2 ** 32), (-2 ** 32 + 4, 0)])
def test_window_that_no_int32_holds(lib, window, sinks):
    """Refused by the binding: the library would get its low bits."""
    import dual_ar_tts_frame_gb300 as D

    class Handle:
        calls = []
        h = None

        class lib:
            dualar_set_attn_window = staticmethod(lambda *a: Handle.calls.append(a) or 0)

        def _check(self, rc):
            assert rc == 0

    with pytest.raises(L.DualARError):
        D.DualARDecoder.set_attn_window(Handle(), window, sinks)
    D.DualARDecoder.set_attn_window(Handle(), 5, 2)
    assert Handle.calls == [(None, 5, 2)]
