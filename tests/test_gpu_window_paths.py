"""The decoder with a sliding window along every path that a stream takes: 9 rows
and more (tensor-core projections), the full width (heads of 128, groups of four),
prompts of several chunks, continued prompts, shared prefixes, 4-bit weights, the
no-allocation call, released slots, and a window that changes between frames.  The
oracle runs the same model with the window in its slow attention's mask."""
import math

import numpy as np
import pytest

import oracle.model as M
from dualar_inputs import CONFIGS, TINY
from dualar_inputs import generators as g
from oracle import DualAROracle
from oracle import Sampling as OSampling
from parity import assert_logits_close

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
L1 = CONFIGS["s2pro_l1"]
SMP = OSampling(temperature=0.8, top_p=0.8, ras_win=10, allow_eos=False)


class WindowOracle(DualAROracle):
    """window positions back (itself among them) and the first sinks; 0: all."""
    window = sinks = 0

    def slow_rows(self, seq, x):
        def attention(q, k, v, n_rep, causal_offset=None):
            p = causal_offset + np.arange(q.shape[0])[:, None]
            j = np.arange(k.shape[0])[None, :]
            see = j <= p
            if self.window:
                see &= (j > p - self.window) | (j < self.sinks)
            s = np.einsum("qhd,khd->hqk", q, np.repeat(k, n_rep, 1)) / np.float32(math.sqrt(q.shape[2]))
            s = np.where(see[None], s, -np.inf)
            w = np.exp(s - s.max(-1, keepdims=True))
            return np.einsum("hqk,khd->qhd", w / w.sum(-1, keepdims=True), np.repeat(v, n_rep, 1)).astype(np.float32)

        plain = M.gqa_attention
        M.gqa_attention = attention
        try:
            return super().slow_rows(seq, x)
        finally:
            M.gqa_attention = plain


@pytest.fixture(scope="module", autouse=True)
def lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dual_ar_tts_frame_gb300 import build
    build()


@pytest.fixture(scope="module")
def tiny_weights(tiny_bits, lib_built):
    from dual_ar_tts_frame_gb300 import upload_weights
    return upload_weights(tiny_bits)


class Pair:
    """A decoder and its oracle."""

    def __init__(self, cfg, bits, weights, window, sinks, w4=None, **size):
        from dual_ar_tts_frame_gb300 import DualARDecoder, pack_w4a16
        size = dict(dict(max_pages=64, max_seqs=4, max_ctx=1024), **size)
        self.cfg, self.d, self.seqs = cfg, DualARDecoder(cfg, weights, **size), {}
        self.o = WindowOracle(cfg, bits, max_pos=size["max_ctx"] + 1, w4a16_keys=w4)
        if w4:
            self.d.set_w4a16({k: pack_w4a16(weights[k]) for k in w4})
        self.set(window, sinks)

    def set(self, window, sinks):
        self.d.set_attn_window(window, sinks)
        self.o.window, self.o.sinks = window, sinks

    def state(self, slot, what):
        for got, want in zip(self.d.read_state(slot), (self.seqs[slot].h_last, self.seqs[slot].z_last)):
            assert_logits_close(got, want, f"{what}, slot {slot}")

    def prefill(self, slot, prompt):
        self.d.prefill(slot, prompt)
        self.seqs[slot] = self.o.prefill(prompt)
        self.state(slot, "prefill")

    def append(self, slot, prompt):
        self.d.prefill_append(slot, prompt)
        self.o.prefill(prompt, self.seqs[slot])
        self.state(slot, "append")

    def frames(self, n, seed):
        from dual_ar_tts_frame_gb300 import Sampling
        slots = sorted(self.seqs)
        forced = g.make_forced_codes(n, len(slots), self.cfg, seed=seed)
        uni = g.make_uniforms(n, len(slots), self.cfg, seed=seed + 1)
        for f in range(n):
            _, status, slow, fast, _ = self.d.decode_frame_forced(
                slots, torch.from_numpy(uni[f]).cuda(), Sampling(0.8, 0.8, 10, allow_eos=False),
                torch.from_numpy(forced[f]).cuda())
            self.d.sync()
            assert (status == 0).all()
            for i, s in enumerate(slots):
                r = self.o.decode_frame(self.seqs[s], uni[f, i], SMP, forced=forced[f, i])
                assert_logits_close(slow[i].cpu().numpy(), r.slow_logits, f"frame {f} slot {s} slow")
                assert_logits_close(fast[i].cpu().numpy(), r.fast_logits, f"frame {f} slot {s} fast")
        for s in slots:
            self.state(s, "frames")


def test_twelve_rows(tiny_bits, tiny_weights):
    p = Pair(TINY, tiny_bits, tiny_weights, 30, 4, max_pages=128, max_seqs=16)
    for s, n in enumerate(g.make_lengths(12, 20, 200, seed=41, stream="tc_b12")):
        p.prefill(s, g.make_prompt(TINY, int(n), seed=140 + s))
    p.frames(3, 142)
    p.d.close()


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (100, 70), (513, 1)])
def test_prompts_of_several_chunks_and_continued_ones(tiny_bits, tiny_weights, window, sinks):
    """Chunks of 128 rows and what is left of them (1, 3 and 129 rows: either
    attention kernel), across pages."""
    p = Pair(TINY, tiny_bits, tiny_weights, window, sinks)
    p.prefill(0, g.make_prompt(TINY, 300, seed=150))
    p.prefill(2, g.make_prompt(TINY, 3, seed=151))
    for n in (1, 3, 129):
        p.append(0, g.make_prompt(TINY, n, seed=152 + n))
    p.append(2, g.make_prompt(TINY, 64, seed=153))
    p.frames(2, 154)
    p.append(2, g.make_prompt(TINY, 2, seed=155))
    p.frames(1, 156)
    p.d.close()


def test_shared_prefix(tiny_bits, tiny_weights):
    p = Pair(TINY, tiny_bits, tiny_weights, 40, 8)
    prefix = g.make_prompt(TINY, 150, seed=160)
    p.prefill(0, prefix)
    for s, n in ((1, 40), (3, 90)):
        p.d.share_prefix(0, s, 100)
        p.seqs[s] = p.o.prefill(prefix[:100])
        p.append(s, g.make_prompt(TINY, n, seed=161 + s))
    p.frames(2, 164)
    p.d.release(0)
    del p.seqs[0]
    p.frames(1, 165)
    p.prefill(0, g.make_prompt(TINY, 70, seed=166))      # the pages again
    p.frames(1, 167)
    p.d.close()


def test_four_bit_weights(tiny_bits, tiny_weights):
    from dual_ar_tts_frame_gb300 import late_attn_keys
    p = Pair(TINY, tiny_bits, tiny_weights, 50, 2, w4=late_attn_keys(TINY.n_layer, TINY.fast_n_layer, 1))
    for s, n in enumerate((170, 20)):
        p.prefill(s, g.make_prompt(TINY, n, seed=170 + s))
    p.frames(3, 172)
    p.d.close()


def test_window_that_changes_between_frames(tiny_bits, tiny_weights):
    """From the next call on; off goes back to the persistent kernel."""
    p = Pair(TINY, tiny_bits, tiny_weights, 0, 0)
    p.prefill(0, g.make_prompt(TINY, 180, seed=180))
    for k, setting in enumerate(((20, 0), (0, 5), (90, 65), (1000, 0), (0, 0))):
        p.set(*setting)
        p.frames(1, 181 + 2 * k)
    p.d.close()


def test_noalloc_call(tiny_weights):
    """The same frames by dualar_decode_frame_noalloc."""
    from dual_ar_tts_frame_gb300 import DualARDecoder, Sampling
    d = DualARDecoder(TINY, tiny_weights, max_pages=32, max_seqs=4, max_ctx=512)
    d.set_attn_window(60, 4)
    prompt = g.make_prompt(TINY, 150, seed=190)
    d.prefill(0, prompt)
    d.prefill(1, prompt)
    smp = Sampling(temperature=0.8, top_p=0.8, ras_win=10)
    uni = torch.from_numpy(g.make_uniforms(3, 1, TINY, seed=191)).cuda()
    codes = torch.empty((1, TINY.n_codebooks), dtype=torch.int32, device="cuda")
    status = torch.empty((1,), dtype=torch.int32, device="cuda")
    for call in range(3):
        want, want_status = d.decode_frame([0], uni[call], smp)
        d.decode_frame_noalloc([1], uni[call], smp, codes, status)
        d.sync()
        assert torch.equal(codes, want) and torch.equal(status, want_status)
        for a, b in zip(d.read_state(0), d.read_state(1)):
            assert_logits_close(b, a, f"call {call}")
    d.close()


def test_full_width():
    """32 query and 8 key/value heads of 128, one layer each."""
    from dual_ar_tts_frame_gb300 import upload_weights
    bits = g.make_weights(L1, seed=0)
    p = Pair(L1, bits, upload_weights(bits), 200, 6, max_pages=64, max_seqs=12)
    p.prefill(0, g.make_prompt(L1, 700, seed=200))
    p.frames(2, 201)
    for s, n in ((1, 130), (2, 9)):
        p.prefill(s, g.make_prompt(L1, n, seed=202 + s))
    p.append(2, g.make_prompt(L1, 150, seed=206))
    p.frames(2, 207)
    for s in range(3, 10):
        p.prefill(s, g.make_prompt(L1, 20 + 11 * s, seed=210 + s))
    p.frames(1, 220)
    p.d.close()
    torch.cuda.empty_cache()
