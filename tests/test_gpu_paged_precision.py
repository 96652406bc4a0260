"""How many bits of a weight and of a query the attention kernels keep, by inputs
whose leading bits cancel: what is left of the output is what a narrower weight
or query would lose.  Both kernels (few and many rows per request), both caches,
both types of activations."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
PAGE, D = 64, 64


@pytest.fixture(scope="module", autouse=True)
def lib_built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dual_ar_tts_frame_gb300 import build
    build()


def bf16(x):
    return float(torch.tensor(x, dtype=torch.float64).to(torch.bfloat16))


def one_page(keys, values, bits):
    """One head's page whose first tokens have the given vectors ({element: value},
    every value a power of two, or its token's only one), the others zeros."""
    y = torch.zeros((2, PAGE, D), dtype=torch.float64)
    for side, vectors in ((0, keys), (1, values)):
        for t, v in enumerate(vectors):
            for i, x in v.items():
                y[side, t, i] = x
    if bits == 16:
        kv = y.to(torch.bfloat16)[None, :, None].cuda()
        assert torch.equal(kv[0, :, 0].cpu().double(), y)
        return kv
    # the scale is the largest element, or a quarter of it, with codes 1 to 4
    scale = y.abs().amax(-1, keepdim=True)
    least = torch.where(y != 0, y.abs(), math.inf).amin(-1, keepdim=True)
    scale = torch.where(least < scale, scale / 4, scale)
    code = torch.where(scale > 0, y / torch.where(scale > 0, scale, 1.0), 0.0)
    assert torch.equal(code.round() * scale, y) and code.abs().max() <= 7
    u = (code + 8).to(torch.int32)
    byte = (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8).flatten(1)
    sc = scale.to(torch.bfloat16)
    assert torch.equal(sc.double(), scale)
    return torch.cat([byte, sc.flatten(1).contiguous().view(torch.uint8)], 1)[None, :, None].contiguous().cuda()


def attend(q, kv, n, scale):
    """A query [D] that sees the page's first n tokens, by each kernel: alone, and as
    the 32 heads of the last of two tokens of a request (64 rows)."""
    from dual_ar_tts_frame_gb300 import paged_attention

    def call(rows, heads):
        def i32(*v):
            return torch.tensor(v, dtype=torch.int32, device="cuda")

        x = q[None, None].expand(rows, heads, D).contiguous()
        return paged_attention(x, kv, i32(0)[None], i32(0, rows), i32(n), scale=scale)[-1].double().cpu()

    return {"few": call(1, 1), "many": call(2, 32)}


# Weights.  Tokens with equal scores of 0 (weight 1) take off a leading part of the last
# token's weight w = e^-s, 0.5 < w < 1; what is left of sum_j w_j v_j is w's next bits.
# What else may be off, relative to w: 2^-22 by the exponential's instruction, 2^-24 each
# by the product with log2(e) and the rounded scale (their effect is s <= 0.7 times
# that), and at most 2^-23 for each of the additions in an accumulator that truncates:
# 3 for a tile's parts and one to the running output.
REST = 2.0 ** -22 + 2 * 2.0 ** -24 + 4 * 2.0 ** -23


def weight_with(bits_off, at_least):
    """s (an fp32 value) whose weight keeps `at_least` of itself behind its first
    bits_off bf16 parts; those parts."""
    rng = np.random.default_rng(3)
    while True:
        s = float(np.float32(rng.uniform(0.1, 0.6)))
        w, parts = math.exp(-s), []
        for _ in range(bits_off):
            parts.append(bf16(w - sum(parts)))
        left = w - sum(parts)
        if left > at_least and all(p > 0 for p in parts):
            return s, w, parts, left


# what a weight may be off by itself: fp32 rows keep three bf16 parts (24 bits), bf16 rows
# two (16 bits); over 4 bits few rows keep two fp16 parts (22 bits)
KEPT = {(torch.float32, 16, "few"): 24, (torch.float32, 4, "few"): 22, (torch.float32, 16, "many"): 24,
        (torch.float32, 4, "many"): 24, (torch.bfloat16, 16, "few"): 16, (torch.bfloat16, 4, "few"): 22,
        (torch.bfloat16, 16, "many"): 16, (torch.bfloat16, 4, "many"): 16}


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("act,off", [(torch.float32, 2), (torch.bfloat16, 1)])
def test_bits_of_a_weight(bits, act, off):
    s, w, parts, left = weight_with(off, 0.9 * 2.0 ** (-10 if off == 1 else -19))
    keys = [{}] * off + [{0: -1.0}]
    values = [{5: -p} for p in parts] + [{5: 1.0}]
    kv = one_page(keys, values, bits)
    q = torch.zeros(D, dtype=act, device="cuda")
    q[0] = 1
    exact = left / (off + w)
    for kernel, got in attend(q, kv, off + 1, s).items():
        # half a step: of n significant bits, at most 2^-n of the value (just above a power
        # of two the step is 2^(1 - n) of it)
        kept = 2.0 ** -KEPT[act, bits, kernel]
        tol = w * (kept + REST) / (off + w) + exact * torch.finfo(act).eps / 2
        other = 0.0                                         # of elements that are zero in all values
        if act == torch.bfloat16 and bits == 4 and kernel == "few":
            # sums over u = q + 8 that start at -8 times the weights' sum: 8 additions for
            # the start and at most 8 for the codes, of terms up to 15 w_j s_j (s_j the value's
            # scale), each truncated at 2^-23 of its size: 16 * 15 * 2^-23 < 2^-15 of sum w_j s_j
            other = 2.0 ** -15 * (sum(parts) + w) / (off + w)
            tol += other
        err = (got[:, 5] - exact).abs().max().item()
        assert err <= tol, (kernel, err, tol, exact)
        assert max(got[:, :5].abs().max().item(), got[:, 6:].abs().max().item()) <= other


@pytest.mark.parametrize("bits", [16, 4])
def test_bits_of_a_query(bits):
    """fp32 queries: the two tokens' scores, near 400 each, differ by what the
    query's bits behind the 16th say.  A score is off by half a step of fp32 twice (as
    scaled, and in the exponent, of which the maximum's share cancels) and a step for
    each of up to 8 truncated additions: 400 * (2 * 2^-24 + 8 * 2^-23); a query of 22
    bits (fp16 parts) adds 400 * 2^-22."""
    scale, rng = 256.0, np.random.default_rng(4)
    while True:
        x = float(np.float32(rng.uniform(1.0, 2.0)))
        top = bf16(x) + bf16(x - bf16(x))                   # two bf16 parts
        if x - top > 0.85 * 2.0 ** -17:
            break
    q = torch.zeros(D, device="cuda")
    q[0], q[1] = x, top
    kv = one_page([{0: 1.0}, {1: 1.0}], [{3: 1.0}, {4: 1.0}], bits)
    diff = scale * (x - top)
    exact = torch.tensor([1 / (1 + math.exp(-diff)), 1 / (1 + math.exp(diff))], dtype=torch.float64)
    ds = scale * x * (2 * 2.0 ** -24 + 8 * 2.0 ** -23 + (2.0 ** -22 if bits == 4 else 0.0))
    assert ds < diff / 2.5
    for kernel, got in attend(q, kv, 2, scale).items():
        # an output moves by at most a quarter of a score difference's error (two scores)
        err = (got[:, 3:5] - exact).abs().max().item()
        assert err <= 0.25 * 2 * ds + 2.0 ** -20, (kernel, err, ds, diff)
