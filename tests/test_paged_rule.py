"""The 4-bit rule of the paged cache on the CPU: its device text (paged.cuh)
compiled for the host with a warp of 32 threads (tests/warpsim), against the
plain 64-bit rule.  The lanes of a warp hold vectors of different kinds (queries
and values as they are, keys normed and rotated); whatever each takes, all lanes
have to go through every shuffle together."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_ref as R  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIM = os.path.join(ROOT, "tests", "warpsim")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("rule")
    text = open(os.path.join(ROOT, "dual_ar_tts_frame_gb300", "csrc", "paged.cuh")).read()
    a, b = text.index("// ---- the 4-bit rule, exact"), text.rindex("}  // namespace")
    (out / "rule.h").write_text(text[a:b])
    so = str(out / "rule.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-fPIC", "-shared", "-pthread", "-w", "-I", SIM, "-I",
                           str(out), os.path.join(SIM, "quantize.cpp"), "-o", so])
    return ctypes.CDLL(so)


def ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def quantized(rule, x, g, cos, sin, raw, norm, eps=1e-6):
    """Codes, scales (as float64) and whether the warp kept together, of its
    vectors x [n, d]."""
    n, d = x.shape
    x = x.astype(np.float32)
    v = x.copy()
    ss = np.ones(n, np.float32)
    for i in range(n):
        if norm[i]:
            ss[i] = np.sum(x[i] * x[i], dtype=np.float32)
            v[i] = x[i] * np.float32(1 / np.sqrt(ss[i] / np.float32(d) + np.float32(eps))) * g[i]
        if not raw[i]:
            a, b = v[i, 0::2].copy(), v[i, 1::2].copy()
            v[i, 0::2], v[i, 1::2] = a * cos - b * sin, a * sin + b * cos
    code, scale = np.zeros((n, d), np.uint8), np.zeros(n, np.uint16)
    raw, norm = np.asarray(raw, np.int32), np.asarray(norm, np.int32)
    together = rule.quantize_warp(d // 8, ptr(x), ptr(v), ptr(g), ptr(cos), ptr(sin), ptr(raw), ptr(norm), ptr(ss),
                                  ctypes.c_float(eps), ptr(code), ptr(scale))
    return code.astype(np.int32) - 8, (scale.astype(np.uint32) << 16).view(np.float32).astype(np.float64), bool(together)


@pytest.mark.parametrize("d,kinds", [(128, "kv"), (128, "vk"), (128, "qk"), (128, "kk"), (128, "vv"), (64, "kkvv"),
                                     (64, "qkvv"), (64, "kvkv"), (64, "qqkv"), (64, "kkkk")])
@pytest.mark.parametrize("gain", [True, False])
@pytest.mark.parametrize("size", [1e-17, 1.0, 1e17])
def test_warps_of_mixed_vectors(rule, d, kinds, gain, size):
    """size 1e-17 and 1e17: squares outside the fp32 rule's range send the normed
    vectors through 64 bits, beside others that take nothing of the kind."""
    rng = np.random.default_rng(d + len(kinds) + gain)
    n = len(kinds)
    x = (rng.standard_normal((n, d)) * size).astype(np.float32)
    g = (1 + 0.2 * rng.standard_normal((n, d))).astype(np.float32)
    ang = rng.uniform(0, 6, d // 2)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    raw = [k != "k" for k in kinds]
    norm = [gain and k == "k" for k in kinds]
    code, scale, together = quantized(rule, x, g, cos, sin, raw, norm)
    assert together, "some lanes called a shuffle that others did not"
    for i, k in enumerate(kinds):
        y = torch.from_numpy(x[i].astype(np.float64))[None, None]
        if k == "k":
            y = R.norm_rope(y, torch.from_numpy(g[i].astype(np.float64)) if gain else None,
                            torch.from_numpy(cos.astype(np.float64))[None], torch.from_numpy(sin.astype(np.float64))[None],
                            float(np.float32(1e-6)))
        q, s = R.quantize(y[0, 0])
        assert np.array_equal(code[i], q.numpy()) and scale[i] == s.item()
