"""Paged key/value operators (include/dualar_paged.h) on torch tensors.

Argument marshalling only: each function checks its tensors, allocates its
outputs, and calls one libdualar.so entry point on the current stream of the
tensors' device.  One step of a model's own loop:

    pool = kv_pool(n_pages, n_kv_head, head_dim, bits=4, n_layer=n_layer)
    cos, sin = rope_tables(n_pos, head_dim)
    plan = kv_plan(kv_len, n_new, page_refs, table, max_rows)          # once
    for layer in range(n_layer):
        kv = pool[:, layer]
        q = qk_norm_rope(qkv, kv, plan.pos, plan.slot, q_norm, k_norm, cos, sin)
        y = paged_attention(q, kv, table, plan.row_start, plan.new_len, window, sinks)

Nothing here synchronises, and a step can be captured into a CUDA graph.
Values on the device (lengths, pages, slots) are checked there: pass err (an
int32 tensor of one element, zeros) and read it with check_errors.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import numpy as np
import torch

from . import _lib as L

PAGE_TOKENS = 64
_ACT = {torch.float32: 0, torch.bfloat16: 1}
_raw_stream = torch._C._cuda_getCurrentRawStream


class KVPlan(NamedTuple):
    """Outputs of kv_plan, int32: row_start [n_seq + 1], pos and slot
    [max_rows], new_len [n_seq], status [3] (code, rows, pages)."""
    row_start: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor
    new_len: torch.Tensor
    status: torch.Tensor


def _bad(msg: str):
    raise L.DualARError(-1, msg)


def _raise(lib, rc: int):
    buf = ctypes.create_string_buffer(256)
    lib.dualar_paged_error(buf, 256)
    raise L.DualARError(rc, buf.value.decode())


# A step calls these functions once per layer, often faster than the GPU runs
# them: the checks below read as few tensor attributes as they can.
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def _not_i32(name: str, dev: int, n):
    _bad(f"{name}: a contiguous int32 tensor on cuda:{dev}" + ("" if n is None else f" with {n} elements") + " is needed")


def _i32(name: str, t: torch.Tensor, dev: int, n: int | None = None) -> int:
    """Address of a contiguous int32 tensor (of n elements) on device dev."""
    if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous() or (n is not None and t.numel() != n):
        _not_i32(name, dev, n)
    return t.data_ptr()


def _kv(kv: torch.Tensor) -> L.dualar_kv:
    """The C view of one layer of a pool (pool[:, layer])."""
    shape, st, ok = kv.shape, kv.stride(), False
    if kv.dtype is _BF16 and len(shape) == 5:
        n, two, h, pt, d = shape
        ok = two == 2 and pt == 64 and st[4] == 1 and st[3] == d and st[2] == 64 * d and st[1] == 64 * d * h
        bits, step, size = 16, st[0] * 2, 256 * d * h
    elif kv.dtype is torch.uint8 and len(shape) == 4:
        n, two, h, b = shape
        d = (b - 128) // 32
        ok = two == 2 and b == 32 * d + 128 and st[3] == 1 and st[2] == b and st[1] == b * h
        bits, step, size = 4, st[0], 2 * b * h
    if not ok or not kv.is_cuda:
        _bad(f"kv: {tuple(shape)} {kv.dtype} on {kv.device} is no layer of a pool (kv_pool(...)[:, layer])")
    # (a single page's stride says nothing)
    return L.dualar_kv(kv.data_ptr(), step if n > 1 else max(step, size), n, h, d, bits)


def _act(name: str, t: torch.Tensor, dev: int) -> int:
    a = _ACT.get(t.dtype)
    if a is None or t.get_device() != dev:
        _bad(f"{name}: float32 or bfloat16 on cuda:{dev} is needed, not {t.dtype} on {t.device}")
    return a


def _ld(stride: int, width: int, rows: int) -> int:
    """Row stride for the library, which refuses one below the width (rows that
    overlap, such as expanded ones); a single row's says nothing."""
    return stride if rows > 1 else width


def _out(out: torch.Tensor, like: torch.Tensor, dev: int, rows: int, h: int, d: int) -> int:
    """Row stride of a given output."""
    st = out.stride()
    if (out.dtype is not like.dtype or out.get_device() != dev or out.shape != (rows, h, d) or st[2] != 1 or
            st[1] != d):
        _bad(f"out: {like.dtype} {(rows, h, d)} on cuda:{dev} with contiguous rows is needed")
    return _ld(st[0], h * d, rows)


def _err(err, dev: int):
    return None if err is None else _i32("err", err, dev, 1)


_here = contextlib.nullcontext()
_current = torch._C._cuda_getDevice


def _on(dev: int):
    """Device dev made current (nothing to do where it is already)."""
    return _here if _current() == dev else torch.cuda.device(dev)


def kv_page_bytes(n_kv_head: int, head_dim: int, bits: int = 16) -> int:
    """Bytes of one layer of one page."""
    L.check_int32(n_kv_head=n_kv_head, head_dim=head_dim, bits=bits)
    n = L.lib().dualar_kv_page_bytes(n_kv_head, head_dim, bits)
    if n < 0:
        _bad(f"kv: {n_kv_head} heads of {head_dim} in {bits} bits (head_dim 64 or 128, bits 16 or 4)")
    return n


def kv_pool(n_pages: int, n_kv_head: int, head_dim: int, bits: int = 16, n_layer: int = 1,
            device="cuda") -> torch.Tensor:
    """An empty pool (zeros): bf16 [n_pages, n_layer, 2, n_kv_head, 64, head_dim]
    or, in 4 bits, uint8 [n_pages, n_layer, 2, n_kv_head, 32 head_dim + 128].
    pool[:, layer] is the kv argument of the operators."""
    block = kv_page_bytes(n_kv_head, head_dim, bits) // (2 * n_kv_head)
    if bits == 16:
        return torch.zeros((n_pages, n_layer, 2, n_kv_head, PAGE_TOKENS, head_dim), dtype=torch.bfloat16, device=device)
    return torch.zeros((n_pages, n_layer, 2, n_kv_head, block), dtype=torch.uint8, device=device)


def rope_tables(n_pos: int, head_dim: int, base: float = 1.0e6, device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 [n_pos, head_dim / 2] cos and sin, the decoder's tables: angles
    pos * base^(-2i/head_dim) and their cosines in float64, rounded to fp32,
    then to bf16."""
    ang = np.arange(n_pos, dtype=np.float64)[:, None] * np.power(
        float(base), -2.0 * np.arange(head_dim // 2, dtype=np.float64) / head_dim)
    return tuple(torch.from_numpy(f(ang).astype(np.float32)).to(torch.bfloat16).to(device) for f in (np.cos, np.sin))


def kv_plan(kv_len: torch.Tensor, n_new: torch.Tensor, page_refs: torch.Tensor, table: torch.Tensor,
            max_rows: int) -> KVPlan:
    """dualar_kv_plan: takes pages for n_new more tokens of each request (in
    place in page_refs [n_pages] and table [n_seq, width]) and lays out the
    step's rows."""
    dev = kv_len.get_device()
    if dev < 0 or kv_len.dim() != 1 or table.dim() != 2 or page_refs.dim() != 1 or not (
            0 <= max_rows <= 2 ** 24):
        _bad("kv_plan: kv_len is [n_seq] on a CUDA device, table [n_seq, width], page_refs [n_pages], max_rows in [0, 2^24]")
    n, (nt, width) = kv_len.shape[0], table.shape
    if nt != n:
        _bad(f"kv_plan: a table of {nt} rows for {n} requests")
    lens, new = _i32("kv_len", kv_len, dev), _i32("n_new", n_new, dev, n)
    tab, refs = _i32("table", table, dev), _i32("page_refs", page_refs, dev)
    lib = L.lib()
    with _on(dev):
        buf = torch.empty(2 * n + 4 + 2 * max_rows, dtype=_I32, device=kv_len.device)
        at = buf.data_ptr()
        rc = lib.dualar_kv_plan(lens, new, n, refs, page_refs.shape[0], tab, width, max_rows, at, at + 4 * (n + 1),
                                at + 4 * (n + 1 + max_rows), at + 4 * (n + 1 + 2 * max_rows),
                                at + 4 * (2 * n + 1 + 2 * max_rows), _raw_stream(dev))
    if rc:
        _raise(lib, rc)
    return KVPlan(*buf.split_with_sizes((n + 1, max_rows, max_rows, n, 3)))


def qk_norm_rope(qkv: torch.Tensor, kv: torch.Tensor, pos: torch.Tensor, slot: torch.Tensor,
                 q_norm: torch.Tensor | None, k_norm: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor,
                 eps: float = 1e-6, out: torch.Tensor | None = None, err: torch.Tensor | None = None) -> torch.Tensor:
    """dualar_qk_norm_rope: qkv [rows, (n_head + 2 n_kv_head) head_dim] ->
    queries [rows, n_head, head_dim], keys and values appended to kv."""
    c, dev, lib = _kv(kv), kv.get_device(), L.lib()
    d, hk = c.head_dim, c.n_kv_head
    rows, width = qkv.shape if qkv.dim() == 2 else (0, 1)
    h = width // d - 2 * hk
    ld, one = qkv.stride() if qkv.dim() == 2 else (0, 0)
    if width % d or h < 1 or one != 1:
        _bad(f"qk_norm_rope: qkv {tuple(qkv.shape)} is no matrix of contiguous rows of queries and 2 x {hk} heads of {d}")
    act = _act("qkv", qkv, dev)
    pp, ps = _i32("pos", pos, dev, rows), _i32("slot", slot, dev, rows)
    if q_norm is not None:
        if not (q_norm.dtype is _BF16 and q_norm.get_device() == dev and q_norm.numel() == d and q_norm.is_contiguous()):
            _bad(f"q_norm: bfloat16 [{d}] on cuda:{dev} is needed")
        q_norm = q_norm.data_ptr()
    if k_norm is not None:
        if not (k_norm.dtype is _BF16 and k_norm.get_device() == dev and k_norm.numel() == d and k_norm.is_contiguous()):
            _bad(f"k_norm: bfloat16 [{d}] on cuda:{dev} is needed")
        k_norm = k_norm.data_ptr()
    n_pos = cos.shape[0]
    if not (cos.dtype is _BF16 and sin.dtype is _BF16 and cos.get_device() == dev and sin.get_device() == dev and
            cos.numel() == n_pos * (d // 2) and sin.shape == cos.shape and cos.is_contiguous() and sin.is_contiguous()):
        _bad(f"cos, sin: contiguous bfloat16 [n_pos, {d // 2}] on cuda:{dev} are needed")
    with _on(dev):
        if out is None:
            out, ldo = torch.empty((rows, h, d), dtype=qkv.dtype, device=kv.device), h * d
        else:
            ldo = _out(out, qkv, dev, rows, h, d)
        rc = lib.dualar_qk_norm_rope(qkv.data_ptr(), act, _ld(ld, width, rows), rows, h, c, pp, ps, q_norm, k_norm, eps,
                                     cos.data_ptr(), sin.data_ptr(), n_pos, out.data_ptr(), ldo, _err(err, dev),
                                     _raw_stream(dev))
    if rc:
        _raise(lib, rc)
    return out


def kv_read(kv: torch.Tensor, slot: torch.Tensor, err: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """dualar_kv_read: keys and values of slots as float32 [n, n_kv_head, head_dim]."""
    c, dev, n, lib = _kv(kv), kv.get_device(), slot.numel(), L.lib()
    ps = _i32("slot", slot, dev)
    L.check_int32(slots=n)
    shape = (n, c.n_kv_head, c.head_dim)
    with _on(dev):
        k = torch.empty(shape, dtype=_F32, device=kv.device)
        v = torch.empty(shape, dtype=_F32, device=kv.device)
        rc = lib.dualar_kv_read(c, ps, n, k.data_ptr(), v.data_ptr(), _err(err, dev), _raw_stream(dev))
    if rc:
        _raise(lib, rc)
    return k, v


def paged_attention(q: torch.Tensor, kv: torch.Tensor, table: torch.Tensor, row_start: torch.Tensor,
                    kv_len: torch.Tensor, window: int = 0, sinks: int = 0, scale: float | None = None,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    err: torch.Tensor | None = None) -> torch.Tensor:
    """dualar_paged_attention: q [rows, n_head, head_dim] against the cached
    positions each row sees.  kv_len [n_seq] counts the new tokens (KVPlan.new_len);
    table [n_seq, width]; row_start [n_seq + 1].  window 0: every position up to
    the row's own; else the last `window` of them and the first `sinks`.  scale:
    head_dim^-0.5 by default.  Rows before the first request and behind the last are
    left as they are in `out` (undefined where it is allocated here).  workspace: by default one
    that the call allocates; a given one belongs to one call at a time."""
    c, dev, lib = _kv(kv), kv.get_device(), L.lib()
    d = c.head_dim
    rows, h, dq = q.shape if q.dim() == 3 else (0, 0, 0)
    st = q.stride()
    if dq != d or st[2] != 1 or st[1] != d:
        _bad(f"paged_attention: q {tuple(q.shape)}: [rows, n_head, {d}] with contiguous rows is needed")
    act = _act("q", q, dev)
    L.check_int32(window=window, sinks=sinks)
    if kv_len.dim() != 1 or table.dim() != 2:
        _bad("paged_attention: kv_len is [n_seq], table [n_seq, width]")
    n, (nt, width) = kv_len.shape[0], table.shape
    if nt != n:
        _bad(f"paged_attention: a table of {nt} rows for {n} requests")
    lens, tab = _i32("kv_len", kv_len, dev), _i32("table", table, dev)
    start = _i32("row_start", row_start, dev, n + 1)
    with _on(dev):
        if out is None:
            out, ldo = torch.empty((rows, h, d), dtype=q.dtype, device=kv.device), h * d
        else:
            ldo = _out(out, q, dev, rows, h, d)
        if workspace is None:
            size = lib.dualar_paged_attention_workspace(act, rows, h, c, n)
            # this call's own: a call queues two kernels, and another thread's may come
            # between them on the same stream (the allocator reuses it in stream order)
            workspace = torch.empty(max(size, 0), dtype=torch.uint8, device=kv.device)
            ws = workspace.data_ptr()
        else:
            if workspace.get_device() != dev or not workspace.is_contiguous():
                _bad(f"workspace: a contiguous tensor on cuda:{dev} is needed")
            size, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
        rc = lib.dualar_paged_attention(q.data_ptr(), act, _ld(st[0], h * d, rows), rows, h, c, tab, width, start, lens, n,
                                        window, sinks, d ** -0.5 if scale is None else scale, out.data_ptr(), ldo, ws, size,
                                        _err(err, dev), _raw_stream(dev))
    if rc:
        _raise(lib, rc)
    return out


def paged_attention_workspace(q: torch.Tensor, kv: torch.Tensor, n_seq: int) -> int:
    """Bytes of the workspace argument of paged_attention for these sizes (a
    caller that captures graphs keeps one per graph that may run beside others)."""
    need = L.lib().dualar_paged_attention_workspace(_act("q", q, kv.get_device()), q.shape[0], q.shape[1], _kv(kv), n_seq)
    if need < 0:
        _bad(f"paged_attention: q {tuple(q.shape)} over kv {tuple(kv.shape)}, {n_seq} requests")
    return need


def check_errors(err: torch.Tensor) -> None:
    """Synchronises with err's device (the calls that report into err may be queued
    on any stream), raises DualARError (DUALAR_ERR_DEVICE) if a bounds check failed
    there or a wait ran out, and clears it."""
    if err.is_cuda:
        torch.cuda.synchronize(err.device)
    word = int(err.item())
    if word:
        err.zero_()
        what = [s for b, s in ((1, "a wait inside a kernel that ran out"),
                               (4, "a row, slot, position or length out of range"), (8, "a page out of range"))
                if word & b]
        raise L.DualARError(-7, " and ".join(what) or f"error word 0x{word:x}")
