"""PyTorch-facing calls with the same names as the C ABI.

Argument marshalling only: shapes are read from the tensors, output and
workspace tensors are allocated with torch, and the call goes through the C
library on the tensors' current CUDA stream. Every step of the attention runs
in the library's kernels.
"""

from __future__ import annotations

import ctypes
import math

import torch

from ._lib import (
    FA_DTYPE_BF16,
    FA_DTYPE_F32,
    FA_ERR_UNSUPPORTED,
    FA_PLAN_MAX_T,
    FA_ROPE_SCALINGS,
    FA_TREE_MASK_MAX_B,
    FA_TREE_MASK_MAX_T,
    FAError,
    check,
    fast,
    lib,
)


def _ptr(t: torch.Tensor | None):
    # the C signatures declare c_void_p: a plain int address (or None for NULL) is passed as is
    return None if t is None else t.data_ptr()


# the current stream's raw handle, without building a torch Stream object per call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")


def _on_current_device(t: torch.Tensor):
    """The library launches on the current CUDA device; tensors elsewhere would be read
    through another device's pointers."""
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device)")


def _check_qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    """q [B][Hq][T][d], k and v [B][Hkv][S][d] on one device, the current one. The
    library takes every size from q and k, so v must match k exactly and q must share
    B and d."""
    if not (q.device == k.device == v.device):
        raise ValueError("q, k and v must be on one device")
    _on_current_device(q)
    if tuple(k.shape) != tuple(v.shape):
        raise ValueError(f"k and v must have one shape, got {tuple(k.shape)} and {tuple(v.shape)}")
    if q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must share batch and head dimension")


def _out(t, name: str, shape, dtype, like: torch.Tensor) -> torch.Tensor:
    """A caller's output tensor, checked (the library writes it through a bare pointer,
    so a smaller or strided tensor would be written past its end), or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if not isinstance(t, torch.Tensor) or t.device != like.device:
        raise ValueError(f"{name} must be a tensor on {like.device}")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t


def fa_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, want_lse: bool = True):
    """Prefill forward: q [B][Hq][T][d], k, v [B][Hkv][S][d] bf16 -> (o bf16, lse fp32 or None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    _check_qkv(q, k, v)
    B, Hq, T, d = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, "out", q.shape, torch.bfloat16, q)
    if want_lse or lse is not None:
        lse = _out(lse, "lse", (B, Hq, T), torch.float32, q)
    st = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, S, d, scale, int(causal), _stream(q))
    check(st, "fa_fwd")
    return o, lse


def fa_fwd_f32(q, k, v, causal: bool = False, scale: float | None = None):
    """The same forward in fp32 on the CUDA cores: fp32 q, k, v -> (o fp32, lse fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.float32, 4)
    _check_qkv(q, k, v)
    B, Hq, T, d = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    st = lib().fa_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, S, d, scale, int(causal), _stream(q))
    check(st, "fa_fwd_f32")
    return o, lse


def _ws_bytes(workspace, nbytes: int, device) -> int:
    """Size in bytes of a caller's workspace tensor (any dtype), checked against what the call needs."""
    if workspace.device != torch.device(device) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    size = workspace.numel() * workspace.element_size()
    if size < nbytes:
        raise ValueError(f"workspace needs {nbytes} bytes, got {size}")
    return size


def fa_bwd_workspace_bytes(B: int, Hq: int, T: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, Hq, T))


def fa_bwd(q, k, v, o, lse, d_o, causal: bool = False, scale: float | None = None, workspace=None,
           dq=None, dk=None, dv=None):
    """Backward: q, o, d_o [B][Hq][T][d], k, v [B][Hkv][S][d] bf16, lse [B][Hq][T] fp32
    (the forward's) -> (dq, dk, dv) bf16."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (d_o, "d_o")):
        _need(t, n, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    _check_qkv(q, k, v)
    B, Hq, T, d = q.shape
    for t, n in ((o, "o"), (d_o, "d_o")):
        if t.device != q.device or tuple(t.shape) != tuple(q.shape):
            raise ValueError(f"{n} must have q's shape {tuple(q.shape)} on its device")
    if lse.device != q.device or tuple(lse.shape) != (B, Hq, T):
        raise ValueError(f"lse must be [B][Hq][T] = {(B, Hq, T)} on q's device")
    Hkv, S = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = fa_bwd_workspace_bytes(B, Hq, T)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    ws_bytes = _ws_bytes(workspace, nbytes, q.device)
    dq = _out(dq, "dq", q.shape, torch.bfloat16, q)
    dk = _out(dk, "dk", k.shape, torch.bfloat16, q)
    dv = _out(dv, "dv", v.shape, torch.bfloat16, q)
    st = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dk), _ptr(dv), B, Hq,
                      Hkv, T, S, d, scale, int(causal), _ptr(workspace), ws_bytes, _stream(q))
    check(st, "fa_bwd")
    return dq, dk, dv


def fa_fwd_kv_outer_workspace_bytes(B: int, Hq: int, T: int, d: int) -> int:
    return int(lib().fa_fwd_kv_outer_workspace_bytes(B, Hq, T, d))


def fa_fwd_kv_outer(q, k, v, causal: bool = False, scale: float | None = None, row_bands: int = 1, workspace=None,
                    out=None, lse=None):
    """The forward in the FlashAttention-1 loop order (key tiles outer, running
    state through HBM): q [B][Hq][T][d], k, v [B][Hkv][S][d] bf16 -> (o, lse)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    _check_qkv(q, k, v)
    B, Hq, T, d = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = fa_fwd_kv_outer_workspace_bytes(B, Hq, T, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    ws_bytes = _ws_bytes(workspace, nbytes, q.device)
    o = _out(out, "out", q.shape, torch.bfloat16, q)
    lse = _out(lse, "lse", (B, Hq, T), torch.float32, q)
    st = lib().fa_fwd_kv_outer(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, S, d, scale,
                               int(causal), int(row_bands), _ptr(workspace), ws_bytes, _stream(q))
    check(st, "fa_fwd_kv_outer")
    return o, lse


def fa_num_splits_heuristic(B: int, Hkv: int, S: int, num_sms: int) -> int:
    return int(lib().fa_num_splits_heuristic(B, Hkv, S, num_sms))


def fa_decode_workspace_bytes(B: int, Hq: int, T: int, d: int, num_splits: int) -> int:
    return int(lib().fa_decode_workspace_bytes(B, Hq, T, d, num_splits))


def fa_num_splits_prefill(B: int, Hq: int, Hkv: int, T: int, S: int, num_sms: int) -> int:
    return int(lib().fa_num_splits_prefill(B, Hq, Hkv, T, S, num_sms))


def fa_decode_num_splits(B: int, Hq: int, Hkv: int, T: int, S: int, paged: bool = False,
                         num_sms: int | None = None, device=None) -> int:
    """The split count the decode calls take for num_splits = 0 (chosen by the C library)."""
    if num_sms is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        num_sms = torch.cuda.get_device_properties(dev).multi_processor_count
    return int(lib().fa_decode_num_splits(B, Hq, Hkv, T, S, int(paged), int(num_sms)))


def _workspace(B, Hq, T, d, n, device, workspace):
    nbytes = fa_decode_workspace_bytes(B, Hq, T, d, n)
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace, _ws_bytes(workspace, nbytes, device)


def fa_decode_splitkv(q, k, v, causal: bool = True, num_splits: int = 0, scale: float | None = None,
                      workspace=None, out=None, lse=None):
    """Split-KV decode: q [B][Hq][T][d], k, v [B][Hkv][S][d] bf16 -> (o, lse)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    _check_qkv(q, k, v)
    B, Hq, T, d = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    # the workspace is sized for the count the library takes; num_splits passes through as given
    n = int(num_splits) or fa_decode_num_splits(B, Hq, Hkv, T, S, False, device=q.device)
    ws, ws_bytes = _workspace(B, Hq, T, d, n, q.device, workspace)
    o = _out(out, "out", q.shape, torch.bfloat16, q)
    lse = _out(lse, "lse", (B, Hq, T), torch.float32, q)
    st = lib().fa_decode_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, S, d, scale,
                                 int(causal), int(num_splits), _ptr(ws), ws_bytes, _stream(q))
    check(st, "fa_decode_splitkv")
    return o, lse


def fa_decode_splitkv_static(q, k, v, causal: bool = True, num_splits: int = 0, scale: float | None = None,
                             out=None, lse=None):
    """Split-KV decode with the partials in the library's fixed 4 MiB device array
    (no workspace, no allocation inside the call); see include/fa_gb300.h."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    _check_qkv(q, k, v)
    B, Hq, T, d = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = _out(out, "out", q.shape, torch.bfloat16, q)
    lse = _out(lse, "lse", (B, Hq, T), torch.float32, q)
    st = lib().fa_decode_splitkv_static(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, T, S, d, scale,
                                        int(causal), int(num_splits), _stream(q))
    check(st, "fa_decode_splitkv_static")
    return o, lse


def fa_lse_merge(o_part, lse_part):
    """Merge o_part [n][rows][d] fp32 and lse_part [n][rows] fp32 -> (o [rows][d] bf16, lse [rows] fp32)."""
    _need(o_part, "o_part", torch.float32, 3)
    _need(lse_part, "lse_part", torch.float32, 2)
    n, rows, d = o_part.shape
    if tuple(lse_part.shape) != (n, rows) or lse_part.device != o_part.device:
        raise ValueError("lse_part must be [n][rows] on o_part's device")
    _on_current_device(o_part)
    o = torch.empty((rows, d), dtype=torch.bfloat16, device=o_part.device)
    lse = torch.empty((rows,), dtype=torch.float32, device=o_part.device)
    st = lib().fa_lse_merge(_ptr(o_part), _ptr(lse_part), _ptr(o), _ptr(lse), n, rows, d, _stream(o_part))
    check(st, "fa_lse_merge")
    return o, lse


def fa_decode_paged(q, k_pages, v_pages, block_table, seqlens, causal: bool = True, num_splits: int = 0,
                    scale: float | None = None, workspace=None, out=None, lse=None):
    """Paged decode: pools [P][16][Hkv][d] bf16, block_table [B][max_pages] int32, seqlens [B] int32."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k_pages, "k_pages", torch.bfloat16, 4)
    _need(v_pages, "v_pages", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seqlens, "seqlens", torch.int32, 1)
    B, Hq, T, d = q.shape
    P, page_size, Hkv, _ = k_pages.shape
    max_pages = block_table.shape[1]
    if not (q.device == k_pages.device == v_pages.device == block_table.device == seqlens.device):
        raise ValueError("q, the pools, block_table and seqlens must be on one device")
    _on_current_device(q)
    if tuple(k_pages.shape) != tuple(v_pages.shape) or k_pages.shape[3] != d:
        raise ValueError(f"k_pages and v_pages must both be [P][page_size][Hkv][{d}]")
    if block_table.shape[0] != B or tuple(seqlens.shape) != (B,):
        raise ValueError(f"block_table must be [{B}][max_pages] and seqlens [{B}]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    n = int(num_splits) or fa_decode_num_splits(B, Hq, Hkv, T, max_pages * page_size, True, device=q.device)
    ws, ws_bytes = _workspace(B, Hq, T, d, n, q.device, workspace)
    o = _out(out, "out", q.shape, torch.bfloat16, q)
    lse = _out(lse, "lse", (B, Hq, T), torch.float32, q)
    st = lib().fa_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seqlens), _ptr(o),
                               _ptr(lse), B, Hq, Hkv, T, max_pages, page_size, P, d, scale, int(causal),
                               int(num_splits), _ptr(ws), ws_bytes, _stream(q))
    check(st, "fa_decode_paged")
    return o, lse


# What follows is called between the layers of a decode step, where a microsecond of the
# host counts. A call goes through the extension module first (fast(): the same tests,
# outputs and library call, in one step; the plan and the attention calls without given
# outputs only); it answers None where an argument is not plainly right, and the checks
# below then name it.
_BF16, _I32, _F64 = torch.bfloat16, torch.int32, torch.float64


def _answer(got, name: str):
    if type(got) is int:
        check(got, name)
    return got


def _need_ints(name: str, t: torch.Tensor, shape, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or tuple(t.shape) != tuple(shape) \
            or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")


def fa_paged_plan(cached_lens, new_lens, free_pages, block_table, T: int, align_end: bool = False, seqlens=None,
                  slots=None, positions=None, pages_used=None):
    """Block tables, slot maps and positions of a step: cached_lens, new_lens [B], free_pages [F],
    block_table [B][max_pages] (extended in place), all int32 on one device
    -> (seqlens [B], slots [B][T], positions [B][T], pages_used [1]), new ones in one allocation."""
    if seqlens is None and slots is None and positions is None and pages_used is None:
        got = fast().paged_plan(cached_lens, new_lens, free_pages, block_table, T, align_end)
        if got is not None:
            return _answer(got, "fa_paged_plan")
    _need(block_table, "block_table", _I32, 2)
    _need(free_pages, "free_pages", _I32, 1)
    B, max_pages = block_table.shape
    dev = block_table.device
    _need_ints("cached_lens", cached_lens, (B,), dev)
    _need_ints("new_lens", new_lens, (B,), dev)
    if free_pages.device != dev:
        raise ValueError(f"free_pages must be on {dev}")
    _on_current_device(block_table)
    T = int(T)
    if T < 1:
        raise ValueError(f"T must be at least 1, got {T}")
    if T > FA_PLAN_MAX_T or B * T >= 2**31:  # before outputs of that size are made
        check(FA_ERR_UNSUPPORTED, "fa_paged_plan")
    seqlens = _out(seqlens, "seqlens", (B,), _I32, block_table)
    slots = _out(slots, "slots", (B, T), _I32, block_table)
    positions = _out(positions, "positions", (B, T), _I32, block_table)
    pages_used = _out(pages_used, "pages_used", (1,), _I32, block_table)
    st = lib().fa_paged_plan(_ptr(cached_lens), _ptr(new_lens), _ptr(free_pages), free_pages.shape[0],
                             _ptr(block_table), _ptr(seqlens), _ptr(slots), _ptr(positions), _ptr(pages_used), B, T,
                             max_pages, 16, int(align_end), _stream(block_table))
    check(st, "fa_paged_plan")
    return seqlens, slots, positions, pages_used


def fa_tree_mask(parents, seqlens, tree_lens=None, mask=None, positions=None):
    """Visibility mask and positions of drafted trees: parents [B][T], seqlens [B], tree_lens [B] or
    None (T nodes each), int32 -> (mask [B][T][ceil(T/32)] int32, positions [B][T] int32), new ones in
    one allocation."""
    if mask is None and positions is None:
        got = fast().tree_mask(parents, seqlens, tree_lens)
        if got is not None:
            return _answer(got, "fa_tree_mask")
    _need(parents, "parents", _I32, 2)
    B, T = parents.shape
    _need_ints("seqlens", seqlens, (B,), parents.device)
    if tree_lens is not None:
        _need_ints("tree_lens", tree_lens, (B,), parents.device)
    _on_current_device(parents)
    if B > FA_TREE_MASK_MAX_B or T > FA_TREE_MASK_MAX_T:
        check(FA_ERR_UNSUPPORTED, "fa_tree_mask")
    mask = _out(mask, "mask", (B, T, (T + 31) // 32), _I32, parents)
    positions = _out(positions, "positions", (B, T), _I32, parents)
    st = lib().fa_tree_mask(_ptr(parents), _ptr(seqlens), _ptr(tree_lens), _ptr(mask), _ptr(positions), B, T,
                            _stream(parents))
    check(st, "fa_tree_mask")
    return mask, positions


def fa_rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Angles per position of rot_dim / 2 rotary pairs, stretched for long contexts by scaling in
    {"none", "linear", "ntk", "yarn"} -> (inv_freq fp64 on device, mscale)."""
    if scaling not in FA_ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(FA_ROPE_SCALINGS)}, got {scaling!r}")
    rot_dim = int(rot_dim)
    host = torch.empty(max(rot_dim, 0) // 2, dtype=_F64)
    mscale = ctypes.c_float(1.0)
    st = lib().fa_rope_inv_freq(_ptr(host), ctypes.byref(mscale), rot_dim, float(base), FA_ROPE_SCALINGS[scaling],
                                float(factor), float(original_len), float(beta_fast), float(beta_slow))
    check(st, "fa_rope_inv_freq")
    return host.to(device), mscale.value


_ROPE_DTYPES = {torch.bfloat16: FA_DTYPE_BF16, torch.float32: FA_DTYPE_F32}
_Strides = ctypes.c_longlong * 12  # host memory of the C call's strides


def _need_rows(t, name: str, dtype, device, shape=None):
    """A [B][heads][T][d] operand whose rows of d are dense; the strides between rows are free."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or t.dim() != 4 or t.device != device or t.stride(3) != 1:
        raise ValueError(f"{name} must be a 4-D {dtype} tensor on {device} whose last stride is 1")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows_out(t, name: str, like: torch.Tensor):
    """A caller's output of like's shape, no two of its rows on one another, or a new dense one."""
    if t is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _need_rows(t, name, like.dtype, like.device, like.shape)
    if not t.is_contiguous():
        reach = t.shape[3]  # values up to the end of the rows of the dimensions so far
        for stride, size in sorted((st, n) for st, n in zip(t.stride()[:3], t.shape[:3]) if n > 1):
            if stride < reach:
                raise ValueError(f"{name} has rows that overlap (shape {tuple(t.shape)}, strides {t.stride()})")
            reach += stride * (size - 1)
    return t


def _need_angles(positions, inv_freq, B: int, T: int, device, shared_ok: bool) -> bool:
    if not isinstance(positions, torch.Tensor) or positions.dtype != _I32 or positions.device != device \
            or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int32 tensor on {device}")
    shape = tuple(positions.shape)
    if shape != (B, T) and not (shared_ok and shape == (T,)):
        raise ValueError(f"positions must be [{B}][{T}]{f' or [{T}]' if shared_ok else ''}, got {shape}")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != _F64 or inv_freq.device != device \
            or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous 1-D float64 tensor on {device} (fa_rope_inv_freq)")
    return len(shape) == 1


def _rope(name: str, q, k, positions, inv_freq, interleaved, mscale, q_out, k_out):
    got = fast().rope(q, k, positions, inv_freq, interleaved, mscale, name == "fa_rope_bwd", q_out, k_out)
    if got is not None:
        return _answer(got, name)
    if not isinstance(q, torch.Tensor) or q.dtype not in _ROPE_DTYPES:
        raise ValueError(f"{name}: q must be a bfloat16 or float32 tensor")
    dev = q.device
    _need_rows(q, "q", q.dtype, dev)
    _on_current_device(q)
    B, Hq, T, d = q.shape
    shared = _need_angles(positions, inv_freq, B, T, dev, True)
    q_out = _rows_out(q_out, "q_out", q)
    Hk, sk, sko = 0, (0, 0, 0), (0, 0, 0)
    if k is not None:
        _need_rows(k, "k", q.dtype, dev)
        Hk = k.shape[1]
        if k.shape[0] != B or k.shape[2] != T or k.shape[3] != d:
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must share batch, length and head dimension")
        k_out = _rows_out(k_out, "k_out", k)
        sk, sko = k.stride()[:3], k_out.stride()[:3]
    elif k_out is not None:
        raise ValueError("k_out without k")
    strides = _Strides(*q.stride()[:3], *q_out.stride()[:3], *sk, *sko)
    st = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), strides, _ptr(positions), int(shared),
                              _ptr(inv_freq), B, Hq, Hk, T, d, 2 * inv_freq.shape[0], int(interleaved), float(mscale),
                              _ROPE_DTYPES[q.dtype], _stream(q))
    check(st, name)
    return q_out, k_out


def fa_rope(q, k, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, q_out=None, k_out=None):
    """Rotary positions of q [B][Hq][T][d] and k [B][Hk][T][d] (or None), bf16 or fp32, any strides
    between rows; positions [B][T] or [T] int32, inv_freq [rot/2] fp64 -> (q_out, k_out). Outputs are
    dense [B][H][T][d] unless given; they may be q and k themselves."""
    return _rope("fa_rope", q, k, positions, inv_freq, interleaved, mscale, q_out, k_out)


def fa_rope_bwd(dq_out, dk_out, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, q_out=None,
                k_out=None):
    """Gradients of fa_rope: those of its outputs -> (dq, dk), into q_out and k_out where given."""
    return _rope("fa_rope_bwd", dq_out, dk_out, positions, inv_freq, interleaved, mscale, q_out, k_out)


def fa_rope_append_paged(q, k, v, positions, slots, inv_freq, k_pages, v_pages, interleaved: bool = False,
                         mscale: float = 1.0, q_out=None):
    """New rows of a step over the paged cache: q [B][Hq][T][d] rotated -> q_out; k [B][Hkv][T][d] rotated
    and v written to rows slots [B][T] of the pools [P][16][Hkv][d] (-1: not written). bf16."""
    got = fast().rope_append_paged(q, k, v, positions, slots, inv_freq, k_pages, v_pages, interleaved, mscale, q_out)
    if got is not None:
        return _answer(got, "fa_rope_append_paged")
    if not isinstance(q, torch.Tensor):
        raise ValueError("q must be a CUDA tensor")
    dev = q.device
    _need_rows(q, "q", _BF16, dev)
    B, Hq, T, d = q.shape
    _need(k_pages, "k_pages", _BF16, 4)
    _need(v_pages, "v_pages", _BF16, 4)
    P, page_size, Hkv, _ = k_pages.shape
    if tuple(v_pages.shape) != tuple(k_pages.shape) or k_pages.shape[3] != d or k_pages.device != dev \
            or v_pages.device != dev:
        raise ValueError(f"k_pages and v_pages must both be [P][page_size][Hkv][{d}] on {dev}")
    _need_rows(k, "k", _BF16, dev, (B, Hkv, T, d))
    _need_rows(v, "v", _BF16, dev, (B, Hkv, T, d))
    _on_current_device(q)
    _need_angles(positions, inv_freq, B, T, dev, False)
    _need_ints("slots", slots, (B, T), dev)
    q_out = _rows_out(q_out, "q_out", q)
    strides = _Strides(*q.stride()[:3], *q_out.stride()[:3], *k.stride()[:3], *v.stride()[:3])
    st = lib().fa_rope_append_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(q_out), strides, _ptr(positions), _ptr(slots),
                                    _ptr(inv_freq), _ptr(k_pages), _ptr(v_pages), B, Hq, Hkv, T, page_size, P, d,
                                    2 * inv_freq.shape[0], int(interleaved), float(mscale), _stream(q))
    check(st, "fa_rope_append_paged")
    return q_out


def fa_tree_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, max_pages: int, d: int,
                            num_sms: int | None = None, device=None) -> int:
    """Bytes of workspace fa_tree_decode_paged needs on a device with num_sms SMs (None: this one), for this shape: a
    smaller batch or a narrower table may need more. num_sms * (2 * rows * (4 * d + 16) + 16) holds for every batch and
    table, rows = 128 where Hq / Hkv * T <= 128, else 256."""
    if num_sms is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        num_sms = torch.cuda.get_device_properties(dev).multi_processor_count
    return int(lib().fa_tree_workspace_bytes(B, Hq, Hkv, T, max_pages, d, int(num_sms)))


def fa_tree_decode_paged(q, k_pages, v_pages, block_table, seqlens, tree_mask, tree_lens=None,
                         scale: float | None = None, workspace=None, out=None, lse=None):
    """Attention of drafted trees over the paged cache: q [B][Hq][T][d], pools [P][16][Hkv][d] bf16,
    block_table [B][max_pages], seqlens [B], tree_mask [B][T][ceil(T/32)] or [T][ceil(T/32)] (one for
    all), tree_lens [B] or None (T nodes each), int32 -> (o, lse)."""
    if workspace is None and out is None and lse is None:
        got = fast().tree_decode_paged(q, k_pages, v_pages, block_table, seqlens, tree_mask, tree_lens, scale)
        if got is not None:
            return _answer(got, "fa_tree_decode_paged")
    _need(q, "q", _BF16, 4)
    _need(k_pages, "k_pages", _BF16, 4)
    _need(v_pages, "v_pages", _BF16, 4)
    _need(block_table, "block_table", _I32, 2)
    B, Hq, T, d = q.shape
    P, page_size, Hkv, _ = k_pages.shape
    max_pages = block_table.shape[1]
    dev = q.device
    if not (dev == k_pages.device == v_pages.device == block_table.device):
        raise ValueError("q, the pools and block_table must be on one device")
    _on_current_device(q)
    if tuple(k_pages.shape) != tuple(v_pages.shape) or k_pages.shape[3] != d:
        raise ValueError(f"k_pages and v_pages must both be [P][page_size][Hkv][{d}]")
    if block_table.shape[0] != B:
        raise ValueError(f"block_table must be [{B}][max_pages]")
    _need_ints("seqlens", seqlens, (B,), dev)
    words = (T + 31) // 32
    shared = isinstance(tree_mask, torch.Tensor) and tree_mask.dim() == 2
    _need_ints("tree_mask", tree_mask, (T, words) if shared else (B, T, words), dev)
    if tree_lens is not None:
        _need_ints("tree_lens", tree_lens, (B,), dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    nbytes = fa_tree_workspace_bytes(B, Hq, Hkv, T, max_pages, d, device=dev)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws_bytes = _ws_bytes(workspace, nbytes, dev)
    o = _out(out, "out", q.shape, _BF16, q)
    lse = _out(lse, "lse", (B, Hq, T), torch.float32, q)
    st = lib().fa_tree_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seqlens),
                                    _ptr(tree_mask), int(shared), _ptr(tree_lens), _ptr(o), _ptr(lse), B, Hq, Hkv, T,
                                    max_pages, page_size, P, d, scale, _ptr(workspace), ws_bytes, _stream(q))
    check(st, "fa_tree_decode_paged")
    return o, lse


def fa_get_last_device_error(device=None) -> tuple[int, int]:
    """Synchronise the current stream and read/clear the device error word -> (status, raw word)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    detail = ctypes.c_int(0)
    st = lib().fa_get_last_device_error(ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def fa_set_wait_timeout_ns(ns: int) -> None:
    lib().fa_set_wait_timeout_ns(int(ns))


def fa_get_wait_timeouts() -> tuple[int, int]:
    """(bound of the waits between roles, bound of the waits before a CTA exits), in ns."""
    w, u = ctypes.c_ulonglong(0), ctypes.c_ulonglong(0)
    lib().fa_get_wait_timeouts(ctypes.byref(w), ctypes.byref(u))
    return int(w.value), int(u.value)


def fa_selftest_wait_timeout(timeout_ns: int, device=None) -> None:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = lib().fa_selftest_wait_timeout(int(timeout_ns), ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream))
    check(st, "fa_selftest_wait_timeout")


__all__ = [
    "FAError",
    "fa_fwd",
    "fa_fwd_f32",
    "fa_bwd",
    "fa_bwd_workspace_bytes",
    "fa_num_splits_heuristic",
    "fa_num_splits_prefill",
    "fa_decode_num_splits",
    "fa_decode_workspace_bytes",
    "fa_decode_splitkv",
    "fa_decode_splitkv_static",
    "fa_lse_merge",
    "fa_decode_paged",
    "fa_paged_plan",
    "fa_tree_mask",
    "fa_rope_inv_freq",
    "fa_rope",
    "fa_rope_bwd",
    "fa_rope_append_paged",
    "fa_tree_decode_paged",
    "fa_tree_workspace_bytes",
    "fa_get_last_device_error",
    "fa_set_wait_timeout_ns",
    "fa_get_wait_timeouts",
    "fa_selftest_wait_timeout",
]
