"""Python binding of the C ABI (include/mla.h), same names, torch tensors in.

Only argument marshalling happens here: shapes, dtypes and devices are
checked, raw pointers and the current CUDA stream are passed to libmla, and a
non-zero status raises :class:`MlaError`.  Every step of the path runs in the
library's CUDA kernels.
"""
from __future__ import annotations

import ctypes as C
import operator
from dataclasses import dataclass, field, replace
from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import lib, mla_plan_info, mla_window_info

H, D_HC, D_C, D_R, PAGE = 128, 128, 512, 64, 64
D_QK = D_C + D_R

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_MISALIGNED", 3: "MLA_ERR_UNSUPPORTED",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_DEVICE", 6: "MLA_ERR_TIMEOUT", 7: "MLA_ERR_NO_SPACE"}
DEVERR_PAGE_OOB, DEVERR_SLOT_OOB, DEVERR_TIMEOUT, DEVERR_PLAN, DEVERR_POS_OOB, DEVERR_FP8_RANGE = 1, 2, 4, 8, 16, 32
DEVERR_BATCH = 64


class MlaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def _check(status: int) -> None:
    if status != 0:
        raise MlaError(status, lib().mla_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, shape=None, cuda: bool = True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


_Tensor = torch.Tensor


def _raw_stream(dev: int) -> int:
    # looked up at a call: a PyTorch without CUDA lacks the name, and the host-only calls serve there too
    return torch._C._cuda_getCurrentRawStream(dev)


def _in(t, name: str, dtype, shape, dev: int) -> int:
    """A device argument's address: what _need checks, and that the tensor lives
    on the current device `dev` (the one the call launches on)."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        _need(t, name, dtype, shape)
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    return t.data_ptr()


def _on(stream, dev: int) -> int:
    """The raw handle of `stream`, or of the current stream of device `dev`."""
    return _raw_stream(dev) if stream is None else stream.cuda_stream


# ------------------------------------------------------------------ host-only calls
def mla_version() -> int:
    return int(lib().mla_version())


def mla_config_default():
    return lib().mla_config_default()


def mla_kv_bytes(layers: int, dc: int, dr: int, elem_bytes: int, tokens: int, seqs: int = 1) -> int:
    out = C.c_uint64()
    _check(lib().mla_kv_bytes(layers, dc, dr, elem_bytes, tokens, seqs, C.byref(out)))
    return int(out.value)


class MlaPool:
    """Host page pool (mla_pool_*)."""

    def __init__(self, num_pages: int):
        self._h = C.c_void_p()
        _check(lib().mla_pool_create(int(num_pages), C.byref(self._h)))

    def alloc(self, n: int) -> np.ndarray:
        ids = np.zeros(max(n, 1), dtype=np.int32)
        _check(lib().mla_pool_alloc(self._h, int(n), ids.ctypes.data_as(C.POINTER(C.c_int32))))
        return ids[:n]

    def free(self, ids) -> None:
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        _check(lib().mla_pool_free(self._h, ids.ctypes.data_as(C.POINTER(C.c_int32)), int(ids.size)))

    def available(self) -> int:
        out = C.c_int32()
        _check(lib().mla_pool_available(self._h, C.byref(out)))
        return int(out.value)

    def close(self) -> None:
        if self._h:
            lib().mla_pool_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mla_slot_mapping(block_table: np.ndarray, seq_ids: np.ndarray, positions: np.ndarray) -> np.ndarray:
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    sid = np.ascontiguousarray(seq_ids, dtype=np.int32)
    pos = np.ascontiguousarray(positions, dtype=np.int32)
    n = int(sid.size)
    out = np.zeros(max(n, 1), dtype=np.int64)
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_slot_mapping(bt.ctypes.data_as(P32), int(bt.shape[0]), int(bt.shape[1]),
                                  sid.ctypes.data_as(P32), pos.ctypes.data_as(P32), n,
                                  out.ctypes.data_as(C.POINTER(C.c_int64))))
    return out[:n]


# ------------------------------------------------------------------ device steps
def mla_cache_init(kv_cache: torch.Tensor, stream=None) -> None:
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _check(lib().mla_cache_init(_ptr(kv_cache), kv_cache.shape[0], _stream(stream)))


def mla_kv_append(c_kv_new, k_r_new, slots, kv_cache, dev_err, stream=None) -> None:
    n = c_kv_new.shape[0]
    _need(c_kv_new, "c_kv_new", torch.bfloat16, (n, D_C))
    _need(k_r_new, "k_r_new", torch.bfloat16, (n, D_R))
    _need(slots, "slots", torch.int64, (n,))
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_kv_append(_ptr(c_kv_new), _ptr(k_r_new), _ptr(slots), int(n), _ptr(kv_cache),
                               kv_cache.shape[0], _ptr(dev_err), _stream(stream)))


FP8_ROW_BYTES = 640


def mla_kv_append_fp8(c_kv_new, k_r_new, slots, rows, scales, dev_err, stream=None) -> None:
    """Quantise new tokens into the FP8 cache: rows uint8 [pages, 64, 640], scales fp32 [pages, 64]."""
    n = c_kv_new.shape[0]
    _need(c_kv_new, "c_kv_new", torch.bfloat16, (n, D_C))
    _need(k_r_new, "k_r_new", torch.bfloat16, (n, D_R))
    _need(slots, "slots", torch.int64, (n,))
    _need(rows, "rows", torch.uint8, (rows.shape[0], PAGE, FP8_ROW_BYTES))
    _need(scales, "scales", torch.float32, (rows.shape[0], PAGE))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_kv_append_fp8(_ptr(c_kv_new), _ptr(k_r_new), _ptr(slots), int(n), _ptr(rows), _ptr(scales),
                                   rows.shape[0], _ptr(dev_err), _stream(stream)))


def mla_kv_append_rope_fp8(c_kv_new, k_pe_new, positions, table, slots, rows, scales, dev_err, q_pe=None, q_r=None,
                           stream=None) -> None:
    """Append to the FP8 cache with the RoPE key rotated on the way in; with
    q_pe (bf16 [n, 128, 64], the same tokens' queries) also rotate them into q_r."""
    dev = torch.cuda.current_device()
    n, pages, max_pos = c_kv_new.shape[0], rows.shape[0], table.shape[0]
    _check(lib().mla_kv_append_rope_fp8(
        _in(c_kv_new, "c_kv_new", torch.bfloat16, (n, D_C), dev), _in(k_pe_new, "k_pe_new", torch.bfloat16, (n, D_R), dev),
        None if q_pe is None else _in(q_pe, "q_pe", torch.bfloat16, (n, H, D_R), dev),
        _in(positions, "positions", torch.int32, (n,), dev),
        _in(table, "table", torch.float32, (max_pos, D_R // 2, 2), dev), max_pos,
        _in(slots, "slots", torch.int64, (n,), dev), n, _in(rows, "rows", torch.uint8, (pages, PAGE, FP8_ROW_BYTES), dev),
        _in(scales, "scales", torch.float32, (pages, PAGE), dev), pages,
        None if q_r is None else _in(q_r, "q_r", torch.bfloat16, (n, H, D_R), dev),
        _in(dev_err, "dev_err", torch.int32, (1,), dev), _on(stream, dev)))


def mla_gather_paged_fp8(rows, scales, block_table, b: int, n_tokens: int, out, dev_err, stream=None) -> None:
    _need(rows, "rows", torch.uint8, (rows.shape[0], PAGE, FP8_ROW_BYTES))
    _need(scales, "scales", torch.float32, (rows.shape[0], PAGE))
    _need(block_table, "block_table", torch.int32)
    _need(out, "out", torch.bfloat16, (n_tokens, D_QK))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_gather_paged_fp8(_ptr(rows), _ptr(scales), rows.shape[0], _ptr(block_table),
                                      block_table.shape[1], int(b), int(n_tokens), _ptr(out), _ptr(dev_err),
                                      _stream(stream)))


NVFP4_ROW_BYTES = 416


def mla_kv_append_nvfp4(c_kv_new, k_r_new, slots, rows, tensor_scale: float, dev_err, stream=None) -> None:
    """Quantise new tokens into the NVFP4 cache: rows uint8 [pages, 64, 416]."""
    n = c_kv_new.shape[0]
    _need(c_kv_new, "c_kv_new", torch.bfloat16, (n, D_C))
    _need(k_r_new, "k_r_new", torch.bfloat16, (n, D_R))
    _need(slots, "slots", torch.int64, (n,))
    _need(rows, "rows", torch.uint8, (rows.shape[0], PAGE, NVFP4_ROW_BYTES))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_kv_append_nvfp4(_ptr(c_kv_new), _ptr(k_r_new), _ptr(slots), int(n), float(tensor_scale),
                                     _ptr(rows), rows.shape[0], _ptr(dev_err), _stream(stream)))


def mla_gather_paged_nvfp4(rows, tensor_scale: float, block_table, b: int, n_tokens: int, out, dev_err,
                           stream=None) -> None:
    _need(rows, "rows", torch.uint8)
    if rows.dim() != 3 or tuple(rows.shape[1:]) != (PAGE, NVFP4_ROW_BYTES):
        raise ValueError(f"rows has shape {tuple(rows.shape)}, expected (pages, {PAGE}, {NVFP4_ROW_BYTES})")
    _need(block_table, "block_table", torch.int32)
    _need(out, "out", torch.bfloat16, (n_tokens, D_QK))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_gather_paged_nvfp4(_ptr(rows), float(tensor_scale), rows.shape[0], _ptr(block_table),
                                        block_table.shape[1], int(b), int(n_tokens), _ptr(out), _ptr(dev_err),
                                        _stream(stream)))


def mla_gather_paged_nvfp4_batch(rows, tensor_scale: float, block_table, seq_ids, out_offsets, out, dev_err,
                                 stream=None) -> None:
    """Gather the sequences seq_ids (device int32 [nb]) into out bf16 [total, 576]:
    sequence seq_ids[i] fills rows out_offsets[i] .. out_offsets[i+1] (device
    int64 [nb + 1], out_offsets[0] = 0, out_offsets[nb] = total)."""
    _need(rows, "rows", torch.uint8)
    if rows.dim() != 3 or tuple(rows.shape[1:]) != (PAGE, NVFP4_ROW_BYTES):
        raise ValueError(f"rows has shape {tuple(rows.shape)}, expected (pages, {PAGE}, {NVFP4_ROW_BYTES})")
    _need(block_table, "block_table", torch.int32)
    _need(seq_ids, "seq_ids", torch.int32)
    nb = seq_ids.shape[0]
    _need(out_offsets, "out_offsets", torch.int64, (nb + 1,))
    _need(out, "out", torch.bfloat16)
    if out.dim() != 2 or out.shape[1] != D_QK:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected (total, {D_QK})")
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_gather_paged_nvfp4_batch(_ptr(rows), float(tensor_scale), rows.shape[0], _ptr(block_table),
                                              block_table.shape[0], block_table.shape[1], _ptr(seq_ids),
                                              _ptr(out_offsets), nb, out.shape[0], _ptr(out), _ptr(dev_err),
                                              _stream(stream)))


def mla_prefill_threshold() -> int:
    return int(lib().mla_prefill_threshold())


def mla_branch_for(q_len: int) -> int:
    """0 = absorbed (steps A2-A5), 1 = decompress branch."""
    return int(lib().mla_branch_for(int(q_len)))


def mla_expand_kv(rows, w_uk, w_uv, k_c, v_c, dev_err, stream=None) -> None:
    n = rows.shape[0]
    _need(rows, "rows", torch.bfloat16, (n, D_QK))
    _need(w_uk, "w_uk", torch.bfloat16, (H, D_HC, D_C))
    _need(w_uv, "w_uv", torch.bfloat16, (H, D_C, D_HC))
    _need(k_c, "k_c", torch.bfloat16, (H, n, D_HC))
    _need(v_c, "v_c", torch.bfloat16, (H, n, D_HC))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_expand_kv(_ptr(rows), int(n), _ptr(w_uk), _ptr(w_uv), _ptr(k_c), _ptr(v_c), _ptr(dev_err),
                               _stream(stream)))


def mla_prefill_attention(q_c, q_r, rows, k_c, v_c, out, dev_err, scale: float = 1.0 / (192 ** 0.5),
                          stream=None) -> None:
    M, N = q_c.shape[0], rows.shape[0]
    _need(q_c, "q_c", torch.bfloat16, (M, H, D_HC))
    _need(q_r, "q_r", torch.bfloat16, (M, H, D_R))
    _need(rows, "rows", torch.bfloat16, (N, D_QK))
    _need(k_c, "k_c", torch.bfloat16, (H, N, D_HC))
    _need(v_c, "v_c", torch.bfloat16, (H, N, D_HC))
    _need(out, "out", torch.bfloat16, (M, H, D_HC))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_prefill_attention(_ptr(q_c), _ptr(q_r), int(M), _ptr(rows), _ptr(k_c), _ptr(v_c), int(N),
                                       float(scale), _ptr(out), _ptr(dev_err), _stream(stream)))


def mla_prefill_workspace_size(N: int) -> int:
    out = C.c_size_t()
    _check(lib().mla_prefill_workspace_size(int(N), C.byref(out)))
    return int(out.value)


def mla_prefill_decompress(q_c, q_r, kv_cache, block_table, b: int, n_tokens: int, w_uk, w_uv, workspace, out,
                           dev_err, scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    """The decompress branch for sequence b (n_tokens cached, the chunk's M = q_c.shape[0] rows last)."""
    M = q_c.shape[0]
    _need(q_c, "q_c", torch.bfloat16, (M, H, D_HC))
    _need(q_r, "q_r", torch.bfloat16, (M, H, D_R))
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need(block_table, "block_table", torch.int32)
    _need(w_uk, "w_uk", torch.bfloat16, (H, D_HC, D_C))
    _need(w_uv, "w_uv", torch.bfloat16, (H, D_C, D_HC))
    _need(workspace, "workspace", torch.uint8)
    _need(out, "out", torch.bfloat16, (M, H, D_HC))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_prefill_decompress(_ptr(q_c), _ptr(q_r), int(M), _ptr(kv_cache), kv_cache.shape[0],
                                        _ptr(block_table), block_table.shape[1], int(b), int(n_tokens), _ptr(w_uk),
                                        _ptr(w_uv), float(scale), _ptr(workspace), workspace.numel(), _ptr(out),
                                        _ptr(dev_err), _stream(stream)))


def mla_prefill_batch_workspace_size(n_tokens: Sequence[int]) -> int:
    n = np.ascontiguousarray(n_tokens, dtype=np.int32)
    out = C.c_size_t()
    _check(lib().mla_prefill_batch_workspace_size(n.ctypes.data_as(C.POINTER(C.c_int32)), int(n.size),
                                                  C.byref(out)))
    return int(out.value)


def mla_prefill_decompress_batch(q_c, q_r, kv_cache, block_table, seq_ids, q_starts, q_lens, n_tokens, w_uk, w_uv,
                                 workspace, out, dev_err, scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    """The decompress branch for several sequences at once: sequence seq_ids[i]
    (n_tokens[i] cached) with its chunk's q_lens[i] query rows at rows
    q_starts[i].. of q_c, q_r and out."""
    rows = q_c.shape[0]
    _need(q_c, "q_c", torch.bfloat16, (rows, H, D_HC))
    _need(q_r, "q_r", torch.bfloat16, (rows, H, D_R))
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need(block_table, "block_table", torch.int32)
    _need(w_uk, "w_uk", torch.bfloat16, (H, D_HC, D_C))
    _need(w_uv, "w_uv", torch.bfloat16, (H, D_C, D_HC))
    _need(workspace, "workspace", torch.uint8)
    _need(out, "out", torch.bfloat16, (rows, H, D_HC))
    _need(dev_err, "dev_err", torch.int32, (1,))
    arrs = [np.ascontiguousarray(x, dtype=np.int32) for x in (seq_ids, q_starts, q_lens, n_tokens)]
    nb = int(arrs[0].size)
    if any(a.size != nb for a in arrs):
        raise ValueError("seq_ids, q_starts, q_lens and n_tokens must have the same length")
    if any(int(s0) + int(m) > rows for s0, m in zip(arrs[1], arrs[2])):
        raise ValueError("a chunk's rows run past q_c")
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_prefill_decompress_batch(
        _ptr(q_c), _ptr(q_r), *[a.ctypes.data_as(P32) for a in arrs], nb, _ptr(kv_cache), kv_cache.shape[0],
        _ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(w_uk), _ptr(w_uv), float(scale),
        _ptr(workspace), workspace.numel(), _ptr(out), _ptr(dev_err), _stream(stream)))


def mla_rope_table(max_pos: int, table, base: float = 10000.0, stream=None) -> None:
    _need(table, "table", torch.float32, (max_pos, D_R // 2, 2))
    _check(lib().mla_rope_table(int(max_pos), float(base), _ptr(table), _stream(stream)))


def mla_kv_append_rope(c_kv_new, k_pe_new, positions, table, slots, kv_cache, dev_err, stream=None) -> None:
    n = c_kv_new.shape[0]
    _need(c_kv_new, "c_kv_new", torch.bfloat16, (n, D_C))
    _need(k_pe_new, "k_pe_new", torch.bfloat16, (n, D_R))
    _need(positions, "positions", torch.int32, (n,))
    _need(table, "table", torch.float32)
    _need(slots, "slots", torch.int64, (n,))
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need(dev_err, "dev_err", torch.int32, (1,))
    if table.dim() != 3 or tuple(table.shape[1:]) != (D_R // 2, 2):
        raise ValueError(f"table has shape {tuple(table.shape)}, expected (max_pos, {D_R // 2}, 2)")
    _check(lib().mla_kv_append_rope(_ptr(c_kv_new), _ptr(k_pe_new), _ptr(positions), _ptr(table), table.shape[0],
                                    _ptr(slots), int(n), _ptr(kv_cache), kv_cache.shape[0], _ptr(dev_err),
                                    _stream(stream)))


def mla_rope_q(q_pe, positions, table, q_r, dev_err, stream=None) -> None:
    T = q_pe.shape[0]
    _need(q_pe, "q_pe", torch.bfloat16, (T, H, D_R))
    _need(positions, "positions", torch.int32, (T,))
    _need(table, "table", torch.float32)
    _need(q_r, "q_r", torch.bfloat16, (T, H, D_R))
    _need(dev_err, "dev_err", torch.int32, (1,))
    if table.dim() != 3 or tuple(table.shape[1:]) != (D_R // 2, 2):
        raise ValueError(f"table has shape {tuple(table.shape)}, expected (max_pos, {D_R // 2}, 2)")
    _check(lib().mla_rope_q(_ptr(q_pe), _ptr(positions), _ptr(table), table.shape[0], _ptr(q_r), int(T),
                            _ptr(dev_err), _stream(stream)))


def mla_gather_paged(kv_cache, block_table, b: int, n_tokens: int, out, dev_err, stream=None) -> None:
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need(block_table, "block_table", torch.int32)
    _need(out, "out", torch.bfloat16, (n_tokens, D_QK))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_gather_paged(_ptr(kv_cache), kv_cache.shape[0], _ptr(block_table), block_table.shape[1],
                                  int(b), int(n_tokens), _ptr(out), _ptr(dev_err), _stream(stream)))


def mla_absorb_q(q_c, w_uk, q_abs, dev_err, stream=None) -> None:
    T = q_c.shape[0]
    _need(q_c, "q_c", torch.bfloat16, (T, H, D_HC))
    _need(w_uk, "w_uk", torch.bfloat16, (H, D_HC, D_C))
    _need(q_abs, "q_abs", torch.bfloat16, (T, H, D_C))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_absorb_q(_ptr(q_c), _ptr(w_uk), _ptr(q_abs), int(T), _ptr(dev_err), _stream(stream)))


def mla_up_v(o_lat, w_uv, out, dev_err, stream=None) -> None:
    T = o_lat.shape[0]
    _need(o_lat, "o_lat", torch.bfloat16, (T, H, D_C))
    _need(w_uv, "w_uv", torch.bfloat16, (H, D_C, D_HC))
    _need(out, "out", torch.bfloat16, (T, H, D_HC))
    _need(dev_err, "dev_err", torch.int32, (1,))
    _check(lib().mla_up_v(_ptr(o_lat), _ptr(w_uv), _ptr(out), int(T), _ptr(dev_err), _stream(stream)))


def mla_decode_max_clusters() -> int:
    out = C.c_int32()
    _check(lib().mla_decode_max_clusters(C.byref(out)))
    return int(out.value)


def mla_decode_plan_bytes(T: int, num_clusters: int) -> int:
    out = C.c_size_t()
    _check(lib().mla_decode_plan_bytes(int(T), int(num_clusters), C.byref(out)))
    return int(out.value)


def mla_decode_workspace_size(num_clusters: int) -> int:
    out = C.c_size_t()
    _check(lib().mla_decode_workspace_size(int(num_clusters), C.byref(out)))
    return int(out.value)


def mla_decode_plan_host(seq_lens: Sequence[int], q_lens: Sequence[int], num_clusters: int):
    """Host planner only (no GPU): returns (plan int32 array, info)."""
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    ql = np.ascontiguousarray(q_lens, dtype=np.int32)
    T = int(ql.sum()) if ql.size else 0
    nbytes = mla_decode_plan_bytes(T, num_clusters)
    buf = np.zeros(nbytes // 4, dtype=np.int32)
    info = mla_plan_info()
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_decode_plan_host(sl.ctypes.data_as(P32), ql.ctypes.data_as(P32), int(sl.size),
                                      int(num_clusters), buf.ctypes.data_as(C.c_void_p), nbytes, C.byref(info)))
    return buf, info


@dataclass
class DecodePlan:
    """A plan on the device plus its host summary (mla_decode_plan)."""
    plan: torch.Tensor          # int32 device buffer
    info: mla_plan_info
    workspace: torch.Tensor     # uint8 device buffer
    host: Optional[torch.Tensor] = None   # pinned int32 staging of the plan (reused by `into=`)
    streams: set = field(default_factory=set, repr=False, compare=False)  # raw handles of the streams that use the buffers

    @property
    def num_clusters(self) -> int:
        return int(self.info.num_clusters)


def _use(plan, stream, dev: int) -> int:
    """The raw handle of the stream that a call reads or writes a plan's buffers
    on.  The allocator learns of every such stream: a plan may be dropped as soon
    as its last call is queued, and its blocks are handed out again only after
    the work queued there."""
    raw = _on(stream, dev)
    if raw not in plan.streams:
        if stream is None:
            on = torch.cuda.current_stream(dev)
        elif isinstance(stream, torch.cuda.Stream):
            on = stream
        else:  # any object with a `cuda_stream`
            on = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
        plan.plan.record_stream(on)
        plan.workspace.record_stream(on)
        plan.streams.add(raw)
    return raw


def _plan_buffers(cls, words: int, ws_bytes: int, device):
    """A plan without contents.  The blocks are those of the stream that is
    current, the one that uploads: a block that work queued on another stream
    still uses is never overwritten by the upload."""
    plan = torch.empty(words, dtype=torch.int32, device=device)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
    host = torch.zeros(words, dtype=torch.int32).pin_memory()
    return cls(plan=plan, info=None, workspace=ws, host=host, streams={_on(None, plan.get_device())})


def _upload(plan, words: int, stream) -> None:
    with torch.cuda.stream(stream):
        _use(plan, None, plan.plan.get_device())
        plan.plan[:words].copy_(plan.host[:words], non_blocking=True)


def mla_decode_plan(seq_lens: Sequence[int], q_lens: Sequence[int], device=None, num_clusters: Optional[int] = None,
                    stream=None, into: Optional[DecodePlan] = None) -> DecodePlan:
    """Plan on the host into a pinned buffer and upload it with an
    asynchronous copy on `stream` (a copy from pageable memory would make
    the host wait for the stream).  A decode on another stream has to wait
    for the upload (an event); the plan may be dropped once its last decode is
    queued.  `into` reuses a previous plan's buffers when they are large
    enough; the caller must not reuse a plan whose previous upload or decode
    may still be running."""
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    ql = np.ascontiguousarray(q_lens, dtype=np.int32)
    T = int(ql.sum()) if ql.size else 0
    if num_clusters is None:
        num_clusters = into.num_clusters if into is not None else mla_decode_max_clusters()
    nbytes = mla_decode_plan_bytes(T, num_clusters)
    words = (nbytes + 15) // 16 * 4
    device = device or torch.device("cuda", torch.cuda.current_device())
    ws_bytes = max(mla_decode_workspace_size(num_clusters), 16)
    if (into is not None and into.host is not None and into.plan.numel() >= words
            and into.workspace.numel() >= ws_bytes and into.plan.device == torch.device(device)):
        plan = replace(into)
    else:
        with torch.cuda.stream(stream):
            plan = _plan_buffers(DecodePlan, words, ws_bytes, device)
    plan.info = mla_plan_info()
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_decode_plan_host(sl.ctypes.data_as(P32), ql.ctypes.data_as(P32), int(sl.size),
                                      int(num_clusters), C.c_void_p(plan.host.data_ptr()), nbytes, C.byref(plan.info)))
    _upload(plan, words, stream)
    return plan


def plan_rows(plan: DecodePlan) -> dict:
    """The query rows a plan treats specially, read from its host copy (the
    plan layout of csrc/internal.h): rows cut into several pieces (merged by
    the combine) and rows whose segment starts or ends a cluster's range.
    For choosing parity samples; no device work."""
    w = plan.host.numpy() if plan.host is not None else None
    if w is None:
        raise ValueError("the plan has no host copy")
    nc, ns, nsplit = int(w[3]), int(w[4]), int(w[6])
    seg_off = 16
    seg_base = (seg_off + nc + 1 + 7) // 8 * 8
    split_base = seg_base + 8 * ns
    split = sorted(int(w[split_base + 4 * i]) for i in range(nsplit))
    boundary = set()
    for c in range(nc):
        a, b = int(w[seg_off + c]), int(w[seg_off + c + 1])
        if b > a:
            boundary.add(int(w[seg_base + 8 * a]))
            boundary.add(int(w[seg_base + 8 * (b - 1)]))
    return {"split": split, "boundary": sorted(boundary)}


def mla_decode_paged(q_abs, q_r, kv_cache, block_table, plan: DecodePlan, o_lat, dev_err, lse=None,
                     scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    T = q_abs.shape[0]
    _need(q_abs, "q_abs", torch.bfloat16, (T, H, D_C))
    _need(q_r, "q_r", torch.bfloat16, (T, H, D_R))
    _need(kv_cache, "kv_cache", torch.bfloat16)
    if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (PAGE, D_QK):
        raise ValueError("kv_cache must be [num_pages, 64, 576]")
    _need(block_table, "block_table", torch.int32)
    _need(o_lat, "o_lat", torch.bfloat16, (T, H, D_C))
    _need(dev_err, "dev_err", torch.int32, (1,))
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, H))
    if int(plan.info.T) != T:
        raise ValueError(f"plan has {plan.info.T} rows, q_abs has {T}")
    _check(lib().mla_decode_paged(_ptr(q_abs), _ptr(q_r), _ptr(kv_cache), kv_cache.shape[0], _ptr(block_table),
                                  block_table.shape[1], _ptr(plan.plan), C.byref(plan.info), float(scale),
                                  _ptr(plan.workspace), plan.workspace.numel(), _ptr(o_lat), _ptr(lse),
                                  _ptr(dev_err), _use(plan, stream, torch.cuda.current_device())))


def mla_decode_paged_fp8(q_abs, q_r, rows, scales, block_table, plan: DecodePlan, o_lat, dev_err, lse=None,
                         scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    """Steps A3 + A4 over the FP8 cache (rows uint8 [pages, 64, 640], scales fp32 [pages, 64])."""
    T = q_abs.shape[0]
    _need(q_abs, "q_abs", torch.bfloat16, (T, H, D_C))
    _need(q_r, "q_r", torch.bfloat16, (T, H, D_R))
    _need(rows, "rows", torch.uint8, (rows.shape[0], PAGE, FP8_ROW_BYTES))
    _need(scales, "scales", torch.float32, (rows.shape[0], PAGE))
    _need(block_table, "block_table", torch.int32)
    _need(o_lat, "o_lat", torch.bfloat16, (T, H, D_C))
    _need(dev_err, "dev_err", torch.int32, (1,))
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, H))
    if int(plan.info.T) != T:
        raise ValueError(f"plan has {plan.info.T} rows, q_abs has {T}")
    _check(lib().mla_decode_paged_fp8(_ptr(q_abs), _ptr(q_r), _ptr(rows), _ptr(scales), rows.shape[0],
                                      _ptr(block_table), block_table.shape[1], _ptr(plan.plan), C.byref(plan.info),
                                      float(scale), _ptr(plan.workspace), plan.workspace.numel(), _ptr(o_lat),
                                      _ptr(lse), _ptr(dev_err), _use(plan, stream, torch.cuda.current_device())))


# ------------------------------------------------------------------ sliding window with sinks
def _host_i32(*lists):
    """Host lists of sequences as int32 arrays of one length."""
    arrs = []
    for x in lists:
        v = np.asarray(x)
        a = np.ascontiguousarray(v, dtype=np.int32)
        if v.ndim != 1 or (a != v).any():
            raise ValueError("the sequences' lists must be one-dimensional, of values that int32 holds")
        arrs.append(a)
    if any(a.size != arrs[0].size for a in arrs):
        raise ValueError("the sequences' lists must have the same length")
    return arrs


def _window_args(window, sinks):
    """window and sinks as C int32 values (the library judges their signs)."""
    w, s = operator.index(window), operator.index(sinks)
    if max(abs(w), abs(s)) > 2 ** 31 - 1:
        raise ValueError(f"window = {w}, sinks = {s}: at most 2^31 - 1")
    return w, s


def mla_window_plan_host(seq_lens: Sequence[int], q_lens: Sequence[int], window: int, sinks: int, num_clusters: int):
    """Host planner of the windowed decode only (no GPU): returns (plan int32 array, info)."""
    sl, ql = _host_i32(seq_lens, q_lens)
    window, sinks = _window_args(window, sinks)
    nbytes = mla_decode_plan_bytes(int(ql.sum()) if ql.size else 0, num_clusters)
    buf = np.zeros(nbytes // 4, dtype=np.int32)
    info = mla_window_info()
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_window_plan_host(sl.ctypes.data_as(P32), ql.ctypes.data_as(P32), int(sl.size), window,
                                      sinks, int(num_clusters), buf.ctypes.data_as(C.c_void_p), nbytes,
                                      C.byref(info)))
    return buf, info


@dataclass
class WindowPlan:
    """A window plan on the device plus its host summary (mla_window_plan)."""
    plan: torch.Tensor          # int32 device buffer
    info: mla_window_info
    workspace: torch.Tensor     # uint8 device buffer
    host: torch.Tensor          # pinned int32 staging of the plan (reused by `into=`)
    streams: set = field(default_factory=set, repr=False, compare=False)  # raw handles of the streams that use the buffers

    @property
    def num_clusters(self) -> int:
        return int(self.info.plan.num_clusters)


def mla_window_plan(seq_lens: Sequence[int], q_lens: Sequence[int], window: int, sinks: int, device=None,
                    num_clusters: Optional[int] = None, stream=None, into: Optional[WindowPlan] = None) -> WindowPlan:
    """mla_decode_plan for a sliding window with sinks: one plan serves every
    layer of a step.  The upload runs on `stream`; a decode on another stream has
    to wait for it (an event), and the plan may be dropped once its last decode
    is queued.  A plan holds one workspace, so decodes that share it must not
    overlap on the GPU; `into` reuses a previous plan's buffers when they are
    large enough and nothing that reads them may still be running."""
    if num_clusters is None:
        num_clusters = mla_decode_max_clusters()
    buf, info = mla_window_plan_host(seq_lens, q_lens, window, sinks, num_clusters)
    words = (buf.size + 3) // 4 * 4
    device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    ws_bytes = max(mla_decode_workspace_size(num_clusters), 16)
    if (into is not None and into.plan.numel() >= words and into.workspace.numel() >= ws_bytes
            and into.plan.device == device):
        plan = replace(into)
    else:
        with torch.cuda.stream(stream):
            plan = _plan_buffers(WindowPlan, words, ws_bytes, device)
    plan.info = info
    plan.host[:buf.size] = torch.from_numpy(buf)
    _upload(plan, words, stream)
    return plan


def mla_decode_window(q_abs, q_r, kv_cache, block_table, plan: WindowPlan, o_lat, dev_err, lse=None,
                      scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    """mla_decode_paged with the plan's sliding window and sinks."""
    dev = torch.cuda.current_device()
    pages = kv_cache.shape[0]
    cache = (_in(kv_cache, "kv_cache", torch.bfloat16, (pages, PAGE, D_QK), dev),)
    _decode_window(lib().mla_decode_window, cache, pages, q_abs, q_r, block_table, plan, o_lat, dev_err, lse, scale,
                   stream, dev)


def mla_decode_window_fp8(q_abs, q_r, rows, scales, block_table, plan: WindowPlan, o_lat, dev_err, lse=None,
                          scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    """mla_decode_paged_fp8 with the plan's sliding window and sinks."""
    dev = torch.cuda.current_device()
    pages = rows.shape[0]
    cache = (_in(rows, "rows", torch.uint8, (pages, PAGE, FP8_ROW_BYTES), dev),
             _in(scales, "scales", torch.float32, (pages, PAGE), dev))
    _decode_window(lib().mla_decode_window_fp8, cache, pages, q_abs, q_r, block_table, plan, o_lat, dev_err, lse, scale,
                   stream, dev)


def _decode_window(call, cache, pages, q_abs, q_r, block_table, plan, o_lat, dev_err, lse, scale, stream, dev) -> None:
    if not isinstance(plan, WindowPlan):
        raise TypeError("plan must come from mla_window_plan")
    T, sums = q_abs.shape[0], plan.info.plan
    if sums.T != T:
        raise ValueError(f"plan has {sums.T} rows, q_abs has {T}")
    if block_table.dim() != 2 or block_table.shape[0] < sums.B:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}, the plan has {sums.B} sequences")
    cols = block_table.shape[1]
    ws_bytes = plan.workspace.numel()
    _check(call(_in(q_abs, "q_abs", torch.bfloat16, (T, H, D_C), dev), _in(q_r, "q_r", torch.bfloat16, (T, H, D_R), dev),
                *cache, pages, _in(block_table, "block_table", torch.int32, (block_table.shape[0], cols), dev), cols,
                _in(plan.plan, "plan.plan", torch.int32, (plan.plan.numel(),), dev), plan.info, float(scale),
                _in(plan.workspace, "plan.workspace", torch.uint8, (ws_bytes,), dev), ws_bytes,
                _in(o_lat, "o_lat", torch.bfloat16, (T, H, D_C), dev),
                None if lse is None else _in(lse, "lse", torch.float32, (T, H), dev),
                _in(dev_err, "dev_err", torch.int32, (1,), dev), _use(plan, stream, dev)))


def mla_prefill_window_workspace_size(q_lens: Sequence[int], n_tokens: Sequence[int], window: int, sinks: int) -> int:
    q, n = _host_i32(q_lens, n_tokens)
    window, sinks = _window_args(window, sinks)
    out = C.c_size_t()
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_prefill_window_workspace_size(q.ctypes.data_as(P32), n.ctypes.data_as(P32), int(n.size),
                                                   window, sinks, C.byref(out)))
    return int(out.value)


def _prefill_window(call, cache, pages, q_c, q_r, block_table, seq_ids, q_starts, q_lens, n_tokens, window, sinks,
                    w_uk, w_uv, workspace, out, dev_err, scale, stream, dev) -> None:
    rows = q_c.shape[0]
    if block_table.dim() != 2:
        raise ValueError("block_table must be [sequences, pages]")
    batch, cols = block_table.shape
    window, sinks = _window_args(window, sinks)
    arrs = _host_i32(seq_ids, q_starts, q_lens, n_tokens)
    if arrs[0].size and int((arrs[1].astype(np.int64) + arrs[2]).max()) > rows:
        raise ValueError("a chunk's rows run past q_c")
    P32 = C.POINTER(C.c_int32)
    ws_bytes = workspace.numel()
    _check(call(_in(q_c, "q_c", torch.bfloat16, (rows, H, D_HC), dev), _in(q_r, "q_r", torch.bfloat16, (rows, H, D_R), dev),
                *[a.ctypes.data_as(P32) for a in arrs], arrs[0].size, window, sinks, *cache, pages,
                _in(block_table, "block_table", torch.int32, (batch, cols), dev), batch, cols,
                _in(w_uk, "w_uk", torch.bfloat16, (H, D_HC, D_C), dev),
                _in(w_uv, "w_uv", torch.bfloat16, (H, D_C, D_HC), dev), float(scale),
                _in(workspace, "workspace", torch.uint8, (ws_bytes,), dev), ws_bytes,
                _in(out, "out", torch.bfloat16, (rows, H, D_HC), dev), _in(dev_err, "dev_err", torch.int32, (1,), dev),
                _on(stream, dev)))


def mla_prefill_window_batch(q_c, q_r, kv_cache, block_table, seq_ids, q_starts, q_lens, n_tokens, window: int,
                             sinks: int, w_uk, w_uv, workspace, out, dev_err, scale: float = 1.0 / (192 ** 0.5),
                             stream=None) -> None:
    """mla_prefill_decompress_batch with a sliding window and sinks: only the
    tokens that a chunk's rows see are gathered and expanded."""
    dev = torch.cuda.current_device()
    pages = kv_cache.shape[0]
    cache = (_in(kv_cache, "kv_cache", torch.bfloat16, (pages, PAGE, D_QK), dev),)
    _prefill_window(lib().mla_prefill_window_batch, cache, pages, q_c, q_r, block_table, seq_ids, q_starts, q_lens,
                    n_tokens, window, sinks, w_uk, w_uv, workspace, out, dev_err, scale, stream, dev)


def mla_prefill_window_batch_fp8(q_c, q_r, rows, scales, block_table, seq_ids, q_starts, q_lens, n_tokens, window: int,
                                 sinks: int, w_uk, w_uv, workspace, out, dev_err, scale: float = 1.0 / (192 ** 0.5),
                                 stream=None) -> None:
    """mla_prefill_window_batch over the FP8 cache."""
    dev = torch.cuda.current_device()
    pages = rows.shape[0]
    cache = (_in(rows, "rows", torch.uint8, (pages, PAGE, FP8_ROW_BYTES), dev),
             _in(scales, "scales", torch.float32, (pages, PAGE), dev))
    _prefill_window(lib().mla_prefill_window_batch_fp8, cache, pages, q_c, q_r, block_table, seq_ids, q_starts, q_lens,
                    n_tokens, window, sinks, w_uk, w_uv, workspace, out, dev_err, scale, stream, dev)


# ------------------------------------------------------------------ 4-bit weights
def mla_pack_w4(w, group: int, stream=None):
    """Quantise W_UK [128, 128, 512] or W_UV [128, 512, 128] (bf16) to 4-bit codes
    with a bf16 scale per group of the contraction (dim 1); returns (words, scales)."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise TypeError("w must be a torch.Tensor [128, K, N]")
    K, N, group = w.shape[1], w.shape[2], operator.index(group)
    if not 8 <= group <= D_C:  # beyond 32 bits another size would reach the library
        raise ValueError(f"group = {group}: 32, 64 and 128 are supported")
    addr = _in(w, "w", torch.bfloat16, (H, K, N), torch.cuda.current_device())
    with torch.cuda.stream(stream):
        words = torch.empty((H, K // 8, N), dtype=torch.int32, device=w.device)
        scales = torch.empty((H, max(K // group, 1), N), dtype=torch.bfloat16, device=w.device)
    _check(lib().mla_pack_w4(addr, K, N, group, _ptr(words), _ptr(scales), _stream(stream)))
    return words, scales


def _w4(call, x, x_name, words, scales, y, y_name, K, N, dev_err, stream) -> None:
    dev = torch.cuda.current_device()
    T = x.shape[0]
    if scales.dim() != 3 or scales.shape[1] < 1 or K % scales.shape[1]:
        raise ValueError(f"scales has shape {tuple(scales.shape)}, expected ({H}, groups of {K} values, {N})")
    groups = scales.shape[1]
    _check(call(_in(x, x_name, torch.bfloat16, (T, H, K), dev), _in(words, "words", torch.int32, (H, K // 8, N), dev),
                _in(scales, "scales", torch.bfloat16, (H, groups, N), dev), K // groups,
                _in(y, y_name, torch.bfloat16, (T, H, N), dev), T, _in(dev_err, "dev_err", torch.int32, (1,), dev),
                _on(stream, dev)))


def mla_absorb_q_w4(q_c, words, scales, q_abs, dev_err, stream=None) -> None:
    """mla_absorb_q over W_UK in 4 bits (mla_pack_w4); the group is 128 / scales.shape[1]."""
    _w4(lib().mla_absorb_q_w4, q_c, "q_c", words, scales, q_abs, "q_abs", D_HC, D_C, dev_err, stream)


def mla_up_v_w4(o_lat, words, scales, out, dev_err, stream=None) -> None:
    """mla_up_v over W_UV in 4 bits (mla_pack_w4); the group is 512 / scales.shape[1]."""
    _w4(lib().mla_up_v_w4, o_lat, "o_lat", words, scales, out, "out", D_C, D_HC, dev_err, stream)


def mla_check(dev_err, stream=None) -> int:
    """Synchronise and return the device error word; raises on a non-zero word."""
    word = C.c_int32()
    _check(lib().mla_check(_stream(stream), _ptr(dev_err), C.byref(word)))
    return int(word.value)


def mla_debug_set_decode_wait_limit(cycles: int) -> None:
    """Test hook: every wait of the decode loop gives up after `cycles` SM
    cycles (0 restores the default of 2^31); process-wide."""
    _check(lib().mla_debug_set_decode_wait_limit(int(cycles)))


def mla_decode_paged_noalloc(q_abs, q_r, kv_cache, block_table, seq_lens, q_lens, o_lat, dev_err, lse=None,
                             scale: float = 1.0 / (192 ** 0.5), stream=None) -> None:
    """mla_decode_paged without caller-provided plan or workspace: for callers
    that cannot allocate device memory (the library keeps both in a device
    array of its own).  Calls that may overlap on the GPU must be serialised."""
    T = q_abs.shape[0]
    _need(q_abs, "q_abs", torch.bfloat16, (T, H, D_C))
    _need(q_r, "q_r", torch.bfloat16, (T, H, D_R))
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need(block_table, "block_table", torch.int32)
    _need(o_lat, "o_lat", torch.bfloat16, (T, H, D_C))
    _need(dev_err, "dev_err", torch.int32, (1,))
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, H))
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    ql = np.ascontiguousarray(q_lens, dtype=np.int32)
    if int(ql.sum()) != T:
        raise ValueError(f"q_lens sum to {int(ql.sum())} rows, q_abs has {T}")
    P32 = C.POINTER(C.c_int32)
    _check(lib().mla_decode_paged_noalloc(_ptr(q_abs), _ptr(q_r), _ptr(kv_cache), kv_cache.shape[0],
                                          _ptr(block_table), block_table.shape[1], sl.ctypes.data_as(P32),
                                          ql.ctypes.data_as(P32), int(sl.size), float(scale), _ptr(o_lat),
                                          _ptr(lse), _ptr(dev_err), _stream(stream)))
