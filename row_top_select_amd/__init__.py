"""Python binding of the row_top_select C ABI (include/row_top_select.h).

Argument marshalling only: every step runs in the HIP kernels of
``librow_top_select.so``.  PyTorch provides device memory and the current
stream; tensors must live on the GPU.  Importing this package fails loudly if
the library has not been built (``python row_top_select_amd/build.py``).
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librow_top_select.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python row_top_select_amd/build.py` "
        "(hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)

RTS_OK, RTS_EINVAL, RTS_EUNSUPPORTED, RTS_EWORKSPACE, RTS_EHIP = 0, -1, -2, -3, -4
RTS_F32, RTS_BF16, RTS_E4M3 = 0, 1, 2

_i64, _i32, _p, _sz, _f32 = (ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                             ctypes.c_float)
_lib.rts_status_string.argtypes = [ctypes.c_int]
_lib.rts_status_string.restype = ctypes.c_char_p
_lib.topk_rows_workspace_size.argtypes = [ctypes.c_int, _i64, _i64, _i32]
_lib.topk_rows_workspace_size.restype = _sz
_lib.topk_rows.argtypes = [_p, ctypes.c_int, _i64, _i64, _i64, _p, _i32, _p, _i64, _p, _sz, _p]
_lib.topk_rows_noalloc.argtypes = [_p, ctypes.c_int, _i64, _i64, _i64, _p, _i32, _p, _i64, _p]
_lib.pack_candidates.argtypes = [_p, _i64, _i64, _i64, _p, _i32, _i64, _p, _p, _p]
_lib.merge_select_rank_major.argtypes = [_p, _i32, _i64, _i32, _i32, _p, _p, _p]
_lib.pack_pairs.argtypes = [_p, _i64, _i64, _i64, _p, _i32, _i64, _p, _i32, _i32, _p, _p]
_lib.merge_select_pairs_rank_major.argtypes = [_p, _i32, _i64, _i32, _i32, _p, _p]
_lib.merge_select_row_major.argtypes = [_p, _i32, _i64, _i32, _i32, _p, _p, _p]
_lib.merge_select_pairs_row_major.argtypes = [_p, _i32, _i64, _i32, _i32, _p, _p]
_lib.emit_rows.argtypes = [_p, _i64, _i32, _i32, _i32, _p, _p, _i64, _i32, _i64, _i32, _i64, _p, _i32,
                           _p, _p]
_lib.merge_select_rank_major_rows.argtypes = [_p, _i32, _i64, _i32, _i32, _p, _p, _p, _p]
_lib.merge_rescue_rank_major_rows.argtypes = [_p, _p, _i32, _i64, _i32, _i32, _p, _p, _p, _p]
_lib.rescue_push.argtypes = [_p, _i32, _i32, _i64, _i32, _i32, _p, _p, _p]
_lib.merge_rescue_rank_major.argtypes = [_p, _p, _i32, _i64, _i32, _i32, _p, _p, _p]
_lib.assign_slots.argtypes = [_p, _p, _i64, _i64, _i32, _i64, _p, _i64, _p, _i32, _i64, _p, _p, _p, _p, _p,
                              _p]
_lib.indexer_logits.argtypes = [_p, ctypes.c_int, _i64, _i32, _i32, _i64, _p, _i64, _i64, _p, _i64, _p, _p, _p,
                                ctypes.c_int, _i64, _p]
_lib.indexer_logits_paged.argtypes = [_p, ctypes.c_int, _i64, _i32, _i32, _i64, _p, _i64, _i64, _p, _i64, _p,
                                      _p, _p, _p, _i64, _i32, _i64, _i32, _i64, _i64, _p, ctypes.c_int, _i64,
                                      _p]
_lib.latent_attend_rows_workspace_size.argtypes = [_i64, _i32, _i32, _i32]
_lib.latent_attend_rows_workspace_size.restype = _sz
_lib.latent_attend_rows.argtypes = [_p, _i64, _i32, _i32, _i32, _i64, _i64, _p, _i64, _i64, _p, _i32, _i64, _p,
                                    _f32, _p, _p, _p, _sz, _p]
_lib.latent_attend_paged_workspace_size.argtypes = [_i64, _i64, _i32, _i32, _i64]
_lib.latent_attend_paged_workspace_size.restype = _sz
_lib.latent_attend_paged.argtypes = [_p, _i64, _i32, _i32, _i32, _i64, _i64, _p, _i64, _i64, _p, _p, _i64, _p,
                                     _p, _i32, _i64, _i32, _i64, _i64, _f32, _p, _p, _p, _sz, _p]
_lib.merge_attend_rank_major.argtypes = [_p, ctypes.c_int, _p, _i32, _i64, _i32, _i32, _p, ctypes.c_int, _p, _p]
_lib.beam_select_workspace_size.argtypes = [ctypes.c_int, _i64, _i32, _i64, _i32]
_lib.beam_select_workspace_size.restype = _sz
_lib.beam_select.argtypes = [_p, ctypes.c_int, _i64, _i32, _i64, _i64, _p, _i32, _i32, _p, _p, _p, _p, _p, _sz, _p]
_lib.fork_blocks.argtypes = [_p, _i64, _i32, _i64, _p, _p, _i64, _i32, _i32, _p, _p, _i64, _p, _p, _p, _i64, _p, _p, _sz,
                             _p]
_lib.fork_blocks_workspace_size.argtypes = [_i64, _i32, _i32]
_lib.fork_blocks_workspace_size.restype = _sz
_lib.compact_blocks_workspace_size.argtypes = [_i64, _i32, _i32]
_lib.compact_blocks_workspace_size.restype = _sz
_lib.compact_blocks.argtypes = [_p, _i64, _i32, _i64, _p, _i32, _i32, _p, _p, _i64, _p, _i64, _p, _i64, _p, _p, _sz,
                                _p]
_lib.copy_blocks.argtypes = [_p, _i32, _p, _i64, _i32, _i64, _p]
_lib.kv_attend_paged_workspace_size.argtypes = [_i64, _i32, _i32, _i32, ctypes.c_int, _i64, _i64]
_lib.kv_attend_paged_workspace_size.restype = _sz
_lib.kv_attend_paged.argtypes = [_p, _i64, _i32, _i64, _i64, _p, _p, ctypes.c_int, _i32, _i32, _i64, _i64, _i64, _p, _p,
                                 _p, _p, _p, _i64, _i32, _i64, _i32, _i64, _i64, _i64, _f32, _p, _p, _p, _sz, _p]
for _f in (_lib.beam_select, _lib.fork_blocks, _lib.compact_blocks, _lib.copy_blocks, _lib.kv_attend_paged,
           _lib.assign_slots, _lib.indexer_logits, _lib.indexer_logits_paged, _lib.latent_attend_rows,
           _lib.latent_attend_paged, _lib.merge_attend_rank_major, _lib.topk_rows, _lib.topk_rows_noalloc, _lib.pack_candidates, _lib.merge_select_rank_major, _lib.pack_pairs,
           _lib.merge_select_pairs_rank_major, _lib.rescue_push, _lib.merge_rescue_rank_major,
           _lib.merge_select_row_major, _lib.merge_select_pairs_row_major, _lib.emit_rows,
           _lib.merge_select_rank_major_rows, _lib.merge_rescue_rank_major_rows):
    _f.restype = ctypes.c_int


class _KvRows(ctypes.Structure):
    """rts_kv_rows of include/row_top_select.h."""
    _fields_ = [("dcp_rank", ctypes.c_int32), ("req_id", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("table_rows", ctypes.c_int64),
                ("table_cols", ctypes.c_int32), ("ld_table", ctypes.c_int64),
                ("block_size", ctypes.c_int32), ("stride_rows", ctypes.c_int64),
                ("rows_out", ctypes.c_void_p), ("out_cols", ctypes.c_int32),
                ("valid_out", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    """rts_cache of include/row_top_select.h."""
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("row_bytes", ctypes.c_int64),
                ("ld_bytes", ctypes.c_int64)]


class RtsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {rts_status_string(status)}")


def rts_status_string(status: int) -> str:
    return _lib.rts_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != RTS_OK:
        raise RtsError(status, where)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# torch.cuda.current_stream(device).cuda_stream without the Stream object,
# which costs as much as a small call's launch; where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(device: torch.device) -> int:
    return _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream


def _new(shape, dtype, device: torch.device, stream, returned: bool = True) -> torch.Tensor:
    """Memory for a call on ``stream`` (None: the current stream).  A freed block of one stream's pool
    may still be in use by what that stream has yet to run, so a call on another stream takes
    memory from its own.  What is returned is given back when the current stream, which may
    read it, is done with it too."""
    if stream is None or device.type != "cuda" or stream.cuda_stream == _current(device):
        return torch.empty(shape, dtype=dtype, device=device)
    reader = torch.cuda.current_stream(device)
    if device.index == torch.cuda.current_device() and device == stream.device:
        torch.cuda.set_stream(stream)  # less than half of the context manager's time
        try:
            t = torch.empty(shape, dtype=dtype, device=device)
        finally:
            torch.cuda.set_stream(reader)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(reader)
    return t


def _dev(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return ctypes.c_void_p(t.data_ptr())


def _opt(t, name):
    return None if t is None else _dev(t, name)


def _rows_ld(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return rows, cols, (ld if rows > 1 else cols)


def _int32_vec(t, rows, name):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] < rows or (rows > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous int32 vector of >= {rows} entries")
    return t


def topk_rows_workspace_size(dtype, rows: int, cols: int, k: int) -> int:
    dt = RTS_BF16 if dtype in (torch.bfloat16, RTS_BF16) else RTS_F32
    return int(_lib.topk_rows_workspace_size(dt, rows, cols, k))


def topk_rows(logits: torch.Tensor, k: int, row_ends: torch.Tensor | None = None,
              out: torch.Tensor | None = None, workspace="auto", stream=None) -> torch.Tensor:
    """Exact per-row top-k column ids (score desc, id asc), -1 padded; see topk_rows in the header.

    ``out`` may be wider than k (columns past k are left untouched).  ``workspace``:
    "auto" (allocated here when the shape splits rows), None, or a uint8 GPU tensor.
    """
    if logits.dtype == torch.float32:
        dt = RTS_F32
    elif logits.dtype == torch.bfloat16:
        dt = RTS_BF16
    else:
        raise TypeError("logits must be float32 or bfloat16")
    rows, cols, ld = _rows_ld(logits, "logits")
    row_ends = _int32_vec(row_ends, rows, "row_ends")
    if out is None:
        out = _new((rows, k), torch.int32, logits.device, stream)
    if out.dtype != torch.int32:
        raise TypeError("out must be int32")
    if out.device != logits.device:
        raise ValueError("out must be on the device of logits")
    out_rows, out_cols, ld_out = _rows_ld(out, "out")
    if out_rows < rows or out_cols < k:
        raise ValueError(f"out must hold at least [{rows}, {k}] (got {tuple(out.shape)})")
    if rows <= 1:
        ld_out = max(ld_out, k)
    ws, ws_bytes = None, 0
    if isinstance(workspace, str) and workspace == "auto":
        need = topk_rows_workspace_size(dt, rows, cols, k)
        if need:
            ws = _new(need, torch.uint8, logits.device, stream, returned=False)
            ws_bytes = need
    elif workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != logits.device or \
                not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of logits")
        ws, ws_bytes = workspace, workspace.numel() * workspace.element_size()
    _check(_lib.topk_rows(_dev(logits, "logits"), dt, rows, cols, ld, _opt(row_ends, "row_ends"), k,
                          _dev(out, "out"), ld_out, _opt(ws, "workspace"), ws_bytes, _stream(stream)),
           "topk_rows")
    return out


def topk_rows_noalloc(logits: torch.Tensor, k: int, out: torch.Tensor,
                      row_ends: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """topk_rows into a caller-given ``out`` with no allocation at all (split rows use
    the library's static device scratch); see topk_rows_noalloc in the header."""
    if logits.dtype == torch.float32:
        dt = RTS_F32
    elif logits.dtype == torch.bfloat16:
        dt = RTS_BF16
    else:
        raise TypeError("logits must be float32 or bfloat16")
    rows, cols, ld = _rows_ld(logits, "logits")
    row_ends = _int32_vec(row_ends, rows, "row_ends")
    if out.dtype != torch.int32:
        raise TypeError("out must be int32")
    if out.device != logits.device:
        raise ValueError("out must be on the device of logits")
    out_rows, out_cols, ld_out = _rows_ld(out, "out")
    if out_rows < rows or out_cols < k:
        raise ValueError(f"out must hold at least [{rows}, {k}] (got {tuple(out.shape)})")
    if rows <= 1:
        ld_out = max(ld_out, k)
    _check(_lib.topk_rows_noalloc(_dev(logits, "logits"), dt, rows, cols, ld,
                                  _opt(row_ends, "row_ends"), k, _dev(out, "out"), ld_out,
                                  _stream(stream)), "topk_rows_noalloc")
    return out


def pack_candidates(logits_bf16: torch.Tensor, local_idx: torch.Tensor,
                    row_ends: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """B' packed rows int32 [rows, n + n/32] of a local top-n; see pack_candidates in the header."""
    if logits_bf16.dtype != torch.bfloat16:
        raise TypeError("logits must be bfloat16")
    rows, cols, ld = _rows_ld(logits_bf16, "logits")
    if local_idx.dtype != torch.int32:
        raise TypeError("local_idx must be int32")
    r2, n, ld_idx = _rows_ld(local_idx, "local_idx")
    if r2 != rows:
        raise ValueError("local_idx must have one row per logits row")
    if rows <= 1:
        ld_idx = max(ld_idx, n)
    row_ends = _int32_vec(row_ends, rows, "row_ends")
    width = n + n // 32
    if out is None:
        out = _new((rows, width), torch.int32, logits_bf16.device, stream)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, width) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, {width}]")
    _check(_lib.pack_candidates(_dev(logits_bf16, "logits"), rows, cols, ld,
                                _dev(local_idx, "local_idx"), n, ld_idx, _opt(row_ends, "row_ends"),
                                _dev(out, "out"), _stream(stream)), "pack_candidates")
    return out


def merge_select_rank_major(gathered: torch.Tensor, k: int, out: torch.Tensor | None = None,
                            sat_word: torch.Tensor | None = None, want_sat: bool = True,
                            stream=None):
    """Select from int32 [W, R, n + n/32]; returns (ids [R, k], sat_word [R] or None)."""
    if gathered.dtype != torch.int32 or gathered.dim() != 3 or not gathered.is_contiguous():
        raise ValueError("gathered must be contiguous int32 [W, R, n + n/32]")
    world, rows, width = gathered.shape
    n = width * 32 // 33
    if n + n // 32 != width:
        raise ValueError("gathered's last dimension must be n + n/32")
    if out is None:
        out = _new((rows, k), torch.int32, gathered.device, stream)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, {k}]")
    if sat_word is None and want_sat:
        sat_word = _new((rows,), torch.int32, gathered.device, stream)
    _check(_lib.merge_select_rank_major(_dev(gathered, "gathered"), world, rows, n, k, _dev(out, "out"),
                                        _opt(sat_word, "sat_word"), _stream(stream)),
           "merge_select_rank_major")
    return out, sat_word


def rescue_slots(n: int, k: int) -> int:
    """Receive slots per row of the second round: (k - 1) // n."""
    return (k - 1) // n


def _packed_width(t: torch.Tensor, name: str) -> int:
    w = t.shape[-1]
    m = w * 32 // 33
    if m + m // 32 != w:
        raise ValueError(f"{name}'s last dimension must be m + m/32")
    return m


def rescue_push(local_packed: torch.Tensor, rank: int, world: int, n: int, sat_word: torch.Tensor,
                recv: torch.Tensor, stream=None) -> torch.Tensor:
    """Rank ``rank``'s push of its packed local top-k [R, k + k/32] into the
    receive buffer ``recv`` [R, (k-1)//n, k + k/32] (in place); see the header."""
    lp = local_packed
    if lp.dtype != torch.int32 or lp.dim() != 2 or not lp.is_contiguous():
        raise ValueError("local_packed must be contiguous int32 [R, k + k/32]")
    rows = lp.shape[0]
    k = _packed_width(lp, "local_packed")
    sat_word = _int32_vec(sat_word, rows, "sat_word")
    if (recv.dtype != torch.int32 or not recv.is_contiguous() or
            tuple(recv.shape) != (rows, rescue_slots(n, k), k + k // 32)):
        raise ValueError(f"recv must be contiguous int32 [{rows}, {rescue_slots(n, k)}, {k + k // 32}]")
    _check(_lib.rescue_push(_dev(lp, "local_packed"), rank, world, rows, n, k,
                            _dev(sat_word, "sat_word"), _dev(recv, "recv"), _stream(stream)),
           "rescue_push")
    return recv


def merge_rescue_rank_major(gathered: torch.Tensor, recv: torch.Tensor, sat_word: torch.Tensor,
                            out: torch.Tensor, stream=None) -> torch.Tensor:
    """Second round of the packed merge: re-selects, in place in ``out`` [R, k]
    (round 1's ids), every row whose sat_word enters it; see the header."""
    if gathered.dtype != torch.int32 or gathered.dim() != 3 or not gathered.is_contiguous():
        raise ValueError("gathered must be contiguous int32 [W, R, n + n/32]")
    world, rows, _ = gathered.shape
    n = _packed_width(gathered, "gathered")
    if out.dtype != torch.int32 or out.dim() != 2 or out.shape[0] != rows or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, k]")
    k = out.shape[1]
    sat_word = _int32_vec(sat_word, rows, "sat_word")
    if (recv.dtype != torch.int32 or not recv.is_contiguous() or
            tuple(recv.shape) != (rows, rescue_slots(n, k), k + k // 32)):
        raise ValueError(f"recv must be contiguous int32 [{rows}, {rescue_slots(n, k)}, {k + k // 32}]")
    _check(_lib.merge_rescue_rank_major(_dev(gathered, "gathered"), _dev(recv, "recv"), world, rows,
                                        n, k, _dev(sat_word, "sat_word"), _dev(out, "out"),
                                        _stream(stream)), "merge_rescue_rank_major")
    return out


def merge_select_row_major(gathered: torch.Tensor, k: int, out: torch.Tensor | None = None,
                           sat_word: torch.Tensor | None = None, want_sat: bool = True,
                           stream=None):
    """The packed select on row-major int32 [R, W, n + n/32]; returns (ids, sat_word)."""
    if gathered.dtype != torch.int32 or gathered.dim() != 3 or not gathered.is_contiguous():
        raise ValueError("gathered must be contiguous int32 [R, W, n + n/32]")
    rows, world, _ = gathered.shape
    n = _packed_width(gathered, "gathered")
    if out is None:
        out = _new((rows, k), torch.int32, gathered.device, stream)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, {k}]")
    if sat_word is None and want_sat:
        sat_word = _new((rows,), torch.int32, gathered.device, stream)
    _check(_lib.merge_select_row_major(_dev(gathered, "gathered"), world, rows, n, k, _dev(out, "out"),
                                       _opt(sat_word, "sat_word"), _stream(stream)),
           "merge_select_row_major")
    return out, sat_word


def merge_select_pairs_row_major(gathered_pairs: torch.Tensor, k: int, world: int,
                                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The pair select on row-major int32 [R, W * kc, 2]; returns ids [R, k]."""
    g = gathered_pairs
    if g.dtype != torch.int32 or g.dim() != 3 or g.shape[2] != 2 or not g.is_contiguous():
        raise ValueError("gathered_pairs must be contiguous int32 [R, W * kc, 2]")
    rows, wkc, _ = g.shape
    if world < 1 or wkc % world != 0:
        raise ValueError("the candidate dimension must be world * kc")
    if out is None:
        out = _new((rows, k), torch.int32, g.device, stream)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, {k}]")
    _check(_lib.merge_select_pairs_row_major(_dev(g, "gathered_pairs"), world, rows, wkc // world, k,
                                             _dev(out, "out"), _stream(stream)),
           "merge_select_pairs_row_major")
    return out


def emit_rows(ids: torch.Tensor, world: int, dcp_rank: int, req_id: torch.Tensor,
              block_table: torch.Tensor, block_size: int, stride_rows: int,
              rows_out: torch.Tensor | None = None, valid_out: torch.Tensor | None = None,
              stream=None):
    """This rank's owned physical KV rows of ``ids`` [R, k]; returns
    (rows_out [R, out_cols >= k], valid_out [R]); see emit_rows in the header."""
    if ids.dtype != torch.int32 or ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be contiguous int32 [R, k]")
    rows, k = ids.shape
    req_id = _int32_vec(req_id, rows, "req_id")
    if req_id is None:
        raise ValueError("req_id is required")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [Q, B_max] with unit column stride")
    table_rows, table_cols = block_table.shape
    ld_table = block_table.stride(0) if table_rows > 1 else table_cols
    if rows_out is None:
        rows_out = _new((rows, k), torch.int32, ids.device, stream)
    if rows_out.dtype != torch.int32 or rows_out.dim() != 2 or rows_out.shape[0] != rows or \
            rows_out.shape[1] < k or not rows_out.is_contiguous():
        raise ValueError(f"rows_out must be contiguous int32 [{rows}, >= {k}]")
    if valid_out is None:
        valid_out = _new((rows,), torch.int32, ids.device, stream)
    valid_out = _int32_vec(valid_out, rows, "valid_out")
    _check(_lib.emit_rows(_dev(ids, "ids"), rows, k, world, dcp_rank, _dev(req_id, "req_id"),
                          _dev(block_table, "block_table"), table_rows, table_cols, ld_table,
                          block_size, stride_rows, _dev(rows_out, "rows_out"), rows_out.shape[1],
                          _dev(valid_out, "valid_out"), _stream(stream)), "emit_rows")
    return rows_out, valid_out


def _kv_rows(rows, k, dcp_rank, req_id, block_table, block_size, stride_rows, rows_out, valid_out,
             device, stream):
    req_id = _int32_vec(req_id, rows, "req_id")
    if req_id is None:
        raise ValueError("req_id is required")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [Q, B_max] with unit column stride")
    table_rows, table_cols = block_table.shape
    ld_table = block_table.stride(0) if table_rows > 1 else table_cols
    if rows_out is None:
        rows_out = _new((rows, k), torch.int32, device, stream)
    if rows_out.dtype != torch.int32 or rows_out.dim() != 2 or rows_out.shape[0] != rows or \
            rows_out.shape[1] < k or not rows_out.is_contiguous():
        raise ValueError(f"rows_out must be contiguous int32 [{rows}, >= {k}]")
    if valid_out is None:
        valid_out = _new((rows,), torch.int32, device, stream)
    valid_out = _int32_vec(valid_out, rows, "valid_out")
    kv = _KvRows(dcp_rank, req_id.data_ptr(), block_table.data_ptr(), table_rows, table_cols, ld_table,
                 block_size, stride_rows, rows_out.data_ptr(), rows_out.shape[1], valid_out.data_ptr())
    return kv, rows_out, valid_out


def merge_select_rank_major_rows(gathered: torch.Tensor, k: int, dcp_rank: int, req_id: torch.Tensor,
                                 block_table: torch.Tensor, block_size: int, stride_rows: int,
                                 rows_out: torch.Tensor | None = None,
                                 valid_out: torch.Tensor | None = None,
                                 out_ids: torch.Tensor | None = None,
                                 sat_word: torch.Tensor | None = None, stream=None):
    """Packed select writing this rank's owned physical rows (and optionally
    ids / sat_word); returns (rows_out, valid_out, out_ids, sat_word)."""
    if gathered.dtype != torch.int32 or gathered.dim() != 3 or not gathered.is_contiguous():
        raise ValueError("gathered must be contiguous int32 [W, R, n + n/32]")
    world, rows, _ = gathered.shape
    n = _packed_width(gathered, "gathered")
    kv, rows_out, valid_out = _kv_rows(rows, k, dcp_rank, req_id, block_table, block_size, stride_rows,
                                       rows_out, valid_out, gathered.device, stream)
    if out_ids is not None and (out_ids.dtype != torch.int32 or tuple(out_ids.shape) != (rows, k) or
                                not out_ids.is_contiguous()):
        raise ValueError(f"out_ids must be contiguous int32 [{rows}, {k}]")
    sat_word = _int32_vec(sat_word, rows, "sat_word")
    _check(_lib.merge_select_rank_major_rows(_dev(gathered, "gathered"), world, rows, n, k,
                                             ctypes.byref(kv), _opt(out_ids, "out_ids"),
                                             _opt(sat_word, "sat_word"), _stream(stream)),
           "merge_select_rank_major_rows")
    return rows_out, valid_out, out_ids, sat_word


def merge_rescue_rank_major_rows(gathered: torch.Tensor, recv: torch.Tensor, sat_word: torch.Tensor,
                                 k: int, dcp_rank: int, req_id: torch.Tensor,
                                 block_table: torch.Tensor, block_size: int, stride_rows: int,
                                 rows_out: torch.Tensor, valid_out: torch.Tensor,
                                 out_ids: torch.Tensor | None = None, stream=None):
    """Second round rewriting the owned rows (and optionally ids) of the rows
    that enter it, in place; returns (rows_out, valid_out)."""
    if gathered.dtype != torch.int32 or gathered.dim() != 3 or not gathered.is_contiguous():
        raise ValueError("gathered must be contiguous int32 [W, R, n + n/32]")
    world, rows, _ = gathered.shape
    n = _packed_width(gathered, "gathered")
    kv, rows_out, valid_out = _kv_rows(rows, k, dcp_rank, req_id, block_table, block_size, stride_rows,
                                       rows_out, valid_out, gathered.device, stream)
    sat_word = _int32_vec(sat_word, rows, "sat_word")
    if (recv.dtype != torch.int32 or not recv.is_contiguous() or
            tuple(recv.shape) != (rows, rescue_slots(n, k), k + k // 32)):
        raise ValueError(f"recv must be contiguous int32 [{rows}, {rescue_slots(n, k)}, {k + k // 32}]")
    if out_ids is not None and (out_ids.dtype != torch.int32 or tuple(out_ids.shape) != (rows, k) or
                                not out_ids.is_contiguous()):
        raise ValueError(f"out_ids must be contiguous int32 [{rows}, {k}]")
    _check(_lib.merge_rescue_rank_major_rows(_dev(gathered, "gathered"), _dev(recv, "recv"), world, rows,
                                             n, k, _dev(sat_word, "sat_word"), ctypes.byref(kv),
                                             _opt(out_ids, "out_ids"), _stream(stream)),
           "merge_rescue_rank_major_rows")
    return rows_out, valid_out


def pack_pairs(logits: torch.Tensor, local_idx: torch.Tensor, rank: int, world: int,
               row_ends: torch.Tensor | None = None, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """(score bits, gid) pairs int32 [rows, kc, 2]; see pack_pairs in the header."""
    if logits.dtype != torch.float32:
        raise TypeError("logits must be float32")
    rows, cols, ld = _rows_ld(logits, "logits")
    if local_idx.dtype != torch.int32:
        raise TypeError("local_idx must be int32")
    r2, kc, ld_idx = _rows_ld(local_idx, "local_idx")
    if r2 != rows:
        raise ValueError("local_idx must have one row per logits row")
    if rows <= 1:
        ld_idx = max(ld_idx, kc)
    row_ends = _int32_vec(row_ends, rows, "row_ends")
    if out is None:
        out = _new((rows, kc, 2), torch.int32, logits.device, stream)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, kc, 2) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, {kc}, 2]")
    _check(_lib.pack_pairs(_dev(logits, "logits"), rows, cols, ld, _dev(local_idx, "local_idx"), kc,
                           ld_idx, _opt(row_ends, "row_ends"), rank, world, _dev(out, "out"),
                           _stream(stream)), "pack_pairs")
    return out


def merge_select_pairs_rank_major(gathered_pairs: torch.Tensor, k: int,
                                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Select from int32 [W, R, kc, 2] read in place; returns ids [R, k]."""
    g = gathered_pairs
    if g.dtype != torch.int32 or g.dim() != 4 or g.shape[3] != 2 or not g.is_contiguous():
        raise ValueError("gathered_pairs must be contiguous int32 [W, R, kc, 2]")
    world, rows, kc, _ = g.shape
    if out is None:
        out = _new((rows, k), torch.int32, g.device, stream)
    if out.dtype != torch.int32 or tuple(out.shape) != (rows, k) or not out.is_contiguous():
        raise ValueError(f"out must be contiguous int32 [{rows}, {k}]")
    _check(_lib.merge_select_pairs_rank_major(_dev(g, "gathered_pairs"), world, rows, kc, k,
                                              _dev(out, "out"), _stream(stream)),
           "merge_select_pairs_rank_major")
    return out


def _launch(fn, where: str, device: torch.device, stream, *args) -> None:
    """Calls ``fn(*args, stream)`` with ``device`` current."""
    if stream is None:
        s = _current(device)
    else:
        if stream.device != device:
            raise ValueError(f"{where}: stream must belong to the device of the tensors")
        s = stream.cuda_stream
    if device.index == torch.cuda.current_device():
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != RTS_OK:
        raise RtsError(status, where)


def _no_grad(where: str, *tensors) -> None:
    """Refuses inputs whose gradients a caller would wait for in vain."""
    for t in tensors:
        if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            raise ValueError(f"{where} has no backward pass: call it under torch.no_grad(), or detach its inputs")


def _on(device: torch.device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"all tensors must be on {device}, one is on {t.device}")


def _gpu(t, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _out(t, shape, dtype, device, name: str, stream) -> torch.Tensor:
    """A caller's output tensor, checked, or a new one."""
    if t is None:
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=device)
        t = _new(shape, dtype, device, stream)
    elif t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {device}")
    return t


def _scratch(workspace, need: int, device, stream):
    """(tensor or None, bytes) of a call's workspace argument."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a GPU tensor')
        if not need:
            return None, 0
        return _new(need, torch.uint8, device, stream, returned=False), need
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of q")
    return workspace, workspace.numel() * workspace.element_size()


def _too_large(name: str, bits: int):
    """For numbers that ctypes would cut to their low bits."""
    return ValueError(f"{name} must be below 2^{bits - 1}")


def _pages(block_size: int, stride_rows) -> tuple:
    """(tokens, physical rows) of a block."""
    if not -0x80000000 <= block_size <= 0x7FFFFFFF:
        raise _too_large("block_size", 32)
    if stride_rows is None:
        return block_size, block_size
    if not -2 ** 63 <= stride_rows < 2 ** 63:
        raise _too_large("stride_rows", 64)
    return block_size, stride_rows


def _table(block_table: torch.Tensor):
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [Q, B_max] with unit column stride")
    (rows, cols), (ld, step) = block_table.shape, block_table.stride()
    if cols > 1 and rows > 0 and step != 1:
        raise ValueError("block_table must be int32 [Q, B_max] with unit column stride")
    if cols > 0x7FFFFFFF:
        raise _too_large("the width of block_table", 32)
    return rows, cols, (ld if rows > 1 and cols > 0 else cols)


def _int32_all(t: torch.Tensor, name: str) -> int:
    """The length of a contiguous int32 vector."""
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector")
    return t.shape[0]


class SlotMap(NamedTuple):
    """What assign_slots returns, int32 each; see assign_slots in the header."""
    query_starts: torch.Tensor  # [Q + 1]
    req_id: torch.Tensor        # [tokens]
    row_ends: torch.Tensor      # [tokens]
    slots: torch.Tensor         # [tokens]
    used: torch.Tensor          # [1]


def assign_slots(ctx_lens: torch.Tensor, new_lens: torch.Tensor, tokens: int, block_table: torch.Tensor,
                 free_blocks: torch.Tensor, block_size: int, stride_rows: int | None = None,
                 out: SlotMap | None = None, stream=None) -> SlotMap:
    """Places a batch's new tokens in the paged cache: extends ``block_table`` [Q, B_max] in
    place from ``free_blocks`` and returns the batch's SlotMap; see assign_slots in the header.

    ``stride_rows`` defaults to ``block_size``."""
    device = _gpu(ctx_lens, "ctx_lens")
    reqs, n_free = _int32_all(ctx_lens, "ctx_lens"), _int32_all(free_blocks, "free_blocks")
    table_rows, table_cols, ld_table = _table(block_table)
    if _int32_all(new_lens, "new_lens") != reqs or table_rows != reqs:
        raise ValueError("new_lens and block_table must have one entry per request")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    _on(device, new_lens, block_table, free_blocks)
    if out is None:
        flat = _new(reqs + 2 + 3 * tokens, torch.int32, device, stream)
        out = SlotMap(*torch.split_with_sizes(flat, (reqs + 1, tokens, tokens, tokens, 1)))
    else:
        for name, t, n in zip(SlotMap._fields, out, (reqs + 1, tokens, tokens, tokens, 1)):
            _out(t, (n,), torch.int32, device, name, stream)
    _launch(_lib.assign_slots, "assign_slots", device, stream, ctx_lens.data_ptr(),
            new_lens.data_ptr(), reqs, tokens, *_pages(block_size, stride_rows),
            free_blocks.data_ptr(), n_free, block_table.data_ptr(), table_cols, ld_table,
            out.query_starts.data_ptr(), out.req_id.data_ptr(), out.row_ends.data_ptr(),
            out.slots.data_ptr(), out.used.data_ptr())
    return out


_INDEX_DTYPES = {torch.bfloat16: RTS_BF16, torch.float8_e4m3fn: RTS_E4M3}
_FLOAT_DTYPES = {torch.float32: RTS_F32, torch.bfloat16: RTS_BF16}


def _logits_inputs(q, keys, weights, key_scales, row_ends, out, out_dtype, cols, stream):
    """What indexer_logits and indexer_logits_paged check alike."""
    _no_grad("indexer_logits", q, keys, weights, key_scales)
    device = _gpu(q, "q")
    if q.dtype not in _INDEX_DTYPES or keys.dtype != q.dtype:
        raise TypeError("q and keys must both be bfloat16 or both float8_e4m3fn")
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, dim] with contiguous heads")
    (rows, heads, dim), (ld_q, head_step, step) = q.shape, q.stride()
    if step != 1 or (heads > 1 and head_step != dim):
        raise ValueError("q must be [rows, heads, dim] with contiguous heads")
    n_keys, kdim, ld_keys = _rows_ld(keys, "keys")
    if kdim != dim:
        raise ValueError("q and keys must have the same last dimension")
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    w_rows, w_cols, ld_w = _rows_ld(weights, "weights")
    if (w_rows, w_cols) != (rows, heads):
        raise ValueError(f"weights must be [{rows}, {heads}]")
    if key_scales is not None and (key_scales.dtype != torch.float32 or key_scales.dim() != 1 or
                                   key_scales.shape[0] != n_keys or not key_scales.is_contiguous()):
        raise ValueError(f"key_scales must be a contiguous float32 vector of {n_keys} entries")
    row_ends = _int32_vec(row_ends, rows, "row_ends")
    if out is None:
        if out_dtype not in _FLOAT_DTYPES:
            raise TypeError("out_dtype must be float32 or bfloat16")
        out = _new((rows, cols), out_dtype, device, stream)
    if out.dtype not in _FLOAT_DTYPES:
        raise TypeError("out must be float32 or bfloat16")
    out_rows, out_cols, ld_out = _rows_ld(out, "out")
    if out_rows < rows or out_cols < cols:
        raise ValueError(f"out must hold at least [{rows}, {cols}] (got {tuple(out.shape)})")
    _on(device, keys, weights, key_scales, row_ends, out)
    if rows <= 1:
        ld_q = heads * dim
        ld_out = max(ld_out, cols)
    return device, rows, heads, dim, ld_q, n_keys, ld_keys, ld_w, row_ends, out, ld_out


def _ptr(t):
    return None if t is None else t.data_ptr()


def indexer_logits(q: torch.Tensor, keys: torch.Tensor, weights: torch.Tensor,
                   key_scales: torch.Tensor | None = None, row_ends: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """The logits [rows, cols] that topk_rows selects from: for ``q`` [rows, heads, dim], ``keys``
    [cols, dim] and ``weights`` [rows, heads], the weighted sum over heads of relu(q . k), times the
    key's scale; see indexer_logits in the header.  Columns at or past a row's end are not written.
    Without a backward pass: inputs that require gradients are refused."""
    cols = keys.shape[0]
    device, rows, heads, dim, ld_q, _, ld_keys, ld_w, row_ends, out, ld_out = _logits_inputs(
        q, keys, weights, key_scales, row_ends, out, out_dtype, cols, stream)
    _launch(_lib.indexer_logits, "indexer_logits", device, stream, q.data_ptr(),
            _INDEX_DTYPES[q.dtype], rows, heads, dim, ld_q, keys.data_ptr(), cols, ld_keys,
            weights.data_ptr(), ld_w, _ptr(key_scales), _ptr(row_ends), out.data_ptr(),
            _FLOAT_DTYPES[out.dtype], ld_out)
    return out


def indexer_logits_paged(q: torch.Tensor, key_cache: torch.Tensor, weights: torch.Tensor,
                         req_id: torch.Tensor, row_ends: torch.Tensor, block_table: torch.Tensor,
                         block_size: int, cols: int, key_scales: torch.Tensor | None = None,
                         stride_rows: int | None = None, out: torch.Tensor | None = None,
                         out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """indexer_logits over the paged ``key_cache`` [cache_rows, dim] of each token's request (the
    ``req_id`` and ``row_ends`` of assign_slots); see indexer_logits_paged in the header.  Without a
    backward pass, as indexer_logits."""
    if not 0 <= cols < 2 ** 63:
        raise ValueError("cols must not be negative, and below 2^63")
    device, rows, heads, dim, ld_q, n_keys, ld_keys, ld_w, row_ends, out, ld_out = _logits_inputs(
        q, key_cache, weights, key_scales, row_ends, out, out_dtype, cols, stream)
    req_id = _int32_vec(req_id, rows, "req_id")
    if req_id is None or row_ends is None:
        raise ValueError("req_id and row_ends are required")
    table_rows, table_cols, ld_table = _table(block_table)
    _on(device, req_id, block_table)
    _launch(_lib.indexer_logits_paged, "indexer_logits_paged", device, stream, q.data_ptr(),
            _INDEX_DTYPES[q.dtype], rows, heads, dim, ld_q, key_cache.data_ptr(), n_keys, ld_keys,
            weights.data_ptr(), ld_w, _ptr(key_scales), req_id.data_ptr(), row_ends.data_ptr(),
            block_table.data_ptr(), table_rows, table_cols, ld_table,
            *_pages(block_size, stride_rows), cols, out.data_ptr(),
            _FLOAT_DTYPES[out.dtype], ld_out)
    return out


def _attend_inputs(q, cache, d_latent, out, lse, stream):
    """What latent_attend_rows and latent_attend_paged check alike."""
    _no_grad("latent attention", q, cache)
    device = _gpu(q, "q")
    if q.dtype != torch.bfloat16 or cache.dtype != torch.bfloat16:
        raise TypeError("q and cache must be bfloat16")
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, d_latent + d_rope] with unit element stride")
    (rows, heads, d), (ld_q, ld_head, step) = q.shape, q.stride()
    if step != 1:
        raise ValueError("q must be [rows, heads, d_latent + d_rope] with unit element stride")
    cache_rows, cd, ld_cache = _rows_ld(cache, "cache")
    if cd != d or not 0 < d_latent <= d:
        raise ValueError("q and cache must have the same last dimension, at least d_latent")
    ld_head = ld_head if heads > 1 else d
    ld_q = ld_q if rows > 1 else heads * d
    out = _out(out, (rows, heads, d_latent), torch.bfloat16, device, "out", stream)
    lse = _out(lse, (rows, heads), torch.float32, device, "lse", stream)
    _on(device, cache)
    return device, rows, heads, d, cache_rows, ld_cache, ld_q, ld_head, out, lse


def latent_attend_rows_workspace_size(rows: int, heads: int, d_latent: int, k: int) -> int:
    return int(_lib.latent_attend_rows_workspace_size(rows, heads, d_latent, k))


def latent_attend_rows(q: torch.Tensor, cache: torch.Tensor, ids: torch.Tensor, scale: float,
                       d_latent: int = 512, counts: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace="auto", stream=None):
    """Attention of ``q`` [rows, heads, d] over the rows ``ids`` [rows, k] of the latent ``cache``
    [cache_rows, d], whose first ``d_latent`` elements are the values; ``ids`` and ``counts`` as emit_rows
    writes them (rows_out, valid_out).  Returns (out [rows, heads, d_latent], lse [rows, heads]); see
    latent_attend_rows in the header.  ``workspace`` as in topk_rows.  Without a backward pass: inputs that
    require gradients are refused."""
    device, rows, heads, d, cache_rows, ld_cache, ld_q, ld_head, out, lse = _attend_inputs(
        q, cache, d_latent, out, lse, stream)
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    id_rows, k, ld_ids = _rows_ld(ids, "ids")
    if k > 0x7FFFFFFF:
        raise _too_large("the width of ids", 32)
    if id_rows != rows:
        raise ValueError("ids must have one row per query row")
    if rows <= 1:
        ld_ids = max(ld_ids, k)
    counts = _int32_vec(counts, rows, "counts")
    _on(device, ids, counts)
    ws, ws_bytes = _scratch(workspace, latent_attend_rows_workspace_size(rows, heads, d_latent, k)
                            if isinstance(workspace, str) else 0, device, stream)
    _launch(_lib.latent_attend_rows, "latent_attend_rows", device, stream, q.data_ptr(), rows, heads,
            d_latent, d - d_latent, ld_q, ld_head, cache.data_ptr(), cache_rows, ld_cache, ids.data_ptr(), k,
            ld_ids, _ptr(counts), scale, out.data_ptr(), lse.data_ptr(), _ptr(ws), ws_bytes)
    return out, lse


def latent_attend_paged_workspace_size(tokens: int, reqs: int, heads: int, d_latent: int,
                                       max_len: int) -> int:
    return int(_lib.latent_attend_paged_workspace_size(tokens, reqs, heads, d_latent, max_len))


def latent_attend_paged(q: torch.Tensor, cache: torch.Tensor, query_starts: torch.Tensor,
                        ctx_lens: torch.Tensor, block_table: torch.Tensor, block_size: int, scale: float,
                        d_latent: int = 512, stride_rows: int | None = None,
                        tree: torch.Tensor | None = None, max_len: int | None = None,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        workspace="auto", stream=None):
    """Attention of a batch's new tokens ``q`` [tokens, heads, d] over their requests' whole paged
    latent cache, causal or by the ancestor masks ``tree`` (int64 or uint64 [tokens], bit j: draft j of the
    request is seen); ``query_starts`` as assign_slots writes it.  ``max_len`` bounds the requests' lengths
    and only steers the split (default: what the table holds).  Returns (out, lse); see
    latent_attend_paged in the header.  ``workspace`` as in topk_rows.  Without a backward pass, as
    latent_attend_rows."""
    device, tokens, heads, d, cache_rows, ld_cache, ld_q, ld_head, out, lse = _attend_inputs(
        q, cache, d_latent, out, lse, stream)
    table_rows, table_cols, ld_table = _table(block_table)
    ctx_lens = _int32_vec(ctx_lens, table_rows, "ctx_lens")
    query_starts = _int32_vec(query_starts, table_rows + 1, "query_starts")
    if ctx_lens is None or query_starts is None:
        raise ValueError("query_starts and ctx_lens are required")
    if tree is not None and (tree.dtype not in (torch.int64, torch.uint64) or tree.dim() != 1 or
                             tree.shape[0] < tokens or not tree.is_contiguous()):
        raise ValueError(f"tree must be a contiguous 64-bit vector of >= {tokens} entries")
    pages = _pages(block_size, stride_rows)
    if max_len is None:
        max_len = table_cols * block_size
    elif max_len >= 2 ** 63:
        raise _too_large("max_len", 64)
    _on(device, query_starts, ctx_lens, block_table, tree)
    ws, ws_bytes = _scratch(workspace,
                            latent_attend_paged_workspace_size(tokens, table_rows, heads, d_latent, max_len)
                            if isinstance(workspace, str) else 0, device, stream)
    _launch(_lib.latent_attend_paged, "latent_attend_paged", device, stream, q.data_ptr(), tokens,
            heads, d_latent, d - d_latent, ld_q, ld_head, cache.data_ptr(), cache_rows, ld_cache,
            query_starts.data_ptr(), ctx_lens.data_ptr(), table_rows, _ptr(tree), block_table.data_ptr(),
            table_cols, ld_table, *pages, max_len, scale, out.data_ptr(), lse.data_ptr(), _ptr(ws), ws_bytes)
    return out, lse


def merge_attend_rank_major(parts: torch.Tensor, lse: torch.Tensor, out: torch.Tensor | None = None,
                            out_dtype=None, out_lse: torch.Tensor | None = None, stream=None):
    """Joins the partial attentions ``parts`` [W, rows, heads, dim] of W ranks by their ``lse``
    [W, rows, heads]; returns (out [rows, heads, dim], lse [rows, heads]); see merge_attend_rank_major in
    the header.  ``out_dtype`` defaults to the parts' type.  Without a backward pass."""
    _no_grad("merge_attend_rank_major", parts, lse)
    device = _gpu(parts, "parts")
    if parts.dtype not in _FLOAT_DTYPES:
        raise TypeError("parts must be float32 or bfloat16")
    if parts.dim() != 4 or not parts.is_contiguous():
        raise ValueError("parts must be contiguous [W, rows, heads, dim]")
    world, rows, heads, dim = parts.shape
    if lse.dtype != torch.float32 or lse.shape != (world, rows, heads) or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous float32 [{world}, {rows}, {heads}]")
    if out_dtype is None:
        out_dtype = parts.dtype if out is None else out.dtype
    if out_dtype not in _FLOAT_DTYPES:
        raise TypeError("out must be float32 or bfloat16")
    out = _out(out, (rows, heads, dim), out_dtype, device, "out", stream)
    out_lse = _out(out_lse, (rows, heads), torch.float32, device, "out_lse", stream)
    _on(device, lse)
    _launch(_lib.merge_attend_rank_major, "merge_attend_rank_major", device, stream, parts.data_ptr(),
            _FLOAT_DTYPES[parts.dtype], lse.data_ptr(), world, rows, heads, dim, out.data_ptr(),
            _FLOAT_DTYPES[out.dtype], out_lse.data_ptr())
    return out, out_lse


# Workspace sizes by the sizes of a call: a query costs a microsecond, a step's calls make the same ones.
_sizes = functools.lru_cache(maxsize=1024)
_beam_bytes = _sizes(lambda *a: int(_lib.beam_select_workspace_size(*a)))
_fork_bytes = _sizes(lambda *a: int(_lib.fork_blocks_workspace_size(*a)))
_compact_bytes = _sizes(lambda *a: int(_lib.compact_blocks_workspace_size(*a)))
_kv_bytes = _sizes(lambda *a: int(_lib.kv_attend_paged_workspace_size(*a)))


class BeamStep(NamedTuple):
    """What beam_select returns; see beam_select in the header."""
    scores: torch.Tensor        # float32 [G, k]
    parents: torch.Tensor       # int32 [G, k]
    tokens: torch.Tensor        # int32 [G, k]
    ended: torch.Tensor | None  # float32 [G, beams], None without an eos


def beam_select_workspace_size(dtype, groups: int, beams: int, vocab: int, k: int) -> int:
    dt = RTS_BF16 if dtype in (torch.bfloat16, RTS_BF16) else RTS_F32
    return int(_lib.beam_select_workspace_size(dt, groups, beams, vocab, k))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, k: int, eos: int = -1, out: BeamStep | None = None,
                workspace="auto", stream=None) -> BeamStep:
    """The k best continuations of each group's beams by ``scores`` [G, beams] plus the log-softmax of the beams'
    ``logits`` [G * beams, vocab] (float32 or bfloat16), the token ``eos`` apart (-1: none); see beam_select in the
    header.  ``workspace``: "auto" (allocated here) or a GPU tensor.  Without a backward pass: inputs that require
    gradients are refused."""
    _no_grad("beam_select", logits, scores)
    device = _gpu(logits, "logits")
    if logits.dtype not in _FLOAT_DTYPES:
        raise TypeError("logits must be float32 or bfloat16")
    rows, vocab, ld = _rows_ld(logits, "logits")
    if scores.dtype != torch.float32 or scores.dim() != 2 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous float32 [G, beams]")
    groups, beams = scores.shape
    if groups * beams != rows:
        raise ValueError("logits must have one row per score")
    if not -0x80000000 <= k <= 0x7FFFFFFF or not -0x80000000 <= eos <= 0x7FFFFFFF:
        raise _too_large("k and eos", 32)
    _on(device, scores)
    dt = _FLOAT_DTYPES[logits.dtype]
    if out is None:
        if k < 1 or beams < 1:
            raise RtsError(RTS_EINVAL, "beam_select")
        best, parents, tokens = _new((3, groups, k), torch.int32, device, stream).unbind(0)
        ended = None
        if eos >= 0:
            ended = torch.empty_like(scores) if stream is None else _new((groups, beams), torch.float32, device, stream)
        out = BeamStep(best.view(torch.float32), parents, tokens, ended)
    else:
        for name, t, d in zip(BeamStep._fields, out, (torch.float32, torch.int32, torch.int32)):
            _out(t, (groups, k), d, device, name, stream)
        if eos >= 0:
            _out(out.ended, (groups, beams), torch.float32, device, "ended", stream)
        elif out.ended is not None:
            raise ValueError("ended is written only with an eos")
    if workspace is None:
        raise ValueError('workspace must be "auto" or a GPU tensor')
    ws, ws_bytes = _scratch(workspace, _beam_bytes(dt, groups, beams, vocab, k)
                            if isinstance(workspace, str) else 0, device, stream)
    _launch(_lib.beam_select, "beam_select", device, stream, logits.data_ptr(), dt, groups, beams, vocab, ld,
            scores.data_ptr(), k, eos, out.scores.data_ptr(), out.parents.data_ptr(), out.tokens.data_ptr(),
            _ptr(out.ended), _ptr(ws), ws_bytes)
    return out


class Fork(NamedTuple):
    """What fork_blocks returns, int32 each; see fork_blocks in the header."""
    block_table: torch.Tensor  # [rows, B_max]
    ctx_lens: torch.Tensor     # [rows]
    copies: torch.Tensor       # [rows, 2]: pairs for copy_blocks, then -1
    free_blocks: torch.Tensor  # [n_free]: a list for assign_slots, then -1
    counts: torch.Tensor       # [2]: free blocks, blocks wanted


class Compaction(NamedTuple):
    """What compact_blocks returns, int32 each; see compact_blocks in the header."""
    block_table: torch.Tensor  # [rows, B_max]
    moves: torch.Tensor        # [max_moves, 2]: pairs for copy_blocks, then -1
    free_blocks: torch.Tensor  # [n_free], then -1
    counts: torch.Tensor       # [2]: free blocks, moves in all


def _pool(pool_blocks: int, held, n_free, block_size: int):
    """(n_free, pointer to held, block size) of a pool, checked."""
    if not 0 <= pool_blocks <= 0x7FFFFFFF:
        raise ValueError("pool_blocks must not be negative, and below 2^31")
    if held is not None and (held.dtype not in (torch.bool, torch.uint8) or held.shape != (pool_blocks,) or
                             not held.is_contiguous()):
        raise ValueError(f"held must be a contiguous bool or uint8 vector of {pool_blocks} entries")
    if n_free is None:
        n_free = pool_blocks
    if not 0 <= n_free < 2 ** 31:
        raise ValueError("n_free must not be negative, and below 2^31")
    return n_free, _ptr(held), _pages(block_size, None)[0]


def _named_out(out, shapes, device, stream):
    """A caller's int32 outputs of a block call, checked."""
    for name, t, shape in zip(out._fields, out, shapes):
        _out(t, shape, torch.int32, device, name, stream)
    return out


def fork_blocks(block_table: torch.Tensor, ctx_lens: torch.Tensor, parents: torch.Tensor, block_size: int,
                pool_blocks: int, held: torch.Tensor | None = None, n_free: int | None = None,
                out: Fork | None = None, workspace="auto", stream=None) -> Fork:
    """The block table whose row i continues row ``parents[i]`` of ``block_table`` (the parents of beam_select; -1:
    an empty row), with fresh blocks where rows would write into the same one; see fork_blocks in the header.
    ``copies`` are the caller's to make (copy_blocks).  ``n_free``: length of the list of free blocks (default: the
    pool's).  ``workspace`` as in topk_rows."""
    device = _gpu(block_table, "block_table")
    rows_in, cols, ld = _table(block_table)
    if _int32_all(ctx_lens, "ctx_lens") != rows_in:
        raise ValueError("ctx_lens must have one entry per row of block_table")
    rows = _int32_all(parents, "parents")
    n_free, held_ptr, block_size = _pool(pool_blocks, held, n_free, block_size)
    _on(device, ctx_lens, parents, held)
    if out is None:
        copies, counts, table, lens, free = torch.split_with_sizes(
            _new(rows * (cols + 3) + n_free + 2, torch.int32, device, stream),
            (rows * 2, 2, rows * cols, rows, n_free))
        out = Fork(table.view(rows, cols), lens, copies.view(rows, 2), free, counts)
    else:
        _named_out(out, ((rows, cols), (rows,), (rows, 2), (n_free,), (2,)), device, stream)
    ws, ws_bytes = _scratch(workspace, _fork_bytes(rows_in, cols, pool_blocks)
                            if isinstance(workspace, str) else 0, device, stream)
    _launch(_lib.fork_blocks, "fork_blocks", device, stream, block_table.data_ptr(), rows_in, cols, ld,
            ctx_lens.data_ptr(), parents.data_ptr(), rows, block_size, pool_blocks, held_ptr,
            out.block_table.data_ptr(), cols, out.ctx_lens.data_ptr(), out.copies.data_ptr(),
            out.free_blocks.data_ptr(), n_free, out.counts.data_ptr(), _ptr(ws), ws_bytes)
    return out


def compact_blocks(block_table: torch.Tensor, ctx_lens: torch.Tensor, block_size: int, pool_blocks: int,
                   held: torch.Tensor | None = None, max_moves: int | None = None, n_free: int | None = None,
                   out: Compaction | None = None, workspace="auto", stream=None) -> Compaction:
    """Moves (pairs for copy_blocks) that bring the blocks in use to the lowest ids, and the block table after
    them; see compact_blocks in the header.  ``max_moves`` defaults to half of the pool, which is always enough;
    ``workspace`` as in topk_rows."""
    device = _gpu(block_table, "block_table")
    rows, cols, ld = _table(block_table)
    if _int32_all(ctx_lens, "ctx_lens") != rows:
        raise ValueError("ctx_lens must have one entry per row of block_table")
    n_free, held_ptr, block_size = _pool(pool_blocks, held, n_free, block_size)
    if max_moves is None:
        max_moves = pool_blocks // 2
    if not 0 <= max_moves < 2 ** 31:
        raise ValueError("max_moves must not be negative, and below 2^31")
    _on(device, ctx_lens, held)
    if out is None:
        moves, counts, table, free = torch.split_with_sizes(
            _new(rows * cols + max_moves * 2 + n_free + 2, torch.int32, device, stream),
            (max_moves * 2, 2, rows * cols, n_free))
        out = Compaction(table.view(rows, cols), moves.view(max_moves, 2), free, counts)
    else:
        _named_out(out, ((rows, cols), (max_moves, 2), (n_free,), (2,)), device, stream)
    ws, ws_bytes = _scratch(workspace, _compact_bytes(rows, cols, pool_blocks)
                            if isinstance(workspace, str) else 0, device, stream)
    _launch(_lib.compact_blocks, "compact_blocks", device, stream, block_table.data_ptr(), rows, cols, ld,
            ctx_lens.data_ptr(), block_size, pool_blocks, held_ptr, out.block_table.data_ptr(), cols,
            out.moves.data_ptr(), max_moves, out.free_blocks.data_ptr(), n_free, out.counts.data_ptr(), _ptr(ws), ws_bytes)
    return out


def copy_blocks(caches, pairs: torch.Tensor, block_size: int, stride_rows: int | None = None, stream=None) -> None:
    """Copies blocks within each of ``caches`` (one tensor or any iterable of them, [cache_rows, ...] of any type, a row contiguous) by the
    ``pairs`` int32 [n, 2] of (from, to), -1 skipped, in place; see copy_blocks in the header.  ``stride_rows``
    defaults to ``block_size``."""
    device = _gpu(pairs, "pairs")
    caches = (caches,) if isinstance(caches, torch.Tensor) else tuple(caches)  # walked more than once
    if pairs.dtype != torch.int32 or pairs.dim() != 2 or pairs.shape[1] != 2 or not pairs.is_contiguous():
        raise ValueError("pairs must be contiguous int32 [n, 2]")
    pages = _pages(block_size, stride_rows)
    _on(device, *caches)
    _no_grad("copy_blocks", *caches)
    described = []
    for t in caches:
        if t.dim() < 1:
            raise ValueError("a cache must be [cache_rows, ...]")
        n, esz = 1, t.element_size()
        for size, step in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
            if size != 1 and step != n:
                raise ValueError("a cache's rows must be contiguous")
            n *= size
        ld = t.stride(0) if t.shape[0] > 1 else n
        if ld < n:
            raise ValueError("a cache's rows must not overlap")
        if n > 0:
            described.append((t.data_ptr(), t.shape[0], n * esz, ld * esz))
    n_pairs, where = pairs.shape[0], pairs.data_ptr()
    for at in range(0, len(described), 64):
        some = described[at:at + 64]
        _launch(_lib.copy_blocks, "copy_blocks", device, stream, (_Cache * len(some))(*some), len(some), where, n_pairs,
                *pages)


def kv_attend_paged_workspace_size(dtype, rows: int, heads: int, kv_heads: int, dim: int, max_len: int,
                                   window: int = 0) -> int:
    dt = RTS_E4M3 if dtype in (torch.float8_e4m3fn, RTS_E4M3) else RTS_BF16
    return int(_lib.kv_attend_paged_workspace_size(rows, heads, kv_heads, dim, dt, max_len, window))


def kv_attend_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, req_id: torch.Tensor,
                    row_ends: torch.Tensor, block_table: torch.Tensor, block_size: int, scale: float,
                    k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None, window: int = 0,
                    stride_rows: int | None = None, max_len: int | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace="auto", stream=None):
    """Attention of new tokens ``q`` [rows, heads, dim] over their requests' paged ``k_cache`` and ``v_cache``
    [cache_rows, kv_heads, dim] (bfloat16, or float8_e4m3fn with ``k_scales`` and ``v_scales`` [kv_heads]), a token
    seeing the positions below its ``row_ends``, the last ``window`` of them where that is not 0; ``req_id`` and
    ``row_ends`` as assign_slots writes them.  ``max_len`` bounds row_ends and only steers the split (default: what
    the table holds, which for short contexts in wide tables costs some microseconds).  Returns (out, lse); see kv_attend_paged in the header.  ``workspace`` as in topk_rows.
    Without a backward pass: inputs that require gradients are refused."""
    _no_grad("kv_attend_paged", q, k_cache, v_cache, k_scales, v_scales)
    device = _gpu(q, "q")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16")
    if k_cache.dtype not in _INDEX_DTYPES or v_cache.dtype != k_cache.dtype:
        raise TypeError("k_cache and v_cache must both be bfloat16 or both float8_e4m3fn")
    shape, steps, cache, cache_steps = q.shape, q.stride(), k_cache.shape, k_cache.stride()
    if len(shape) != 3 or len(cache) != 3 or steps[2] != 1 or cache_steps[2] != 1:
        raise ValueError("q must be [rows, heads, dim], the caches [cache_rows, kv_heads, dim], with unit element stride")
    if v_cache.shape != cache or v_cache.stride() != cache_steps and any(
            n > 1 and x != y for n, x, y in zip(cache, cache_steps, v_cache.stride())):
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    (rows, heads, dim), (ld_q, ld_qhead, _) = shape, steps
    (cache_rows, kv_heads, cdim), (ld_cache, ld_head, _) = cache, cache_steps
    if cdim != dim:
        raise ValueError("q and the caches must have the same last dimension")
    if heads > 0x7FFFFFFF or dim > 0x7FFFFFFF:
        raise _too_large("the sizes of q", 32)
    if kv_heads < 1 or heads % kv_heads != 0:
        raise ValueError("heads must be a multiple of kv_heads")
    ld_qhead = ld_qhead if heads > 1 else dim
    ld_q = ld_q if rows > 1 else heads * dim
    ld_head = ld_head if kv_heads > 1 else dim
    ld_cache = ld_cache if cache_rows > 1 else kv_heads * dim
    if k_scales is not None or v_scales is not None:
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None and (t.dtype != torch.float32 or t.shape != (kv_heads,) or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous float32 vector of {kv_heads} entries")
    req_id, row_ends = _int32_vec(req_id, rows, "req_id"), _int32_vec(row_ends, rows, "row_ends")
    if req_id is None or row_ends is None:
        raise ValueError("req_id and row_ends are required")
    table_rows, table_cols, ld_table = _table(block_table)
    pages = _pages(block_size, stride_rows)
    if max_len is None:
        max_len = table_cols * block_size
    if not 0 <= window < 2 ** 63 or max_len >= 2 ** 63:
        raise ValueError("window must not be negative, and window and max_len below 2^63")
    if out is None and stream is None and q.is_contiguous():
        out = torch.empty_like(q)  # two thirds of torch.empty's time
    else:
        out = _out(out, (rows, heads, dim), torch.bfloat16, device, "out", stream)
    lse = _out(lse, (rows, heads), torch.float32, device, "lse", stream)
    _on(device, k_cache, v_cache, k_scales, v_scales, req_id, row_ends, block_table)
    dt = _INDEX_DTYPES[k_cache.dtype]
    ws, ws_bytes = _scratch(workspace,
                            _kv_bytes(rows, heads, kv_heads, dim, dt, max_len, window)
                            if isinstance(workspace, str) else 0, device, stream)
    _launch(_lib.kv_attend_paged, "kv_attend_paged", device, stream, q.data_ptr(), rows, heads, ld_q, ld_qhead,
            k_cache.data_ptr(), v_cache.data_ptr(), dt, kv_heads, dim, cache_rows, ld_cache, ld_head, _ptr(k_scales),
            _ptr(v_scales), req_id.data_ptr(), row_ends.data_ptr(), block_table.data_ptr(), table_rows, table_cols,
            ld_table, *pages, window, max_len, scale, out.data_ptr(), lse.data_ptr(), _ptr(ws), ws_bytes)
    return out, lse


def raw_library() -> ctypes.CDLL:
    """The loaded shared library (for ABI-level tests)."""
    return _lib
