"""NVFP4-compressed MLA KV cache and sparse decode attention for GB300 (sm_103a).

Thin Python binding over the C ABI declared in ``include/nvfp4_mla.h``:
the functions below carry the C entry points' names and only marshal
arguments (torch tensors -> device pointers, the current CUDA stream).
With ``stream`` a call runs on that stream instead (a torch stream or a
handle): the caller orders it after what writes the arguments and before
what reads the results. Buffers that the call allocates are that stream's.
Every step of the computation runs in the library's CUDA kernels; if the
library is missing or the device is not an sm_103 part the calls raise.

Method: the Prime Inference post ("Prime Inference: Fast, Reliable Serving
for Frontier Open Models"), sections "Making room for low-latency decode"
(352-byte NVFP4 rows) and "Native NVFP4 sparse MLA decode kernel".
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _native

LATENT_DIM = 512
ROPE_DIM = 64
ROW_NVFP4_352 = 0
ROW_FP8_576 = 1
ROW_BYTES = {ROW_NVFP4_352: 352, ROW_FP8_576: 576}
INDEX_DIM = 128
INDEX_ROW_BYTES = 72

__all__ = [
    "LATENT_DIM", "ROPE_DIM", "ROW_NVFP4_352", "ROW_FP8_576", "ROW_BYTES", "NativeError",
    "nvfp4_mla_row_bytes", "nvfp4_mla_status_string", "nvfp4_mla_append",
    "sparse_mla_decode_num_splits", "sparse_mla_decode_workspace_size", "sparse_mla_decode",
    "nvfp4_mla_set_wait_limit",
    "sparse_mla_merge_states", "nvfp4_mla_staged_rows_per_q", "nvfp4_mla_stage_fp8",
    "staged_fp8_tables", "INDEX_DIM", "INDEX_ROW_BYTES", "nvfp4_mla_plan_step",
    "nvfp4_mla_truncate", "nvfp4_mla_index_append", "nvfp4_mla_index_read",
    "sparse_mla_select_workspace_size", "sparse_mla_select", "library_path",
]


class NativeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({nvfp4_mla_status_string(status)})")


def library_path() -> str:
    return _native.library_path()


def _lib():
    return _native.load()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the C ABI must be contiguous")
    return t.data_ptr()


# Handle of a device's current stream without a Stream object around it: 0.2 us instead of 3.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _launch_stream(stream) -> torch.cuda.Stream:
    if isinstance(stream, torch.cuda.Stream):
        return stream
    # torch would take the default stream's handle, 0, for none and make a new stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _scratch(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """A buffer of the launch stream: torch may hand out its memory again once ``stream`` is past
    what was enqueued on it, and it holds nothing that other streams' pending work still reads."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_launch_stream(stream)):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """The same for what a call returns, which the current stream will read: when it is dropped,
    its memory waits for the current stream's work too."""
    t = _scratch(shape, dtype, device, stream)
    if stream is not None:
        here = torch.cuda.current_stream(t.device)
        if here.cuda_stream != _launch_stream(stream).cuda_stream:
            t.record_stream(here)
    return t


def _check(status: int, where: str) -> None:
    if status != 0:
        raise NativeError(status, where)


def nvfp4_mla_row_bytes(row_format: int) -> int:
    return int(_lib().nvfp4_mla_row_bytes(row_format))


def nvfp4_mla_status_string(status: int) -> str:
    return _lib().nvfp4_mla_status_string(status).decode()


def nvfp4_mla_append(latent: torch.Tensor, rope: torch.Tensor, seq_ids: torch.Tensor,
                     positions: torch.Tensor, block_table: torch.Tensor, page_size: int,
                     cache: torch.Tensor, num_blocks: int, block_stride_bytes: int,
                     row_format: int = ROW_NVFP4_352, latent_scale: float = 1.0,
                     rope_scale: float = 1.0, invalid_count: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Quantize ``latent`` [n,512] / ``rope`` [n,64] (bf16) into their paged cache rows."""
    n = latent.shape[0] if latent.dim() else 0
    st = _lib().nvfp4_mla_append(
        _ptr(latent), _ptr(rope), _ptr(seq_ids), _ptr(positions), n, _ptr(block_table),
        block_table.shape[0], block_table.shape[1], page_size, _ptr(cache), num_blocks,
        block_stride_bytes, row_format, latent_scale, rope_scale, _ptr(invalid_count),
        _stream(stream))
    _check(st, "nvfp4_mla_append")


def sparse_mla_decode_num_splits(num_q: int, num_heads: int, topk: int) -> int:
    return int(_lib().sparse_mla_decode_num_splits(num_q, num_heads, topk))


def nvfp4_mla_set_wait_limit(cycles: int) -> None:
    """Bound (SM clock cycles) of the decode and selection kernels' internal waits; 0 = default."""
    _check(_lib().nvfp4_mla_set_wait_limit(int(cycles)), "nvfp4_mla_set_wait_limit")


def sparse_mla_decode_workspace_size(num_q: int, num_heads: int, topk: int,
                                     num_splits: int = 0) -> int:
    n = int(_lib().sparse_mla_decode_workspace_size(num_q, num_heads, topk, num_splits))
    if n == (1 << 64) - 1:
        raise ValueError("invalid decode shape")
    return n


def sparse_mla_decode(q_latent: torch.Tensor, q_rope: torch.Tensor, q_seq: torch.Tensor,
                      topk_idx: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      page_size: int, cache: torch.Tensor, num_blocks: int,
                      block_stride_bytes: int, row_format: int, sm_scale: float,
                      latent_scale: float = 1.0, rope_scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, out_fp32: bool = False,
                      lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                      invalid_count: Optional[torch.Tensor] = None, stream=None):
    """Sparse absorbed-MLA decode; returns (out [num_q,H,512], lse [num_q,H]).

    ``out`` / ``lse`` / ``workspace`` are allocated with torch when not given.
    """
    num_q, H = q_latent.shape[0], q_latent.shape[1]
    topk = topk_idx.shape[1]
    dev = q_latent.device
    if out is None:
        out = _result((num_q, H, LATENT_DIM), torch.float32 if out_fp32 else torch.bfloat16, dev,
                      stream)
    if lse is None:
        lse = _result((num_q, H), torch.float32, dev, stream)
    need = sparse_mla_decode_workspace_size(num_q, H, topk, num_splits) if num_q else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = _scratch(need, torch.uint8, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib().sparse_mla_decode(
        _ptr(q_latent), _ptr(q_rope), _ptr(q_seq), _ptr(topk_idx), num_q, H, topk,
        _ptr(block_table), block_table.shape[0], block_table.shape[1], _ptr(seq_lens), page_size,
        _ptr(cache), num_blocks, block_stride_bytes, row_format, sm_scale, latent_scale,
        rope_scale, _ptr(out), 1 if out_fp32 else 0, _ptr(lse), _ptr(workspace), ws_bytes,
        num_splits, _ptr(invalid_count), _stream(stream))
    _check(st, "sparse_mla_decode")
    return out, lse


def sparse_mla_merge_states(part_out: torch.Tensor, part_lse: torch.Tensor,
                            out: Optional[torch.Tensor] = None, out_fp32: bool = False,
                            lse: Optional[torch.Tensor] = None, stream=None):
    """Merge P partial attention states (fp32 [P,num_q,H,512], [P,num_q,H]);
    returns (out [num_q,H,512], lse [num_q,H])."""
    P, num_q, H = part_out.shape[0], part_out.shape[1], part_out.shape[2]
    dev = part_out.device
    if out is None:
        out = _result((num_q, H, LATENT_DIM), torch.float32 if out_fp32 else torch.bfloat16, dev,
                      stream)
    if lse is None:
        lse = _result((num_q, H), torch.float32, dev, stream)
    st = _lib().sparse_mla_merge_states(_ptr(part_out), _ptr(part_lse), P, num_q, H, _ptr(out),
                                        1 if out_fp32 else 0, _ptr(lse), _stream(stream))
    _check(st, "sparse_mla_merge_states")
    return out, lse

# ------------------------------------------------ staged-dequant comparison path
def nvfp4_mla_staged_rows_per_q(topk: int, page_size: int) -> int:
    """Staged FP8 rows per query token (topk rounded up to whole pages)."""
    n = int(_lib().nvfp4_mla_staged_rows_per_q(topk, page_size))
    if n == 0:
        raise ValueError("invalid topk or page_size")
    return n


def nvfp4_mla_stage_fp8(q_seq: torch.Tensor, topk_idx: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, page_size: int, cache: torch.Tensor,
                        num_blocks: int, block_stride_bytes: int, latent_scale: float = 1.0,
                        staged: Optional[torch.Tensor] = None,
                        staged_idx: Optional[torch.Tensor] = None,
                        invalid_count: Optional[torch.Tensor] = None, stream=None):
    """Selected NVFP4 rows re-encoded as FP8 rows; returns (staged, staged_idx).

    ``staged`` (uint8, num_q * R * 576 bytes) and ``staged_idx`` (int32
    [num_q, topk]) are allocated with torch when not given.
    """
    num_q, topk = topk_idx.shape[0], topk_idx.shape[1]
    dev = topk_idx.device
    R = nvfp4_mla_staged_rows_per_q(topk, page_size)
    if staged is None:
        staged = _result(max(num_q * R * ROW_BYTES[ROW_FP8_576], 16), torch.uint8, dev, stream)
    if staged_idx is None:
        staged_idx = _result((num_q, topk), torch.int32, dev, stream)
    st = _lib().nvfp4_mla_stage_fp8(
        _ptr(q_seq), _ptr(topk_idx), num_q, topk, _ptr(block_table), block_table.shape[0],
        block_table.shape[1], _ptr(seq_lens), page_size, _ptr(cache), num_blocks,
        block_stride_bytes, latent_scale, _ptr(staged), _ptr(staged_idx), _ptr(invalid_count),
        _stream(stream))
    _check(st, "nvfp4_mla_stage_fp8")
    return staged, staged_idx


def staged_fp8_tables(num_q: int, topk: int, page_size: int, device) -> dict:
    """Index tables for reading the staged rows with sparse_mla_decode (FP8 rows):
    token t is sequence t, its rows fill pages t * P .. t * P + P - 1."""
    R = nvfp4_mla_staged_rows_per_q(topk, page_size)
    P = R // page_size
    return {
        "q_seq": torch.arange(num_q, dtype=torch.int32, device=device),
        "block_table": torch.arange(num_q * P, dtype=torch.int32, device=device).view(num_q, P),
        "seq_lens": torch.full((num_q,), topk, dtype=torch.int32, device=device),
        "num_blocks": num_q * P,
        "block_stride_bytes": page_size * ROW_BYTES[ROW_FP8_576],
    }


# ------------------------------------------------------------ step planning
def _arg(t: torch.Tensor, name: str, dtype: torch.dtype, least: int, device: int) -> int:
    """Device pointer of an argument with at least ``least`` values of ``dtype``."""
    if t.dtype != dtype or t.numel() < least or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {least} values "
                         f"on the current CUDA device")
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, least: int, device: int):
    return None if t is None else _arg(t, name, dtype, least, device)


def _table(t: torch.Tensor, device: int):
    """Pointer, rows and columns of a block table."""
    if t.dim() != 2:
        raise ValueError("block_table must be [num_seqs, max_blocks_per_seq]")
    return _arg(t, "block_table", torch.int32, 0, device), t.shape[0], t.shape[1]


def nvfp4_mla_plan_step(new_lens: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor,
                        page_size: int, free_pages: torch.Tensor, free_count: torch.Tensor,
                        max_tokens: int, seq_lens_out: Optional[torch.Tensor] = None,
                        free_count_out: Optional[torch.Tensor] = None,
                        seq_ids: Optional[torch.Tensor] = None,
                        positions: Optional[torch.Tensor] = None,
                        slots: Optional[torch.Tensor] = None,
                        cu_tokens: Optional[torch.Tensor] = None,
                        refused_count: Optional[torch.Tensor] = None, stream=None):
    """Pages, block-table entries and token rows of a step that adds ``new_lens`` (int32
    [num_seqs]) tokens; returns (seq_ids, positions, slots, cu_tokens).

    ``block_table`` is updated; ``seq_lens`` and ``free_count`` too unless
    ``seq_lens_out`` / ``free_count_out`` are given. The four results
    (int32, int32, int64 [max_tokens], int32 [num_seqs + 1]) are allocated
    with torch when not given.
    """
    dev, i32 = torch.cuda.current_device(), torch.int32
    table, num_seqs, max_blocks = _table(block_table, dev)
    rows = max(max_tokens, 0)
    if seq_ids is None:
        seq_ids = _result(rows, i32, dev, stream)
    if positions is None:
        positions = _result(rows, i32, dev, stream)
    if slots is None:
        slots = _result(rows, torch.int64, dev, stream)
    if cu_tokens is None:
        cu_tokens = _result(num_seqs + 1, i32, dev, stream)
    lens_out = seq_lens if seq_lens_out is None else seq_lens_out
    count_out = free_count if free_count_out is None else free_count_out
    st = _lib().nvfp4_mla_plan_step(
        _arg(new_lens, "new_lens", i32, num_seqs, dev),
        _arg(seq_lens, "seq_lens", i32, num_seqs, dev), num_seqs, table, max_blocks, page_size,
        _arg(free_pages, "free_pages", i32, 0, dev), free_pages.numel(),
        _arg(free_count, "free_count", i32, 1, dev), max_tokens,
        _arg(lens_out, "seq_lens_out", i32, num_seqs, dev),
        _arg(count_out, "free_count_out", i32, 1, dev), _arg(seq_ids, "seq_ids", i32, rows, dev),
        _arg(positions, "positions", i32, rows, dev),
        _arg(slots, "slots", torch.int64, rows, dev),
        _arg(cu_tokens, "cu_tokens", i32, num_seqs + 1, dev),
        _opt(refused_count, "refused_count", i32, 1, dev), _stream(stream))
    _check(st, "nvfp4_mla_plan_step")
    return seq_ids, positions, slots, cu_tokens


def nvfp4_mla_truncate(keep_lens: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor,
                       page_size: int, free_pages: torch.Tensor, free_count: torch.Tensor,
                       seq_lens_out: Optional[torch.Tensor] = None,
                       free_count_out: Optional[torch.Tensor] = None,
                       dropped_count: Optional[torch.Tensor] = None, stream=None) -> None:
    """Shrink sequences to ``keep_lens`` (int32 [num_seqs]); their pages go onto ``free_pages``.

    ``seq_lens`` and ``free_count`` are updated unless ``seq_lens_out`` /
    ``free_count_out`` are given.
    """
    dev, i32 = torch.cuda.current_device(), torch.int32
    table, num_seqs, max_blocks = _table(block_table, dev)
    lens_out = seq_lens if seq_lens_out is None else seq_lens_out
    count_out = free_count if free_count_out is None else free_count_out
    st = _lib().nvfp4_mla_truncate(
        _arg(keep_lens, "keep_lens", i32, num_seqs, dev),
        _arg(seq_lens, "seq_lens", i32, num_seqs, dev), num_seqs, table, max_blocks, page_size,
        _arg(free_pages, "free_pages", i32, 0, dev), free_pages.numel(),
        _arg(free_count, "free_count", i32, 1, dev),
        _arg(lens_out, "seq_lens_out", i32, num_seqs, dev),
        _arg(count_out, "free_count_out", i32, 1, dev),
        _opt(dropped_count, "dropped_count", i32, 1, dev), _stream(stream))
    _check(st, "nvfp4_mla_truncate")


# ------------------------------------------------- index-key cache and selection
def _pool(cache: torch.Tensor, num_blocks: int, block_stride_bytes: int, page_size: int,
          device: int) -> int:
    """Device pointer of a pool that holds num_blocks pages; it may end with the last page's rows
    (a layer's view of a pool that interleaves several)."""
    least = (num_blocks - 1) * block_stride_bytes + page_size * INDEX_ROW_BYTES
    if (not cache.is_contiguous() or cache.get_device() != device
            or cache.numel() * cache.element_size() < least):
        raise ValueError("cache must be a contiguous tensor that reaches to the end of page "
                         "num_blocks - 1, on the current CUDA device")
    return cache.data_ptr()


def nvfp4_mla_index_append(keys: torch.Tensor, seq_ids: torch.Tensor, positions: torch.Tensor,
                           block_table: torch.Tensor, page_size: int, cache: torch.Tensor,
                           num_blocks: int, block_stride_bytes: int,
                           invalid_count: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantize index ``keys`` (bf16 [n,128]) into their rows of the index-key cache."""
    dev, i32 = torch.cuda.current_device(), torch.int32
    if keys.dim() != 2 or keys.shape[1] != INDEX_DIM:
        raise ValueError("keys must be bf16 [n, 128]")
    n = keys.shape[0]
    table, num_seqs, max_blocks = _table(block_table, dev)
    st = _lib().nvfp4_mla_index_append(
        _arg(keys, "keys", torch.bfloat16, 0, dev), _arg(seq_ids, "seq_ids", i32, n, dev),
        _arg(positions, "positions", i32, n, dev), n, table, num_seqs, max_blocks, page_size,
        _pool(cache, num_blocks, block_stride_bytes, page_size, dev), num_blocks, block_stride_bytes,
        _opt(invalid_count, "invalid_count", i32, 1, dev), _stream(stream))
    _check(st, "nvfp4_mla_index_append")


def nvfp4_mla_index_read(seq_ids: torch.Tensor, positions: torch.Tensor,
                         block_table: torch.Tensor, page_size: int, cache: torch.Tensor,
                         num_blocks: int, block_stride_bytes: int,
                         keys: Optional[torch.Tensor] = None,
                         invalid_count: Optional[torch.Tensor] = None, stream=None):
    """The values (bf16 [n,128]) that the index rows of n tokens stand for."""
    dev, i32 = torch.cuda.current_device(), torch.int32
    n = seq_ids.numel()
    if keys is None:
        keys = _result((n, INDEX_DIM), torch.bfloat16, dev, stream)
    table, num_seqs, max_blocks = _table(block_table, dev)
    st = _lib().nvfp4_mla_index_read(
        _arg(seq_ids, "seq_ids", i32, n, dev), _arg(positions, "positions", i32, n, dev), n,
        table, num_seqs, max_blocks, page_size,
        _pool(cache, num_blocks, block_stride_bytes, page_size, dev), num_blocks, block_stride_bytes,
        _arg(keys, "keys", torch.bfloat16, n * INDEX_DIM, dev),
        _opt(invalid_count, "invalid_count", i32, 1, dev), _stream(stream))
    _check(st, "nvfp4_mla_index_read")
    return keys


def sparse_mla_select_workspace_size(num_q: int, num_heads: int, max_blocks: int, page_size: int,
                                     select_block: int = 1) -> int:
    n = int(_lib().sparse_mla_select_workspace_size(num_q, num_heads, max_blocks, page_size,
                                                    select_block))
    if n == (1 << 64) - 1:
        raise ValueError("invalid selection shape")
    return n


def sparse_mla_select(q_index: torch.Tensor, weights: torch.Tensor, q_seq: torch.Tensor,
                      q_pos: torch.Tensor, block_table: torch.Tensor, page_size: int,
                      cache: torch.Tensor, num_blocks: int, block_stride_bytes: int,
                      num_select: int, select_block: int = 1, sink_blocks: int = 0,
                      recent_blocks: int = 0, topk_idx: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Positions of the ``num_select`` blocks of ``select_block`` tokens that score highest;
    returns topk_idx (int32 [num_q, num_select * select_block]) for sparse_mla_decode.

    ``topk_idx`` / ``workspace`` are allocated with torch when not given.
    """
    dev, i32 = torch.cuda.current_device(), torch.int32
    if q_index.dim() != 3 or q_index.shape[2] != INDEX_DIM:
        raise ValueError("q_index must be bf16 [num_q, num_heads, 128]")
    num_q, H = q_index.shape[0], q_index.shape[1]
    table, num_seqs, max_blocks = _table(block_table, dev)
    width = max(num_select * select_block, 0)
    if topk_idx is None:
        topk_idx = _result((num_q, width), i32, dev, stream)
    if workspace is None:
        need = int(_lib().sparse_mla_select_workspace_size(num_q, H, max_blocks, page_size,
                                                           select_block))
        if need < 1 << 63:  # an invalid shape is refused below
            workspace = _scratch(need, torch.uint8, dev, stream)
    ws = None if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib().sparse_mla_select(
        _arg(q_index, "q_index", torch.bfloat16, 0, dev),
        _arg(weights, "weights", torch.float32, num_q * H, dev), _arg(q_seq, "q_seq", i32, num_q, dev),
        _arg(q_pos, "q_pos", i32, num_q, dev), num_q, H, table, num_seqs, max_blocks, page_size,
        _pool(cache, num_blocks, block_stride_bytes, page_size, dev), num_blocks, block_stride_bytes,
        select_block, num_select, sink_blocks, recent_blocks,
        _arg(topk_idx, "topk_idx", i32, num_q * width, dev),
        None if workspace is None else _arg(workspace, "workspace", workspace.dtype, 0, dev),
        ws or 0, _stream(stream))
    _check(st, "sparse_mla_select")
    return topk_idx
