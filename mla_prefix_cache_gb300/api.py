"""PyTorch-facing binding of libmla: argument marshalling only.

Every step of the path runs in the library's CUDA kernels; this module checks
tensor placement/dtypes, allocates outputs and the workspace with torch when the
caller does not pass them, and forwards raw pointers and the current stream.
There is no CPU fallback: without a CUDA device or the built library every call
raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import numpy as np
import torch

from . import _lib
from ._lib import (KV_BF16, KV_FP8_E4M3, OUT_BF16, OUT_FP32, PART_ALL, PART_CONTEXT,  # noqa: F401
                   PART_EXTEND, MLAError)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return ctypes.c_void_p(t.data_ptr())


def set_kernel_events(begin: Optional[torch.cuda.Event], end: Optional[torch.cuda.Event]) -> None:
    """Time the fused prefill kernel of later prefill() calls with these events
    (recorded on the call's stream around the fused kernel launches)."""
    if begin is None or end is None:
        _lib.load().mla_set_kernel_events(None, None)
        return
    for e in (begin, end):      # torch creates the CUDA event lazily on first record
        if not e.cuda_event:
            e.record()
    _lib.load().mla_set_kernel_events(ctypes.c_void_p(begin.cuda_event), ctypes.c_void_p(end.cuda_event))


def launch_count() -> int:
    """Kernels launched by libmla so far in this process."""
    return int(_lib.load().mla_launch_count())


def kv_dtype_code(kv_cache: torch.Tensor) -> int:
    # a pool of other blocks is refused: the kernels find row 64 id + slot of a block id
    block = kv_cache.shape[1:]
    if kv_cache.dtype == torch.bfloat16 and block == (64, 576):
        return KV_BF16
    if kv_cache.dtype == torch.uint8 and block == (64, 640):
        return KV_FP8_E4M3
    raise ValueError("kv_cache must be bf16 [NB,64,576] or uint8 [NB,64,640]")


def prefill_workspace_size(seq_lens, cu_q, num_heads: int, segments=None, chunk: int = 4096,
                           parts: int = PART_ALL) -> int:
    sl, _k1 = _lib.i32_host(seq_lens)
    cq, _k2 = _lib.i32_host(cu_q)
    sp, ns, _k3 = _lib.segments_host(segments)
    n = _lib.load().mla_prefill_workspace_size(len(_k1), sl, cq, int(num_heads), sp, ns, int(chunk), int(parts))
    if n == 0:
        raise MLAError("mla_prefill_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def prefill_min_workspace_size(seq_lens, cu_q, num_heads: int, segments=None, chunk: int = 4096,
                               parts: int = PART_ALL) -> int:
    """The smallest workspace mla_prefill_ctx runs in (shallow K/V rings, one
    piece per launch: slower)."""
    sl, _k1 = _lib.i32_host(seq_lens)
    cq, _k2 = _lib.i32_host(cu_q)
    sp, ns, _k3 = _lib.segments_host(segments)
    n = _lib.load().mla_prefill_min_workspace_size(len(_k1), sl, cq, int(num_heads), sp, ns, int(chunk), int(parts))
    if n == 0:
        raise MLAError("mla_prefill_min_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def absorbed_workspace_size(seq_lens, cu_q, num_heads: int, segments=None, chunk: int = 4096,
                            parts: int = PART_ALL, fp8_scores: bool = False) -> int:
    sl, _k1 = _lib.i32_host(seq_lens)
    cq, _k2 = _lib.i32_host(cu_q)
    sp, ns, _k3 = _lib.segments_host(segments)
    L = _lib.load()
    fn = L.mla_prefill_absorbed_fp8_workspace_size if fp8_scores else L.mla_prefill_absorbed_workspace_size
    if fp8_scores == "auto":
        fn = L.mla_prefill_auto_workspace_size
    n = fn(len(_k1), sl, cq, int(num_heads), sp, ns, int(chunk), int(parts))
    if n == 0:
        raise MLAError("mla_prefill_absorbed_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def prefill(q: torch.Tensor, q_pos: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
            seq_lens, cu_q, kv_b_proj: torch.Tensor, *, chunk: int, softmax_scale: float,
            rope_theta: float = 10000.0, kv_scale: float = 1.0, segments=None, parts: int = PART_ALL,
            out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
            lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None, absorbed=False,
            kv_b_proj_e4m3: Optional[torch.Tensor] = None, w_scale: Optional[float] = None
            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """MLA chunked prefill of one layer (mla_prefill_ctx; absorbed=True:
    mla_prefill_ctx_absorbed, the same result computed in latent space;
    absorbed="fp8": mla_prefill_ctx_absorbed_fp8, FP8 caches, latent scores
    on the FP8 tensor cores; absorbed="auto": mla_prefill_ctx_auto, the path
    chosen per request by its number of queries).  With kv_b_proj_e4m3 (uint8
    [H*256, 512], see kv_b_proj_to_e4m3) and w_scale: mla_prefill_ctx_fp8w,
    FP8 caches, the up-projection on the FP8 tensor cores.

    q bf16 [T_q, H, 192] (q_rope unrotated); q_pos int32 [T_q]; kv_cache bf16
    [NB,64,576] or uint8 [NB,64,640] (FP8); block_table int32 [B, max_blocks];
    seq_lens / cu_q host int32 (numpy or lists); kv_b_proj bf16 [512, H*256];
    segments optional host [S,4] (req, start, len, rope_offset).
    Returns (out [T_q, H, 128] in out_dtype, lse fp32 [T_q, H])."""
    T_q, H = int(q.shape[0]), int(q.shape[1])
    L = _lib.load()
    sl, keep_sl = _lib.i32_host(seq_lens)
    cq, keep_cq = _lib.i32_host(cu_q)
    sp, ns, keep_sp = _lib.segments_host(segments)
    B = int(keep_sl.shape[0])
    if keep_cq.shape[0] != B + 1 or int(keep_cq[-1]) != T_q:
        raise ValueError("cu_q must have num_reqs+1 entries ending at T_q")
    dev = q.device
    if out is None:
        out = torch.empty((T_q, H, 128), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((T_q, H), dtype=torch.float32, device=dev)
    fp8 = absorbed == "fp8"
    auto = absorbed == "auto"
    fp8w = kv_b_proj_e4m3 is not None
    if fp8w and (absorbed or w_scale is None):
        raise ValueError("kv_b_proj_e4m3 takes w_scale and the up-projected path")
    if workspace is None:
        if absorbed:
            ws_bytes = absorbed_workspace_size(keep_sl, keep_cq, H, segments, chunk, parts,
                                               fp8_scores="auto" if auto else fp8)
        else:
            ws_bytes = prefill_workspace_size(keep_sl, keep_cq, H, segments, chunk, parts)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    od = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_FP32
    common = (_dev(q, "q", torch.bfloat16), _dev(q_pos, "q_pos", torch.int32), _dev(kv_cache, "kv_cache"),
              kv_dtype_code(kv_cache), float(kv_scale), int(kv_cache.shape[0]),
              _dev(block_table, "block_table", torch.int32), int(block_table.shape[1]),
              sl, cq, B, H, sp, ns, int(chunk))
    tail = (float(softmax_scale), float(rope_theta), int(parts),
            _dev(out, "out", (torch.float32, torch.bfloat16)), od, _dev(lse, "lse", torch.float32),
            _dev(workspace, "workspace"), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
            _stream_ptr(stream))
    if fp8w:
        name = "mla_prefill_ctx_fp8w"
        st = L.mla_prefill_ctx_fp8w(*common, _dev(kv_b_proj_e4m3, "kv_b_proj_e4m3", torch.uint8), float(w_scale),
                                    *tail)
    else:
        name = ("mla_prefill_ctx_auto" if auto else "mla_prefill_ctx_absorbed_fp8" if fp8
                else "mla_prefill_ctx_absorbed" if absorbed else "mla_prefill_ctx")
        st = getattr(L, name)(*common, _dev(kv_b_proj, "kv_b_proj", torch.bfloat16), *tail)
    _lib.check(name, st)
    prefill.last_workspace = workspace
    return out, lse


def kv_b_proj_absmax(kv_b_proj: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> float:
    """The largest |w| of a bf16 kv_b_proj [512, H*256] (mla_kv_b_proj_absmax; synchronises)."""
    H = int(kv_b_proj.shape[1]) // 256
    out = torch.empty(1, dtype=torch.float32, device=kv_b_proj.device)
    _lib.check("mla_kv_b_proj_absmax", _lib.load().mla_kv_b_proj_absmax(
        _dev(kv_b_proj, "kv_b_proj", torch.bfloat16), H, _dev(out, "absmax"), _stream_ptr(stream)))
    return float(out.item())


def kv_b_proj_to_e4m3(kv_b_proj: torch.Tensor, w_scale: float, out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """E4M3 codes of kv_b_proj / w_scale, transposed: uint8 [H*256, 512]
    (mla_kv_b_proj_to_e4m3).  w_scale = absmax / 448 uses the whole range."""
    cols = int(kv_b_proj.shape[1])
    if out is None:
        out = torch.empty((cols, 512), dtype=torch.uint8, device=kv_b_proj.device)
    _lib.check("mla_kv_b_proj_to_e4m3", _lib.load().mla_kv_b_proj_to_e4m3(
        _dev(kv_b_proj, "kv_b_proj", torch.bfloat16), cols // 256, float(w_scale), _dev(out, "out", torch.uint8),
        _stream_ptr(stream)))
    return out


def _protected_host(protected_rows, T_q: int):
    if protected_rows is None:
        return None, None
    m = np.zeros(T_q, dtype=np.uint8)
    pr = np.asarray(protected_rows)
    if pr.dtype == bool and pr.shape == (T_q,):
        m[:] = pr
    else:
        m[pr.astype(np.int64)] = 1
    return ctypes.c_void_p(m.ctypes.data), m


def reuse_workspace_size(seq_lens, cu_q, num_heads: int, global_heads, protected_rows=None, segments=None,
                         chunk: int = 4096, parts: int = PART_ALL) -> int:
    sl, keep_sl = _lib.i32_host(seq_lens)
    cq, keep_cq = _lib.i32_host(cu_q)
    sp, ns, _k3 = _lib.segments_host(segments)
    gh, keep_gh = _lib.i32_host(list(global_heads))
    pp, _k4 = _protected_host(protected_rows, int(keep_cq[-1]))
    n = _lib.load().mla_prefill_reuse_workspace_size(len(keep_sl), sl, cq, int(num_heads), sp, ns, int(chunk),
                                                     int(parts), gh, int(keep_gh.shape[0]), pp)
    if n == 0:
        raise MLAError("mla_prefill_reuse_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def prefill_reuse(q: torch.Tensor, q_pos: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                  seq_lens, cu_q, kv_b_proj: torch.Tensor, art_out: torch.Tensor, art_lse: torch.Tensor, *,
                  global_heads, protected_rows=None, chunk: int, softmax_scale: float, rope_theta: float = 10000.0,
                  kv_scale: float = 1.0, segments=None, parts: int = PART_ALL,
                  out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Head-split reuse (mla_prefill_reuse): the Global heads and the
    protected rows (host indices or a bool mask over T_q) are recomputed,
    every other (row, head) takes the artifact (art_out fp32 [T_q, H, 128],
    art_lse fp32 [T_q, H])."""
    T_q, H = int(q.shape[0]), int(q.shape[1])
    sl, keep_sl = _lib.i32_host(seq_lens)
    cq, keep_cq = _lib.i32_host(cu_q)
    sp, ns, keep_sp = _lib.segments_host(segments)
    gh, keep_gh = _lib.i32_host(list(global_heads))
    pp, keep_pp = _protected_host(protected_rows, T_q)
    dev = q.device
    if out is None:
        out = torch.empty((T_q, H, 128), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((T_q, H), dtype=torch.float32, device=dev)
    if workspace is None:
        ws_bytes = reuse_workspace_size(keep_sl, keep_cq, H, keep_gh, keep_pp.astype(bool) if keep_pp is not None
                                        else None, segments, chunk, parts)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    od = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_FP32
    st = _lib.load().mla_prefill_reuse(
        _dev(q, "q", torch.bfloat16), _dev(q_pos, "q_pos", torch.int32), _dev(kv_cache, "kv_cache"),
        kv_dtype_code(kv_cache), float(kv_scale), int(kv_cache.shape[0]),
        _dev(block_table, "block_table", torch.int32), int(block_table.shape[1]),
        sl, cq, int(keep_sl.shape[0]), H, sp, ns, int(chunk), _dev(kv_b_proj, "kv_b_proj", torch.bfloat16),
        float(softmax_scale), float(rope_theta), int(parts), gh, int(keep_gh.shape[0]), pp,
        _dev(art_out, "art_out", torch.float32), _dev(art_lse, "art_lse", torch.float32),
        _dev(out, "out", (torch.float32, torch.bfloat16)), od, _dev(lse, "lse", torch.float32),
        _dev(workspace, "workspace"), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
        _stream_ptr(stream))
    _lib.check("mla_prefill_reuse", st)
    prefill_reuse.last_workspace = workspace
    return out, lse


def device_error(workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> int:
    """Reads and clears the device error word of a prefill workspace."""
    return int(_lib.load().mla_get_device_error(_dev(workspace, "workspace"), _stream_ptr(stream)))


def merge_states(out_a, lse_a, out_b, lse_b, out=None, lse=None, stream=None):
    """merge_attn_states on fp32 [rows, d_v] states and fp32 [rows] lse."""
    d_v = int(out_a.shape[-1])
    rows = int(out_a.numel() // d_v)
    out = torch.empty_like(out_a) if out is None else out
    lse = torch.empty_like(lse_a) if lse is None else lse
    f32 = torch.float32
    st = _lib.load().mla_merge_states(_dev(out_a, "out_a", f32), _dev(lse_a, "lse_a", f32), _dev(out_b, "out_b", f32),
                                      _dev(lse_b, "lse_b", f32), _dev(out, "out", f32), _dev(lse, "lse", f32),
                                      rows, d_v, _stream_ptr(stream))
    _lib.check("mla_merge_states", st)
    return out, lse


def rope_relocate(x: torch.Tensor, pos: torch.Tensor, offset: int, theta: float = 10000.0,
                  y: Optional[torch.Tensor] = None, rope_col: Optional[int] = None, stream=None) -> torch.Tensor:
    """Rotate the 64 RoPE columns of bf16 x [tokens, heads, row] by (pos - offset)."""
    tokens, heads, row = int(x.shape[0]), int(x.shape[1]), int(x.shape[2])
    rope_col = row - 64 if rope_col is None else int(rope_col)
    if y is None:
        y = x.clone()
    st = _lib.load().mla_rope_relocate(_dev(x, "x", torch.bfloat16), _dev(pos, "pos", torch.int32), int(offset),
                                       float(theta), _dev(y, "y", torch.bfloat16), tokens, heads, row, rope_col,
                                       _stream_ptr(stream))
    _lib.check("mla_rope_relocate", st)
    return y


def gather_latent(kv_cache: torch.Tensor, block_table_row: torch.Tensor, start: int, length: int,
                  kv_scale: float = 1.0, dst: Optional[torch.Tensor] = None,
                  dev_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows of tokens [start, start+length) of one request as bf16 [length, 576]."""
    if dst is None:
        dst = torch.empty((length, 576), dtype=torch.bfloat16, device=kv_cache.device)
    errp = _dev(dev_error, "dev_error", (torch.int32, torch.uint32)) if dev_error is not None else None
    st = _lib.load().mla_gather_latent(_dev(kv_cache, "kv_cache"), kv_dtype_code(kv_cache), float(kv_scale),
                                       int(kv_cache.shape[0]), _dev(block_table_row, "block_table_row", torch.int32),
                                       int(block_table_row.shape[0]), int(start), int(length),
                                       _dev(dst, "dst", torch.bfloat16), errp, _stream_ptr(stream))
    _lib.check("mla_gather_latent", st)
    return dst


def block_hash(kv_cache: torch.Tensor, block_ids: torch.Tensor, dev_error: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Content hash of whole cache blocks (mla_block_hash): int64 [n] holding
    the uint64 hash bits."""
    n = int(block_ids.numel())
    hashes = torch.empty(n, dtype=torch.int64, device=kv_cache.device)
    errp = _dev(dev_error, "dev_error", (torch.int32, torch.uint32)) if dev_error is not None else None
    st = _lib.load().mla_block_hash(_dev(kv_cache, "kv_cache"), kv_dtype_code(kv_cache), int(kv_cache.shape[0]),
                                    _dev(block_ids, "block_ids", torch.int32), n, _dev(hashes, "hashes"), errp,
                                    _stream_ptr(stream))
    _lib.check("mla_block_hash", st)
    return hashes


def block_compare(kv_cache: torch.Tensor, block_a: torch.Tensor, block_b: torch.Tensor,
                  dev_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Byte equality of block pairs (mla_block_compare): int32 [n], 1 equal, 0 not."""
    n = int(block_a.numel())
    if int(block_b.numel()) != n:
        raise ValueError("block_a and block_b differ in length")
    equal = torch.empty(n, dtype=torch.int32, device=kv_cache.device)
    errp = _dev(dev_error, "dev_error", (torch.int32, torch.uint32)) if dev_error is not None else None
    st = _lib.load().mla_block_compare(_dev(kv_cache, "kv_cache"), kv_dtype_code(kv_cache), int(kv_cache.shape[0]),
                                       _dev(block_a, "block_a", torch.int32), _dev(block_b, "block_b", torch.int32),
                                       n, _dev(equal, "equal"), errp, _stream_ptr(stream))
    _lib.check("mla_block_compare", st)
    return equal


# ------------------------------------------------------------------ serving

# These calls sit in a decoding loop whose kernels take a few microseconds: their checks are one pass over each
# tensor and pointers go to the library as plain integers.

def _at(t: torch.Tensor, name: str, device: int, dtype, shape=None) -> int:
    """Address of a contiguous tensor of `dtype` (and `shape`) on CUDA device `device`."""
    if (isinstance(t, torch.Tensor) and t.get_device() == device and (t.dtype is dtype or dtype is None)
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise ValueError(f"{name} must be a tensor on cuda:{device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} must be contiguous")


def _current(t: torch.Tensor, name: str) -> int:
    """The device of `t`, which has to be the current one: the call launches there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return device


def _stream_on(device: int, stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, expected cuda:{device}")
    return stream.cuda_stream


def _batch_args(block_table, seq_lens, cu_q, rows: int, device: int):
    """Checked (num_reqs, block_table, max_blocks, seq_lens, cu_q) of a serving call."""
    bt = _at(block_table, "block_table", device, torch.int32)
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [num_reqs, max_blocks] and seq_lens [num_reqs]")
    B, max_blocks = shape
    sl = _at(seq_lens, "seq_lens", device, torch.int32, (B,))
    if cu_q is not None:
        return B, bt, max_blocks, sl, _at(cu_q, "cu_q", device, torch.int32, (B + 1,))
    if rows and (B == 0 or rows % B):
        raise ValueError(f"{rows} rows cannot be shared evenly by {B} requests: pass cu_q")
    return B, bt, max_blocks, sl, None


def _error_word(t: torch.Tensor, device: int) -> int:
    return _at(t, "dev_error", device, torch.uint32 if t.dtype is torch.uint32 else torch.int32)


def cache_append(kv: torch.Tensor, pos: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, *, cu_q: Optional[torch.Tensor] = None,
                 norm_weight: Optional[torch.Tensor] = None, norm_eps: float = 1e-6, rope_theta: float = 10000.0,
                 kv_scale: float = 1.0, dev_error: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Writes the rows of new tokens into the paged cache (mla_cache_append):
    RMSNorm of the latent part (with norm_weight bf16 [512]), rotation of the
    RoPE part to pos, rounding to bf16 or E4M3.

    kv bf16 [rows, 576], rows any multiple of 8 elements apart (a column slice
    of a projection's output); pos int32 [rows]; kv_cache bf16 [NB,64,576] or
    uint8 [NB,64,640]; block_table int32 [B, max_blocks]; seq_lens int32 [B],
    new rows included, and cu_q int32 [B+1] (default: rows / B each) on the
    device.  Returns kv_cache."""
    device = _current(kv, "kv")
    if kv.dim() != 2 or kv.dtype is not torch.bfloat16:
        raise ValueError("kv must be bf16 [rows, 576]")
    rows, cols = kv.shape
    stride, unit = kv.stride()
    if cols != 576 or (rows and unit != 1):
        raise ValueError("kv must be bf16 [rows, 576] with unit column stride")
    if rows < 2:
        stride = 576
    elif stride < 576 or stride % 8:
        raise ValueError("kv rows must be a multiple of 8 elements, at least 576, apart")
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, rows, device)
    st = _lib.load().mla_cache_append(
        kv.data_ptr(), stride, _at(pos, "pos", device, torch.int32, (rows,)),
        None if norm_weight is None else _at(norm_weight, "norm_weight", device, torch.bfloat16, (512,)), norm_eps, cq,
        sl, B, rows, bt, max_blocks, rope_theta, _at(kv_cache, "kv_cache", device, None), kv_dtype_code(kv_cache),
        kv_scale, kv_cache.shape[0], None if dev_error is None else _error_word(dev_error, device),
        _stream_on(device, stream))
    if st:
        _lib.check("mla_cache_append", st)
    return kv_cache


def decode_workspace_size(num_reqs: int, total_q: int, num_heads: int) -> int:
    n = _lib.load().mla_decode_workspace_size(int(num_reqs), int(total_q), int(num_heads))
    if n == 0:
        raise MLAError("mla_decode_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def _decode_tensors(device, B, T_q, H, out, out_dtype, lse, return_lse, workspace):
    if out is None:
        out = torch.empty((T_q, H, 128), dtype=out_dtype, device=device)
    if lse is None and return_lse:
        lse = torch.empty((T_q, H), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = torch.empty(decode_workspace_size(B, T_q, H), dtype=torch.uint8, device=device)
        if T_q == 0:      # nothing will be launched that sets the error word
            workspace[:4] = 0
    return out, lse, workspace


def decode(q: torch.Tensor, q_pos: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
           seq_lens: torch.Tensor, kv_b_proj: torch.Tensor, *, softmax_scale: float, rope_theta: float = 10000.0,
           kv_scale: float = 1.0, cu_q: Optional[torch.Tensor] = None, segments: Optional[torch.Tensor] = None,
           seg_ptr: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           out_dtype: torch.dtype = torch.float32, lse: Optional[torch.Tensor] = None, return_lse: bool = False,
           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Attention of one or a few new tokens per request (mla_decode), every
    length on the device: the call can be captured into a CUDA graph.

    q bf16 [T_q, H, 192] (q_rope unrotated); q_pos int32 [T_q]; kv_cache as for
    prefill; block_table int32 [B, max_blocks], seq_lens int32 [B] (the new
    tokens included) and cu_q int32 [B+1] (default: T_q / B rows each) on the
    device; kv_b_proj bf16 [512, H*256].  Relocated documents: segments int64
    [S, 3] (start, length, rope offset) with seg_ptr int32 [B+1], on the device.
    Returns out [T_q, H, 128], and lse fp32 [T_q, H] with it when return_lse is
    set or lse is given."""
    device = _current(q, "q")
    if q.dim() != 3 or q.shape[2] != 192:
        raise ValueError("q must be [T_q, H, 192]")
    T_q, H, _ = q.shape
    if (segments is None) != (seg_ptr is None):
        raise ValueError("segments and seg_ptr go together")
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, T_q, device)
    sp = gp = None
    ns = 0
    if segments is not None:
        ns = segments.shape[0]
        sp = _at(segments, "segments", device, torch.int64, (ns, 3))
        gp = _at(seg_ptr, "seg_ptr", device, torch.int32, (B + 1,))
        if ns == 0:      # an empty tensor has no address: any one will do, nothing of it is read
            sp = gp
    if stream is None:
        out, lse, workspace = _decode_tensors(q.device, B, T_q, H, out, out_dtype, lse, return_lse, workspace)
    else:      # on the stream that uses them: freed memory goes to its later work only
        with torch.cuda.stream(stream):
            out, lse, workspace = _decode_tensors(q.device, B, T_q, H, out, out_dtype, lse, return_lse, workspace)
    bf16 = out.dtype is torch.bfloat16
    st = _lib.load().mla_decode(
        _at(q, "q", device, torch.bfloat16), _at(q_pos, "q_pos", device, torch.int32, (T_q,)),
        _at(kv_cache, "kv_cache", device, None), kv_dtype_code(kv_cache), kv_scale, kv_cache.shape[0], bt, max_blocks,
        sl, cq, B, T_q, H, sp, gp, ns, _at(kv_b_proj, "kv_b_proj", device, torch.bfloat16, (512, H * 256)),
        softmax_scale, rope_theta, _at(out, "out", device, torch.bfloat16 if bf16 else torch.float32, (T_q, H, 128)),
        OUT_BF16 if bf16 else OUT_FP32, None if lse is None else _at(lse, "lse", device, torch.float32, (T_q, H)),
        _at(workspace, "workspace", device, None), workspace.numel() * workspace.element_size(),
        _stream_on(device, stream))
    if st:
        _lib.check("mla_decode", st)
    decode.last_workspace = workspace
    return out if lse is None else (out, lse)


# ------------------------------------------------------- a sparse decoding step

def _not_32_bits(x: int) -> bool:
    """Whether the C entries' ints would cut a number to another one; of several joined by | (beside a negative one, which they refuse, it may say no)."""
    return x >> 31 not in (0, -1)


def assign_blocks(block_table: torch.Tensor, held: torch.Tensor, seq_lens: torch.Tensor, free_blocks: torch.Tensor,
                  free_count: torch.Tensor, *, shared: Optional[torch.Tensor] = None,
                  cu_q: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                  dev_error: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Brings the block tables to the requests' lengths (mla_assign_blocks):
    blocks behind a length go back to the free ones, missing ones are taken
    from them, in place and on the device.

    block_table int32 [B, max_blocks]; held int32 [B], the blocks of each table
    row in use; seq_lens int32 [B], the tokens to hold; free_blocks int32
    [capacity] with free_count int32 [1], a stack; shared int32 [B], leading
    blocks that are not given back (lowered to held where a request grows from
    fewer, as those it gets are its own).  slots int64 [rows]: filled with the cache
    slot of every new row (cu_q int32 [B+1] as for cache_append).  Returns
    slots."""
    device, i32 = _current(block_table, "block_table"), torch.int32
    rows = 0 if slots is None else slots.shape[0]
    capacity = free_blocks.numel()
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, rows, device)
    st = _lib.load().mla_assign_blocks(
        bt, max_blocks, _at(held, "held", device, i32, (B,)), sl, None if shared is None else _at(shared, "shared", device, i32, (B,)),
        B, _at(free_blocks, "free_blocks", device, i32, (capacity,)), capacity,
        _at(free_count, "free_count", device, i32, (1,)), cq, rows,
        None if slots is None else _at(slots, "slots", device, torch.int64, (rows,)),
        None if dev_error is None else _error_word(dev_error, device), _stream_on(device, stream))
    if st:
        _lib.check("mla_assign_blocks", st)
    return slots


def block_means(kv_cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, means: torch.Tensor, *,
                rows: int, cu_q: Optional[torch.Tensor] = None, kv_scale: float = 1.0,
                dev_error: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The mean row of every cache block that the last `rows` new rows of the
    batch fill (mla_block_means), to call after cache_append with its
    block_table, seq_lens and cu_q.

    means bf16 [NB, 576], written at those blocks only.  Returns means."""
    if _not_32_bits(rows):
        raise MLAError("mla_block_means", _lib.MLA_ERR_UNSUPPORTED)
    device = _current(kv_cache, "kv_cache")
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, rows, device)
    st = _lib.load().mla_block_means(
        _at(kv_cache, "kv_cache", device, None), kv_dtype_code(kv_cache), kv_scale, kv_cache.shape[0], bt, max_blocks, sl, cq,
        B, rows, _at(means, "means", device, torch.bfloat16, (kv_cache.shape[0], 576)),
        None if dev_error is None else _error_word(dev_error, device), _stream_on(device, stream))
    if st:
        _lib.check("mla_block_means", st)
    return means


def block_scores_workspace_size(total_q: int, num_heads: int, max_blocks: int) -> int:
    n = _lib.load().mla_block_scores_workspace_size(int(total_q), int(num_heads), int(max_blocks))
    if n == 0:
        raise MLAError("mla_block_scores_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def _scores_tensors(device, T_q, H, max_blocks, out, out_dtype, workspace):
    if out is None:
        out = torch.empty((T_q, max_blocks), dtype=out_dtype, device=device)
    if workspace is None:
        workspace = torch.empty(block_scores_workspace_size(T_q, H, max_blocks), dtype=torch.uint8, device=device)
        if T_q == 0:      # nothing will be launched that sets the error word
            workspace[:4] = 0
    return out, workspace


def block_scores(q: torch.Tensor, q_pos: torch.Tensor, means: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, kv_b_proj: torch.Tensor, *, softmax_scale: float, rope_theta: float = 10000.0,
                 cu_q: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.float32, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The share of each query's attention that the blocks before its own would
    take by their means, over all heads (mla_block_scores).

    q, q_pos, block_table, seq_lens, cu_q, kv_b_proj as for decode; means bf16
    [NB, 576] (see block_means).  Returns out [T_q, max_blocks], -inf where a
    query sees no whole block."""
    device = _current(q, "q")
    if q.dim() != 3 or q.shape[2] != 192:
        raise ValueError("q must be [T_q, H, 192]")
    T_q, H, _ = q.shape
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, T_q, device)
    if stream is None:
        out, workspace = _scores_tensors(q.device, T_q, H, max_blocks, out, out_dtype, workspace)
    else:      # on the stream that uses them, as in decode
        with torch.cuda.stream(stream):
            out, workspace = _scores_tensors(q.device, T_q, H, max_blocks, out, out_dtype, workspace)
    bf16 = out.dtype is torch.bfloat16
    st = _lib.load().mla_block_scores(
        _at(q, "q", device, torch.bfloat16), _at(q_pos, "q_pos", device, torch.int32, (T_q,)),
        _at(means, "means", device, torch.bfloat16, (means.shape[0], 576)), means.shape[0], bt, max_blocks, sl, cq, B, T_q, H,
        _at(kv_b_proj, "kv_b_proj", device, torch.bfloat16, (512, H * 256)), softmax_scale, rope_theta,
        _at(out, "out", device, torch.bfloat16 if bf16 else torch.float32, (T_q, max_blocks)), OUT_BF16 if bf16 else OUT_FP32,
        _at(workspace, "workspace", device, None), workspace.numel() * workspace.element_size(), _stream_on(device, stream))
    if st:
        _lib.check("mla_block_scores", st)
    block_scores.last_workspace = workspace
    return out


def select_blocks(scores: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, *, keep: int, sinks: int = 1,
                  recent: int = 2, cu_q: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None,
                  lens: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The `keep` blocks that each query attends (mla_select_blocks): the first
    `sinks`, the last `recent` and the best scored between them.

    scores fp32 or bf16 [T_q, max_blocks] (see block_scores); block_table,
    seq_lens, cu_q as for decode.  Returns (table int32 [T_q, keep], lens int32
    [T_q]): block_table and seq_lens of decode(q, q_pos, kv_cache, table, lens,
    kv_b_proj, ...), which attends them."""
    if _not_32_bits(keep | sinks | recent):
        raise MLAError("mla_select_blocks", _lib.MLA_ERR_UNSUPPORTED)
    device = _current(scores, "scores")
    if scores.dim() != 2 or block_table.dim() != 2 or scores.shape[1] != block_table.shape[1]:
        raise ValueError("scores must be [T_q, max_blocks]")
    T_q = scores.shape[0]
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, T_q, device)
    if table is None or lens is None:
        with torch.cuda.stream(stream):      # on the stream that uses them (None: the current one)
            if table is None:
                table = torch.empty((T_q, keep), dtype=torch.int32, device=scores.device)
            if lens is None:
                lens = torch.empty(T_q, dtype=torch.int32, device=scores.device)
    bf16 = scores.dtype is torch.bfloat16
    st = _lib.load().mla_select_blocks(
        _at(scores, "scores", device, torch.bfloat16 if bf16 else torch.float32), OUT_BF16 if bf16 else OUT_FP32, bt, max_blocks,
        sl, cq, B, T_q, keep, sinks, recent, _at(table, "table", device, torch.int32, (T_q, keep)), _at(lens, "lens", device, torch.int32, (T_q,)),
        None if dev_error is None else _error_word(dev_error, device), _stream_on(device, stream))
    if st:
        _lib.check("mla_select_blocks", st)
    return table, lens


def decode_sparse_workspace_size(num_reqs: int, total_q: int, num_heads: int, max_blocks: int, keep: int) -> int:
    if _not_32_bits(keep):
        raise MLAError("mla_decode_sparse_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    n = _lib.load().mla_decode_sparse_workspace_size(int(num_reqs), int(total_q), int(num_heads), int(max_blocks), int(keep))
    if n == 0:
        raise MLAError("mla_decode_sparse_workspace_size", _lib.MLA_ERR_INVALID_ARG)
    return int(n)


def _sparse_tensors(device, B, T_q, H, max_blocks, keep, out, out_dtype, lse, return_lse, workspace):
    if out is None:
        out = torch.empty((T_q, H, 128), dtype=out_dtype, device=device)
    if lse is None and return_lse:
        lse = torch.empty((T_q, H), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = torch.empty(decode_sparse_workspace_size(B, T_q, H, max_blocks, keep), dtype=torch.uint8, device=device)
        if T_q == 0:      # nothing will be launched that sets the error word
            workspace[:4] = 0
    return out, lse, workspace


def decode_sparse(q: torch.Tensor, q_pos: torch.Tensor, kv_cache: torch.Tensor, means: torch.Tensor,
                  block_table: torch.Tensor, seq_lens: torch.Tensor, kv_b_proj: torch.Tensor, *, keep: int, sinks: int = 1,
                  recent: int = 2, softmax_scale: float, rope_theta: float = 10000.0, kv_scale: float = 1.0,
                  cu_q: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  out_dtype: torch.dtype = torch.float32, lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                  workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Decode attention over the `keep` blocks of each query that block_scores
    and select_blocks choose (mla_decode_sparse), in one call.

    q, q_pos, kv_cache, block_table, seq_lens, cu_q, kv_b_proj, out, lse as for
    decode; means bf16 [NB, 576] (see block_means).  A keep above max_blocks
    is the same as max_blocks.  Returns out [T_q, H, 128],
    and lse fp32 [T_q, H] with it when return_lse is set or lse is given."""
    if _not_32_bits(keep | sinks | recent):
        raise MLAError("mla_decode_sparse", _lib.MLA_ERR_UNSUPPORTED)
    device = _current(q, "q")
    if q.dim() != 3 or q.shape[2] != 192:
        raise ValueError("q must be [T_q, H, 192]")
    T_q, H, _ = q.shape
    B, bt, max_blocks, sl, cq = _batch_args(block_table, seq_lens, cu_q, T_q, device)
    if stream is None:
        out, lse, workspace = _sparse_tensors(q.device, B, T_q, H, max_blocks, keep, out, out_dtype, lse, return_lse, workspace)
    else:      # on the stream that uses them, as in decode
        with torch.cuda.stream(stream):
            out, lse, workspace = _sparse_tensors(q.device, B, T_q, H, max_blocks, keep, out, out_dtype, lse, return_lse, workspace)
    bf16 = out.dtype is torch.bfloat16
    st = _lib.load().mla_decode_sparse(
        _at(q, "q", device, torch.bfloat16), _at(q_pos, "q_pos", device, torch.int32, (T_q,)),
        _at(kv_cache, "kv_cache", device, None), kv_dtype_code(kv_cache), kv_scale, kv_cache.shape[0],
        _at(means, "means", device, torch.bfloat16, (kv_cache.shape[0], 576)), bt, max_blocks, sl, cq, B, T_q, H, keep, sinks,
        recent, _at(kv_b_proj, "kv_b_proj", device, torch.bfloat16, (512, H * 256)), softmax_scale, rope_theta,
        _at(out, "out", device, torch.bfloat16 if bf16 else torch.float32, (T_q, H, 128)), OUT_BF16 if bf16 else OUT_FP32,
        None if lse is None else _at(lse, "lse", device, torch.float32, (T_q, H)), _at(workspace, "workspace", device, None),
        workspace.numel() * workspace.element_size(), _stream_on(device, stream))
    if st:
        _lib.check("mla_decode_sparse", st)
    decode_sparse.last_workspace = workspace
    return out if lse is None else (out, lse)


# ---------------------------------------------------------------- workloads

class DeviceWorkload:
    """Device copies of a workload's inputs (see workload.Workload)."""

    def __init__(self, wl, device="cuda"):
        self.wl = wl
        dev = torch.device(device)
        self.q = torch.from_numpy(wl.q.view(np.int16)).to(dev).view(torch.bfloat16)
        self.q_pos = torch.from_numpy(wl.q_pos).to(dev)
        if wl.kv_dtype == "bf16":
            self.kv_cache = torch.from_numpy(wl.kv_cache.view(np.int16)).to(dev).view(torch.bfloat16)
        else:
            self.kv_cache = torch.from_numpy(wl.kv_cache).to(dev)
        self.block_table = torch.from_numpy(wl.block_table).to(dev)
        self.kv_b_proj = torch.from_numpy(wl.kv_b_proj.view(np.int16)).to(dev).view(torch.bfloat16)
        self.seq_lens = wl.seq_lens
        self.cu_q = wl.cu_q

    def run(self, parts=PART_ALL, out_dtype=torch.float32, chunk=None, **kw):
        wl = self.wl
        return prefill(self.q, self.q_pos, self.kv_cache, self.block_table, self.seq_lens, self.cu_q,
                       self.kv_b_proj, chunk=wl.chunk if chunk is None else chunk,
                       softmax_scale=wl.softmax_scale, rope_theta=wl.rope_theta, kv_scale=wl.kv_scale,
                       segments=wl.segments, parts=parts, out_dtype=out_dtype, **kw)
