"""GB300-native verification step of speculative decoding with adaptive
verification.

Two stages, both hand-written sm_103a CUDA kernels behind the C ABI of
``include/sd.h`` (``libsdverify.so``):

  sd_plan       survival -> global top-B (or one K for the batch) -> budget
                argmax -> varlen compaction
  sd_verify     vocab-wide speculative rejection sampling on compacted logits
  sd_cache_append, sd_attend, sd_sample
                around the step: the rows' keys and values into a paged
                cache, the rows' attention over it, and truncated sampling
  sd_calibrate  one online step of the per-position acceptance model (and
                sd_calibrate_apply: the calibrated logits for the next plan)

This module is the Python binding: the ``sd_*`` functions mirror the C entry
points one to one (argument marshalling only; tensors are passed as device
pointers), and :func:`plan` / :func:`verify` allocate the outputs with torch
for convenience.  PyTorch provides device memory and streams, nothing else.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import (SD_NOALLOC_SCRATCH_BYTES, SD_BF16, SD_DEV_ERR_CACHE, SD_DEV_ERR_CONF, SD_DEV_ERR_COST, SD_DEV_ERR_CU_SEQLENS,  # noqa: F401
                   SD_DEV_ERR_DRAFT_ID, SD_DEV_ERR_DRAFT_LENS, SD_DEV_ERR_LOGITS, SD_DEV_ERR_OUTCOME,
                   SD_DEV_ERR_TEMP, SD_DEV_ERR_TIMEOUT, SD_DEV_ERR_TRUNC, SD_DEV_ERR_UNIFORM, SD_E4M3, SD_ERR_CUDA,
                   SD_ERR_DEVICE_CHECK, SD_ERR_INVALID_ARG, SD_ERR_SHAPE, SD_ERR_UNSUPPORTED,
                   SD_F32, SD_MAX_HEAD_DIM, SD_MAX_HEAD_GROUP, SD_MAX_K, SD_MAX_LEN, SD_MAX_PLAN_SLOTS, SD_MAX_ROW_BYTES, SD_MAX_SAMPLE_ROW_BYTES, SD_MAX_V, SD_MAX_VERIFY_BS,
                   SD_MODE_ADAPTIVE, SD_MODE_ALL_SLOTS, SD_MODE_UNIFORM_K, SD_OK,
                   SD_TEST_STALL, SD_VERIFY_DRAFT_PADDED, SD_VERIFY_EARLY_EXIT, SD_VERIFY_TEST_STALL, SdError,
                   sd_kv_cache, sd_launch_cfg)

__all__ = [
    "sd_plan", "sd_verify", "sd_verify_ex", "sd_verify_noalloc", "sd_plan_workspace_bytes",
    "sd_verify_workspace_bytes", "sd_verify_launch_info", "sd_calibrate", "sd_calibrate_apply",
    "sd_cache_append", "sd_attend_workspace_bytes", "sd_attend", "sd_attend_ex", "sd_sample", "sd_sample_ex",
    "plan", "verify", "append", "attend", "sample", "attend_workspace", "KVCache", "PlanResult",
    "VerifyResult", "AttendResult", "SampleResult", "SdError", "build", "library_path", "verify_workspace",
]


def build(force: bool = False):
    from ._build import build as _b
    return _b(force=force)


def library_path():
    return _lib.LIB_PATH


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a CUDA tensor, an int address or None, got {type(t)}")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


# The current stream's handle, without building a Stream object for it (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _torch_stream(stream):
    if isinstance(stream, int):  # 0, and 1 by name: the default stream
        return torch.cuda.default_stream() if stream in (0, 1) else torch.cuda.ExternalStream(stream)
    return stream


_CURRENT = contextlib.nullcontext()  # (made once: a call takes 8 us in all)


def _filling(stream):
    """Context in which torch allocates and fills on the stream that the call is given:
    fills are in order before the kernel, and memory that the call lets go of is handed
    out again behind it."""
    return _CURRENT if stream is None else torch.cuda.stream(_torch_stream(stream))


def _used_on(stream, *tensors):
    """The caller's tensors may be freed on return: their memory is not handed out again
    before the given stream has done the call."""
    s = _torch_stream(stream)
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(s)


def _dt(dt):
    if dt in (SD_F32, torch.float32):
        return SD_F32
    if dt in (SD_BF16, torch.bfloat16):
        return SD_BF16
    raise ValueError(f"unsupported logits dtype {dt}")


# ---------------------------------------------------------------------------
# C ABI mirror (same names and argument order as include/sd.h)


def sd_plan_workspace_bytes(bs: int, k_max: int) -> int:
    return _lib.load().sd_plan_workspace_bytes(bs, k_max)


def sd_verify_workspace_bytes(bs: int, k_max: int, V: int, dt) -> int:
    return _lib.load().sd_verify_workspace_bytes(int(bs), int(k_max), int(V), _dt(dt))


def sd_plan(conf_logits, budget_conf, budget_draft_lens, bs_budget, draft_lens, bs, k_max,
            cost_table, cost_len, T, mode, B_out, slot_mask, num_verified, cu_seqlens, err_flag,
            workspace=None, ws_bytes=0, stream=None):
    st = _lib.load().sd_plan(_ptr(conf_logits), _ptr(budget_conf), _ptr(budget_draft_lens),
                             int(bs_budget), _ptr(draft_lens), int(bs), int(k_max),
                             _ptr(cost_table), int(cost_len), int(T), int(mode), _ptr(B_out),
                             _ptr(slot_mask), _ptr(num_verified), _ptr(cu_seqlens),
                             _ptr(err_flag), _ptr(workspace), int(ws_bytes), _stream(stream))
    return _lib.check("sd_plan", st)


def sd_verify(target_logits, draft_logits, dt, V, draft_ids, uniforms, temps, cu_seqlens, bs,
              k_max, accepted_len, out_tokens, probs_out, err_flag, workspace, ws_bytes,
              stream=None):
    st = _lib.load().sd_verify(_ptr(target_logits), _ptr(draft_logits), _dt(dt), int(V),
                               _ptr(draft_ids), _ptr(uniforms), _ptr(temps), _ptr(cu_seqlens),
                               int(bs), int(k_max), _ptr(accepted_len), _ptr(out_tokens),
                               _ptr(probs_out), _ptr(err_flag), _ptr(workspace), int(ws_bytes),
                               _stream(stream))
    return _lib.check("sd_verify", st)


def sd_calibrate(conf_logits, draft_lens, num_verified, accepted_len, bs, k_max, lr, w, b,
                 err_flag, stream=None):
    st = _lib.load().sd_calibrate(_ptr(conf_logits), _ptr(draft_lens), _ptr(num_verified),
                                  _ptr(accepted_len), int(bs), int(k_max), float(lr), _ptr(w),
                                  _ptr(b), _ptr(err_flag), _stream(stream))
    return _lib.check("sd_calibrate", st)


def sd_calibrate_apply(conf_logits, draft_lens, bs, k_max, w, b, conf_out, err_flag, stream=None):
    st = _lib.load().sd_calibrate_apply(_ptr(conf_logits), _ptr(draft_lens), int(bs), int(k_max),
                                        _ptr(w), _ptr(b), _ptr(conf_out), _ptr(err_flag),
                                        _stream(stream))
    return _lib.check("sd_calibrate_apply", st)


def _cfg(cfg):
    """sd_launch_cfg from a dict with any of blocks, flags, wait_limit_us."""
    if cfg is None:
        return None
    if isinstance(cfg, sd_launch_cfg):
        return ctypes.byref(cfg)
    c = sd_launch_cfg(int(cfg.get("blocks", 0)), int(cfg.get("flags", 0)),
                      int(cfg.get("wait_limit_us", 0)), 0)
    return ctypes.byref(c)


def sd_verify_ex(target_logits, draft_logits, dt, V, draft_ids, uniforms, temps, cu_seqlens, bs,
                 k_max, accepted_len, out_tokens, probs_out, err_flag, workspace, ws_bytes,
                 cfg=None, stream=None):
    st = _lib.load().sd_verify_ex(_ptr(target_logits), _ptr(draft_logits), _dt(dt), int(V),
                                  _ptr(draft_ids), _ptr(uniforms), _ptr(temps), _ptr(cu_seqlens),
                                  int(bs), int(k_max), _ptr(accepted_len), _ptr(out_tokens),
                                  _ptr(probs_out), _ptr(err_flag), _ptr(workspace), int(ws_bytes),
                                  _cfg(cfg), _stream(stream))
    return _lib.check("sd_verify_ex", st)


def sd_verify_noalloc(target_logits, draft_logits, dt, V, draft_ids, uniforms, temps, cu_seqlens,
                      bs, k_max, accepted_len, out_tokens, probs_out, err_flag, stream=None):
    st = _lib.load().sd_verify_noalloc(_ptr(target_logits), _ptr(draft_logits), _dt(dt), int(V),
                                       _ptr(draft_ids), _ptr(uniforms), _ptr(temps),
                                       _ptr(cu_seqlens), int(bs), int(k_max), _ptr(accepted_len),
                                       _ptr(out_tokens), _ptr(probs_out), _ptr(err_flag),
                                       _stream(stream))
    return _lib.check("sd_verify_noalloc", st)


def sd_verify_launch_info(V, dt, bs, blocks=0, flags=0) -> dict:
    req = sd_launch_cfg(int(blocks), int(flags), 0, 0)
    out = sd_launch_cfg()
    threads, buffers = ctypes.c_int(0), ctypes.c_int(0)
    smem = ctypes.c_size_t(0)
    st = _lib.load().sd_verify_launch_info(int(V), _dt(dt), int(bs), ctypes.byref(req),
                                           ctypes.byref(out), ctypes.byref(threads),
                                           ctypes.byref(buffers), ctypes.byref(smem))
    _lib.check("sd_verify_launch_info", st)
    return {"blocks": out.blocks, "threads": threads.value, "buffers": buffers.value,
            "smem_bytes": smem.value}


def verify_workspace(bs: int, k_max: int, V: int, dt, device=None) -> torch.Tensor:
    """A zero-filled workspace for sd_verify (zero-filled once; calls keep it
    so).  torch's CUDA allocations are 256-byte aligned, as the call requires."""
    return torch.zeros(sd_verify_workspace_bytes(bs, k_max, V, dt), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


# ---------------------------------------------------------------------------
# Convenience layer: allocate outputs with torch and call the C ABI.  What is
# allocated here belongs to `stream`, as if the call stood under
# torch.cuda.stream(stream); inputs have to be ready on it.


@dataclass
class PlanResult:
    B: torch.Tensor             # [1] int32
    slot_mask: torch.Tensor     # [bs, k_max] uint8
    num_verified: torch.Tensor  # [bs] int32
    cu_seqlens: torch.Tensor    # [bs+1] int32
    err: torch.Tensor           # [1] int32


@dataclass
class VerifyResult:
    accepted_len: torch.Tensor  # [bs] int32
    out_tokens: torch.Tensor    # [bs, k_max+1] int32
    probs: Optional[torch.Tensor]  # [bs*k_max, 2] fp32 or None
    err: torch.Tensor           # [1] int32


def plan(draft_lens: torch.Tensor, k_max: int, conf: Optional[torch.Tensor] = None,
         cost: Optional[torch.Tensor] = None, T: int = 0, mode: int = SD_MODE_ADAPTIVE,
         budget_conf: Optional[torch.Tensor] = None,
         budget_draft_lens: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
         stream=None) -> PlanResult:
    dev = draft_lens.device
    bs = draft_lens.numel()
    bsb = 0 if budget_draft_lens is None else budget_draft_lens.numel()
    with _filling(stream):
        B = torch.empty(1, dtype=torch.int32, device=dev)
        mask = torch.empty((bs, max(k_max, 1)), dtype=torch.uint8, device=dev)
        nv = torch.empty(bs, dtype=torch.int32, device=dev)
        cu = torch.empty(bs + 1, dtype=torch.int32, device=dev)
        if err is None:
            err = torch.zeros(1, dtype=torch.int32, device=dev)
        # an empty packed array is still a valid (unread) buffer for the C ABI
        if conf is not None and conf.numel() == 0:
            conf = torch.zeros(1, dtype=torch.float32, device=dev)
        if budget_conf is not None and budget_conf.numel() == 0:
            budget_conf = torch.zeros(1, dtype=torch.float32, device=dev)
    sd_plan(conf, budget_conf, budget_draft_lens, bsb, draft_lens, bs, k_max, cost,
            0 if cost is None else cost.numel(), T, mode, B, mask, nv, cu, err, None, 0, stream)
    if stream is not None:
        _used_on(stream, draft_lens, conf, cost, budget_conf, budget_draft_lens, err)
    return PlanResult(B, mask[:, :k_max], nv, cu, err)


def verify(target: torch.Tensor, draft: Optional[torch.Tensor], dt, V: int,
           draft_ids: torch.Tensor, uniforms: torch.Tensor, temps: torch.Tensor,
           cu_seqlens: torch.Tensor, k_max: int, probs: bool = False,
           err: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           cfg=None, stream=None) -> VerifyResult:
    dev = target.device
    bs = cu_seqlens.numel() - 1
    with _filling(stream):
        acc = torch.empty(bs, dtype=torch.int32, device=dev)
        out = torch.empty((bs, k_max + 1), dtype=torch.int32, device=dev)
        pr = torch.full((max(bs * k_max, 1), 2), float("nan"), dtype=torch.float32, device=dev) if probs else None
        if err is None:
            err = torch.zeros(1, dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = verify_workspace(bs, k_max, V, dt, dev)
    sd_verify_ex(target, draft, dt, V, draft_ids, uniforms, temps, cu_seqlens, bs, k_max, acc,
                 out, pr, err, workspace, workspace.numel(), cfg=cfg, stream=stream)
    if stream is not None:
        _used_on(stream, target, draft, draft_ids, uniforms, temps, cu_seqlens, err, workspace)
    return VerifyResult(acc, out, pr, err)


# ---------------------------------------------------------------------------
# The operators around the step: paged cache, attention, truncated sampling


class KVCache:
    """A paged key-value cache over the caller's tensors (nothing is copied).

    k, v         [pages, page_size, heads, head_dim], bf16 or float8_e4m3fn, of
                 equal strides, head_dim contiguous.  A cache kept as
                 [pages, heads, page_size, head_dim] is passed as its
                 ``permute(0, 2, 1, 3)``.
    page_table   [bs, max_pages] int32
    k_scale, v_scale   [heads] fp32, for an 8-bit cache: value = stored * scale

    The handle keeps the tensors alive; rows of ``page_table`` may be
    rewritten in place between calls.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-dimensional, of one shape, strides and dtype")
        if k.stride(3) != 1:
            raise ValueError("the head dimension must be contiguous")
        if page_table.dim() != 2 or page_table.dtype != torch.int32:
            raise ValueError("page_table must be [bs, max_pages] int32")
        if k.dtype == torch.bfloat16:
            self.dt = SD_BF16
        elif k.dtype == torch.float8_e4m3fn:
            self.dt = SD_E4M3
        else:
            raise ValueError(f"unsupported cache dtype {k.dtype}")
        self.k, self.v, self.page_table, self.k_scale, self.v_scale = k, v, page_table, k_scale, v_scale
        self.num_pages, self.page_size, self.heads, self.head_dim = k.shape
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or s.shape != (self.heads,)):
                raise ValueError("scales must be [heads] fp32")
        for t in (k, v):
            if not t.is_cuda:
                raise ValueError("tensor arguments must live on the GPU")
        self.c = sd_kv_cache(k.data_ptr(), v.data_ptr(), _ptr(page_table), _ptr(k_scale),
                             _ptr(v_scale), k.stride(0), k.stride(1), k.stride(2), self.dt,
                             self.num_pages, self.page_size, page_table.shape[1], self.heads,
                             self.head_dim)

    def tensors(self):
        return self.k, self.v, self.page_table, self.k_scale, self.v_scale


def _cache(cache):
    return ctypes.byref(cache.c if isinstance(cache, KVCache) else cache)


def _rows(t, heads, dim):
    """(address, row stride) of bf16 rows [rows, heads, dim] with heads and dim contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
        raise ValueError("rows must be a bf16 tensor")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or stride[2] != 1 or \
            (heads > 1 and stride[1] != dim):
        raise ValueError(f"rows must be [rows, {heads}, {dim}] with heads and elements contiguous")
    # a single row's stride is never used to step and may be anything
    return t.data_ptr(), stride[0] if shape[0] > 1 else max(stride[0], heads * dim)


def sd_cache_append(k_new, v_new, row_stride, cache, cu_seqlens, kv_lens, bs, k_max, err_flag,
                    stream=None):
    k_new, v_new = (t if isinstance(t, int) else t.data_ptr() for t in (k_new, v_new))
    st = _lib.load().sd_cache_append(k_new, v_new, int(row_stride), _cache(cache),
                                     _ptr(cu_seqlens), _ptr(kv_lens), int(bs), int(k_max),
                                     _ptr(err_flag), _stream(stream))
    return _lib.check("sd_cache_append", st)


def sd_attend_workspace_bytes(bs: int, k_max: int, q_heads: int, heads: int, head_dim: int) -> int:
    return _lib.load().sd_attend_workspace_bytes(int(bs), int(k_max), int(q_heads), int(heads),
                                                 int(head_dim))


def sd_attend(q, q_row_stride, q_heads, cache, cu_seqlens, kv_lens, bs, k_max, scale, out, lse_out,
              err_flag, workspace, ws_bytes, stream=None):
    st = _lib.load().sd_attend(q if isinstance(q, int) else q.data_ptr(), int(q_row_stride),
                               int(q_heads), _cache(cache), _ptr(cu_seqlens), _ptr(kv_lens),
                               int(bs), int(k_max), float(scale), _ptr(out), _ptr(lse_out),
                               _ptr(err_flag), _ptr(workspace), int(ws_bytes), _stream(stream))
    return _lib.check("sd_attend", st)


def sd_sample(logits, dt, V, rows, cu_seqlens, bs, temps, top_k, top_p, min_p, uniforms, tokens,
              kept_out, err_flag, stream=None):
    st = _lib.load().sd_sample(_ptr(logits), _dt(dt), int(V), int(rows), _ptr(cu_seqlens), int(bs),
                               _ptr(temps), _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(uniforms),
                               _ptr(tokens), _ptr(kept_out), _ptr(err_flag), _stream(stream))
    return _lib.check("sd_sample", st)


def sd_attend_ex(q, q_row_stride, q_heads, cache, cu_seqlens, kv_lens, bs, k_max, scale, out,
                 lse_out, err_flag, workspace, ws_bytes, cfg=None, stream=None):
    st = _lib.load().sd_attend_ex(q if isinstance(q, int) else q.data_ptr(), int(q_row_stride),
                                  int(q_heads), _cache(cache), _ptr(cu_seqlens), _ptr(kv_lens),
                                  int(bs), int(k_max), float(scale), _ptr(out), _ptr(lse_out),
                                  _ptr(err_flag), _ptr(workspace), int(ws_bytes), _cfg(cfg),
                                  _stream(stream))
    return _lib.check("sd_attend_ex", st)


def sd_sample_ex(logits, dt, V, rows, cu_seqlens, bs, temps, top_k, top_p, min_p, uniforms, tokens,
                 kept_out, err_flag, cfg=None, stream=None):
    st = _lib.load().sd_sample_ex(_ptr(logits), _dt(dt), int(V), int(rows), _ptr(cu_seqlens),
                                  int(bs), _ptr(temps), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                                  _ptr(uniforms), _ptr(tokens), _ptr(kept_out), _ptr(err_flag),
                                  _cfg(cfg), _stream(stream))
    return _lib.check("sd_sample_ex", st)


def attend_workspace(bs: int, k_max: int, q_heads: int, cache: KVCache, device=None) -> torch.Tensor:
    """A zero-filled workspace for sd_attend (zero-filled once; calls keep it so)."""
    n = sd_attend_workspace_bytes(bs, k_max, q_heads, cache.heads, cache.head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device or cache.k.device)


@dataclass
class AttendResult:
    out: torch.Tensor            # [rows, q_heads, head_dim] bf16
    lse: Optional[torch.Tensor]  # [rows, q_heads] fp32 or None
    err: torch.Tensor            # [1] int32


@dataclass
class SampleResult:
    tokens: Optional[torch.Tensor]  # [rows] int32, or None when nothing was drawn
    kept: Optional[torch.Tensor]    # [rows, V], the truncated rows, or None
    err: torch.Tensor               # [1] int32


_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def _need(t, what, dtype, n):
    """Refuses a tensor that is not one-dimensional, of another type, or shorter than n."""
    if t is not None and (t.dtype != dtype or t.dim() != 1 or t.shape[0] < n):
        raise ValueError(f"{what} must be {dtype} [at least {n}]")


def _step(cache, cu_seqlens, kv_lens):
    """The batch size, after checking what the step passes along."""
    _need(cu_seqlens, "cu_seqlens", _I32, 2)
    bs = cu_seqlens.shape[0] - 1
    _need(kv_lens, "kv_lens", _I32, bs)
    if cache.page_table.shape[0] < bs:
        raise ValueError(f"the page table has {cache.page_table.shape[0]} rows for {bs} requests")
    return bs


def append(k_new: torch.Tensor, v_new: torch.Tensor, cache: KVCache, cu_seqlens: torch.Tensor,
           kv_lens: torch.Tensor, k_max: int, err: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """Writes the step's rows (packed by cu_seqlens) into the cache, in place; returns err."""
    bs = _step(cache, cu_seqlens, kv_lens)
    ka, ks = _rows(k_new, cache.heads, cache.head_dim)
    va, vs = _rows(v_new, cache.heads, cache.head_dim)
    if k_new.shape[0] != v_new.shape[0] or ks != vs:
        raise ValueError("k_new and v_new must have the same rows and row stride")
    if k_new.shape[0] < bs * (k_max + 1):
        raise ValueError(f"rows for {bs} requests of up to {k_max + 1} are needed")
    if err is None:
        with _filling(stream):
            err = torch.zeros(1, dtype=torch.int32, device=cache.k.device)
    sd_cache_append(ka, va, ks, cache, cu_seqlens, kv_lens, bs, k_max, err, stream)
    if stream is not None:
        _used_on(stream, k_new, v_new, cu_seqlens, kv_lens, err, *cache.tensors())
    return err


def attend(q: torch.Tensor, cache: KVCache, cu_seqlens: torch.Tensor, kv_lens: torch.Tensor,
           k_max: int, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
           lse=False, err: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           stream=None) -> AttendResult:
    """Attention of the step's rows over the cache (scale: 1/sqrt(head_dim) unless given).

    Rows from cu_seqlens[-1] on are left as they are in `out` and `lse`
    (zeros where they are allocated here).  lse: True, or a tensor to fill.
    """
    bs = _step(cache, cu_seqlens, kv_lens)
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    rows, q_heads, dim = q.shape
    qa, qs = _rows(q, q_heads, cache.head_dim)
    if rows < bs * (k_max + 1):
        raise ValueError(f"rows for {bs} requests of up to {k_max + 1} are needed")
    with _filling(stream):
        if out is None:
            out = torch.zeros((rows, q_heads, dim), dtype=torch.bfloat16, device=q.device)
        if lse is True:
            lse = torch.zeros((rows, q_heads), dtype=torch.float32, device=q.device)
        if err is None:
            err = torch.zeros(1, dtype=torch.int32, device=q.device)
        if workspace is None:
            workspace = attend_workspace(bs, k_max, q_heads, cache)
    lse = None if lse is False else lse
    if out.dtype != _BF16 or out.dim() != 3 or out.shape[1:] != q.shape[1:] or out.shape[0] < bs * (k_max + 1):
        raise ValueError(f"out must be bf16 [at least {bs * (k_max + 1)}, {q_heads}, {dim}]")
    if lse is not None and (lse.dtype != _F32 or lse.dim() != 2 or lse.shape[1] != q_heads or
                            lse.shape[0] < bs * (k_max + 1)):
        raise ValueError(f"lse must be fp32 [at least {bs * (k_max + 1)}, {q_heads}]")
    sd_attend(qa, qs, q_heads, cache, cu_seqlens, kv_lens, bs, k_max,
              dim ** -0.5 if scale is None else scale, out, lse, err, workspace, workspace.numel(),
              stream)
    if stream is not None:
        _used_on(stream, q, cu_seqlens, kv_lens, out, lse, err, workspace, *cache.tensors())
    return AttendResult(out, lse, err)


def sample(logits: torch.Tensor, temps: torch.Tensor, uniforms: Optional[torch.Tensor] = None,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
           tokens: Optional[torch.Tensor] = None, kept=False, err: Optional[torch.Tensor] = None,
           stream=None) -> SampleResult:
    """Truncated sampling of rows [rows, V] (fp32 or bf16).

    uniforms None: nothing is drawn.  kept: True, or a tensor to fill (logits
    itself among them): the truncated rows, -inf where a token was dropped.
    cu_seqlens: parameters are per request and rows are a step's packed rows.
    """
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    rows, V = logits.shape
    bs = rows if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(temps, "temps", _F32, bs)
    _need(top_k, "top_k", _I32, bs)
    _need(top_p, "top_p", _F32, bs)
    _need(min_p, "min_p", _F32, bs)
    _need(uniforms, "uniforms", _F32, rows)
    _need(cu_seqlens, "cu_seqlens", _I32, 2)
    if uniforms is None:
        if tokens is not None:
            raise ValueError("tokens are drawn from uniforms: pass both or neither")
    with _filling(stream):
        if uniforms is not None and tokens is None:
            tokens = torch.zeros(rows, dtype=torch.int32, device=logits.device)
        if kept is True:
            kept = torch.zeros_like(logits)
        if err is None:
            err = torch.zeros(1, dtype=torch.int32, device=logits.device)
    _need(tokens, "tokens", _I32, rows)
    kept = None if kept is False else kept
    if kept is not None and (kept.shape != logits.shape or kept.dtype != logits.dtype):
        raise ValueError("kept must have the logits' shape and dtype")
    sd_sample(logits, logits.dtype, V, rows, cu_seqlens, bs, temps, top_k, top_p, min_p, uniforms,
              tokens, kept, err, stream)
    if stream is not None:
        _used_on(stream, logits, temps, uniforms, top_k, top_p, min_p, cu_seqlens, tokens, kept, err)
    return SampleResult(tokens, kept, err)
