"""The operators of a served batch's decode step, beside those of drafted.py.

    norm = HeadNorm(q_weight, k_weight, eps=1e-6)
    cache = mx_cache(pages, page, kv_heads, dim, table, length, format="mx8")   # keys and values in 8 (or 4) bits
    q = cache.append(rope, q, k_new, v_new, row_start, norm=norm)              # normed, rotated, written in one pass
    shared = SharedPrefix(group_start, prompt_length)                          # requests that begin alike
    o = cache.attend(q, row_start, shared=shared)                              # the common tokens are read once
    ... the rest of the layers, logits ...
    tokens, logprobs = sampler.sample(logits, u, temperature=t, top_k=k, top_p=p, min_p=m)

HeadNorm and SharedPrefix serve a PagedCache (16 bits) as well; an MxCache has all of its methods. torch holds
the memory and names the stream; every computation runs in the library's HIP kernels (include/moe_serving.h states what
each computes). Conventions as in drafted.py.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import binding as B
from .drafted import (_DEVICE, _DT, _DTYPE, _INVALID, _LAYOUT_ERR, _LIB, _ROWS, _SHAPE, PagedCache, _Caller, _refuse,
                      _tensor)

_FORMAT = {"mx8": B.MOE_MX8, "mx4": B.MOE_MX4}


class HeadNorm:
    """RMS norm of every head of queries and keys before it turns: x / sqrt(mean(x^2) + eps) * (offset + weight).

    q_weight [dim] (one for all heads) or [heads][dim], k_weight [dim] or [kv_heads][dim]; f32, bf16 or f16, both the
    same. offset: 1 for weights that are stored as differences from 1. The tensors are kept alive by this object."""

    def __init__(self, q_weight: torch.Tensor, k_weight: torch.Tensor, eps: float = 1e-6, offset: float = 0.0):
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w.dtype not in (torch.float32, torch.bfloat16, torch.float16) or w.dtype != q_weight.dtype:
                _refuse(_DTYPE, f"norm {name}: {w.dtype} (float32, bfloat16 or float16, both the same)")
            if w.dim() not in (1, 2) or not w.numel():
                _refuse(_LAYOUT_ERR, f"norm {name}: shape {tuple(w.shape)}, expected (dim,) or (heads, dim)")
            if w.stride(-1) != 1 and w.shape[-1] > 1:
                _refuse(_LAYOUT_ERR, f"norm {name}: last dim not contiguous")
        if not (math.isfinite(eps) and eps >= 0 and math.isfinite(offset)):
            _refuse(_INVALID, f"norm: eps {eps}, offset {offset}")
        self.q_weight, self.k_weight = q_weight, k_weight
        # one row of weights for one head is one for all
        qs, ks = (w.stride(0) if w.dim() == 2 and w.shape[0] > 1 else 0 for w in (q_weight, k_weight))
        self._c = B.moe_head_norm(q_weight.data_ptr(), k_weight.data_ptr(), qs, ks, _DT[q_weight.dtype], eps, offset)
        self._ref = ctypes.addressof(self._c)
        self._fits = None

    def _check(self, device: torch.device, index: int, heads: int, kv_heads: int, dim: int) -> None:
        if self._fits == (index, heads, kv_heads, dim):      # the weights do not change
            return
        for name, w, n in (("q_weight", self.q_weight, heads), ("k_weight", self.k_weight, kv_heads)):
            if w.shape[-1] != dim or (w.dim() == 2 and w.shape[0] != n):
                _refuse(_SHAPE, f"norm {name}: shape {tuple(w.shape)}, expected ({dim},) or ({n}, {dim})")
            if w.get_device() != index:
                _refuse(_DEVICE, f"norm {name}: on {w.device}, the cache is on {device}")
        self._fits = (index, heads, kv_heads, dim)


class SharedPrefix:
    """Sequences that begin with the same tokens: group g has the sequences group_start[g] to group_start[g + 1] - 1, whose first
    length[g] tokens are the same (read from the pages of the group's first one). group_start [groups + 1], ascending from 0 to
    the number of sequences, and length [groups], both i32 on the device; a call reads what they hold when it runs."""

    def __init__(self, group_start: torch.Tensor, length: torch.Tensor):
        for name, t in (("group_start", group_start), ("length", length)):
            if t.dtype != torch.int32:
                _refuse(_DTYPE, f"shared {name}: {t.dtype}, expected torch.int32")
            if t.dim() != 1 or not t.is_contiguous():
                _refuse(_LAYOUT_ERR, f"shared {name}: a contiguous vector")
        self.groups = length.shape[0]
        if self.groups < 1 or group_start.shape[0] != self.groups + 1:
            _refuse(_SHAPE, f"shared group_start: {group_start.shape[0]} starts of {self.groups} groups")
        self.group_start, self.length = group_start, length
        self._c = B.moe_shared_prefix(group_start.data_ptr(), length.data_ptr(), self.groups)
        self._ref = ctypes.addressof(self._c)

    def _check(self, device: torch.device, index: int, seqs: int) -> None:
        if self.groups > seqs:
            _refuse(_SHAPE, f"shared: {self.groups} groups, {seqs} sequences")
        for name, t in (("group_start", self.group_start), ("length", self.length)):
            if t.get_device() != index:
                _refuse(_DEVICE, f"shared {name}: on {t.device}, the cache is on {device}")


class MxCache(PagedCache):
    """A paged cache whose keys and values are held in blocks of 32 along a head, codes under a power of two: format "mx8"
    (e4m3, 8.25 bits a value) or "mx4" (e2m1, 4.25 bits). Methods as PagedCache's, and read().

    k, v [pages][page][kv_heads][dim or dim / 2] and k_scale, v_scale [pages][page][kv_heads][dim / 32], all uint8, over
    tensors that the caller owns (mx_cache() lays them out as they are read fastest); dim 32, 64, 96, 128, 192 or 256. dtype: of the
    rows that are appended, of queries and results, and what codes are read as."""

    _append_call, _keep_call, _plain_append = _LIB.moe_mx_append, _LIB.moe_mx_keep, False

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, table: torch.Tensor,
                 length: torch.Tensor, format: str = "mx8", dtype: torch.dtype = torch.bfloat16):
        _Caller.__init__(self, k.device)
        if format not in _FORMAT:
            _refuse(_INVALID, f"cache format {format!r} (mx8 or mx4)")
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale), ("table", table), ("len", length)):
            if t.device != k.device:
                _refuse(_DEVICE, f"cache {name}: on {t.device}, k is on {k.device}")
        self.k, self.v, self.k_scale, self.v_scale, self.table, self.length = k, v, k_scale, v_scale, table, length
        self._c = B.moe_mx_cache(_tensor(k), _tensor(v), _tensor(k_scale), _tensor(v_scale), _tensor(table),
                                 _tensor(length), self._flags_ptr, _FORMAT[format], _DT.get(dtype, 0))
        self._ref = ctypes.addressof(self._c)
        B._check(_LIB.moe_mx_cache_check(self._ref))
        self.dtype, self.format = dtype, format
        self.seqs, self.kv_heads, self.dim = table.shape[0], k.shape[2], k.shape[3] * (1 if format == "mx8" else 2)

    def read(self, row_start: torch.Tensor, rows: int, start: Optional[torch.Tensor] = None,
             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Keys and values that the cache holds, [rows][kv_heads * dim] in its dtype: row i of sequence b (row_start says which rows
        are whose) is token start[b] + i (start [seqs] i32; None: the length, so what append() wrote for the step's rows).
        out: a pair of tensors to write to; rows of tokens that the cache does not have are left as they were."""
        width = self.kv_heads * self.dim
        sp = self._vector("row_start", row_start, torch.int32, self.seqs + 1)
        tp = None if start is None else self._vector("start", start, torch.int32, self.seqs)
        if out is None:
            k, v = out = (torch.empty((rows, width), dtype=self.dtype, device=self.device),
                          torch.empty((rows, width), dtype=self.dtype, device=self.device))
            kp, vp, ks, vs = k.data_ptr(), v.data_ptr(), width, width
        else:
            kp, ks = self._matrix("out k", out[0], self.dtype, rows, width)
            vp, vs = self._matrix("out v", out[1], self.dtype, rows, width)
        self._launch(_LIB.moe_mx_read, self._ref, rows, sp, tp, kp, ks, vp, vs)
        return out

    def _attend_workspace(self, shared, rows: int, heads: int) -> int:
        return _LIB.moe_mx_attend_workspace(self._ref, 0 if shared is None else shared.groups, rows, heads)

    def _attend(self, shared, *args) -> None:
        self._launch(_LIB.moe_mx_attend, self._ref, None if shared is None else shared._ref, *args)


def mx_cache(pages: int, page: int, kv_heads: int, dim: int, table: torch.Tensor, length: torch.Tensor, format: str = "mx8",
             dtype: torch.dtype = torch.bfloat16) -> MxCache:
    """An MxCache with memory of its own on the table's device, zeroed: a head's tokens of a page lie side by side, and so do
    their scales, which is how attention reads them."""
    if format not in _FORMAT:
        _refuse(_INVALID, f"cache format {format!r} (mx8 or mx4)")
    if dim < 32 or dim % 32:
        _refuse(_SHAPE, f"cache: head width {dim} (32, 64, 96, 128, 192 or 256)")
    codes, scales = (torch.zeros((2, pages, kv_heads, page, w), dtype=torch.uint8, device=table.device).transpose(2, 3)
                     for w in (dim if format == "mx8" else dim // 2, dim // 32))
    return MxCache(codes[0], codes[1], scales[0], scales[1], table, length, format, dtype)


class Sampler(_Caller):
    """Draws a token for each row of logits, for up to max_rows rows over one vocabulary."""

    def __init__(self, vocab: int, max_rows: int, device="cuda"):
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        super().__init__(device)
        need = _LIB.moe_sample_workspace(max_rows, vocab)
        if need < 0:
            B._check(-need)
        self.vocab, self.max_rows = vocab, max_rows

    def sample(self, logits: torch.Tensor, u: torch.Tensor, temperature: Optional[torch.Tensor] = None,
               top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
               min_p: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """tokens [rows] i32 and logprobs [rows] f32 (rules in include/moe_serving.h).

        logits [rows][vocab] f32, bf16 or f16; u [rows] f32 in [0, 1); temperature [rows] f32 (None: 1; 0 or less: the
        largest logit); top_k [rows] i32 (0 or less: no cut), top_p [rows] f32 (1 or more: no cut), min_p [rows] f32 (0 or
        less: no cut), each None: no cut."""
        if logits.dim() != 2:
            _refuse(_LAYOUT_ERR, f"logits: rank {logits.dim()}, expected 2")
        rows = logits.shape[0]
        if not 1 <= rows <= self.max_rows:
            _refuse(_ROWS, f"{rows} rows: 1 to {self.max_rows}")
        if logits.dtype not in (torch.float32, torch.bfloat16, torch.float16):
            _refuse(_DTYPE, f"logits: {logits.dtype} (float32, bfloat16 or float16)")
        zp, zs = self._matrix("logits", logits, logits.dtype, rows, self.vocab)
        z = B.make_tensor(zp, _DT[logits.dtype], (rows, self.vocab), (zs, 1))
        up = self._vector("u", u, torch.float32, rows)
        Tp = None if temperature is None else self._vector("temperature", temperature, torch.float32, rows)
        kp = None if top_k is None else self._vector("top_k", top_k, torch.int32, rows)
        pp = None if top_p is None else self._vector("top_p", top_p, torch.float32, rows)
        mp = None if min_p is None else self._vector("min_p", min_p, torch.float32, rows)
        need = _LIB.moe_sample_workspace(rows, self.vocab)
        if need < 0:
            B._check(-need)
        tokens = torch.empty(rows, dtype=torch.int32, device=self.device)
        logprobs = torch.empty(rows, dtype=torch.float32, device=self.device)
        # from the stream's own pool each time, so that calls on several streams do not share it
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._launch(_LIB.moe_sample, ctypes.byref(z), up, Tp, kp, pp, mp, tokens.data_ptr(), logprobs.data_ptr(),
                     self._flags_ptr, ws.data_ptr(), need)
        return tokens, logprobs
