"""The operators of a drafted (speculative) decode step over a paged key/value cache.

A step passes, for every sequence, its last certain token and the tokens drafted after it (a
chain, or a tree) through the model at once. Row 0 of a sequence is the certain token; row_start
[seqs + 1] says where each sequence's rows begin. Beside the expert layer (layer.py) and the lm_head:

    cache = PagedCache(k, v, table, length)          # borrowed tensors, kept alive by the object
    rope = Rope(*rope_frequencies(128), layout="half")
    q = cache.append(rope, q, k_new, v_new, row_start, positions=positions)
    o = cache.attend(q, row_start, mask=mask)
    ... the rest of the layers, logits ...
    n_keep, path, tokens, logprobs = verifier.verify(logits, drafted, row_start, u_test, u_pick,
                                                     parent=parent, draft_probs=probs)
    keep_paths(caches, row_start, n_keep, path)      # of all layers, whose lengths may be one tensor

torch holds the memory and names the stream; every computation runs in the library's HIP kernels
(include/moe_drafted.h states what each computes). Calls check their tensors, enqueue on torch's
current stream of the tensors' device and return; they can be captured in a HIP graph. What only the
device can see is checked there and reported by status().
"""
from __future__ import annotations

import ctypes
import math
from typing import List, Optional, Sequence, Tuple

import torch

from . import binding as B

_LIB = B.lib()
_DT = {torch.bfloat16: B.MOE_DT_BF16, torch.float16: B.MOE_DT_F16, torch.float32: B.MOE_DT_F32,
       torch.int32: B.MOE_DT_I32}
_LAYOUT = {"half": B.MOE_ROPE_HALF, "interleaved": B.MOE_ROPE_INTERLEAVED}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _refuse(status: int, message: str):
    raise B.MoeError(status, message)


_INVALID, _SHAPE, _MISSING, _DTYPE, _ROWS = 1, 4, 5, 6, 10
_LAYOUT_ERR, _DEVICE = 7, 9


def _tensor(t: torch.Tensor) -> B.moe_tensor:
    """A descriptor of t: its address, type, shape and strides as they are."""
    if not 1 <= t.dim() <= 4:
        _refuse(_LAYOUT_ERR, f"rank {t.dim()} (1 to 4)")
    return B.make_tensor(t.data_ptr(), _DT.get(t.dtype, 0), list(t.shape), list(t.stride()))


class _Caller:
    """What the classes below share: the device their tensors lie on, streams, flags, checks."""

    def __init__(self, device: torch.device):
        self.device = device
        self.index = -1 if device.index is None else device.index
        # copied from the host, which waits: any stream may use it from here on
        self.flags = torch.zeros(1, dtype=torch.int32).to(device)
        self._flags_ptr = self.flags.data_ptr()

    def _stream(self) -> int:
        if self.index < 0:
            _refuse(_DEVICE, f"tensors on {self.device}: the kernels need a GPU")
        return _raw_stream(self.index) if _raw_stream else torch.cuda.current_stream(self.device).cuda_stream

    def _launch(self, call, *args) -> None:
        """call(*args, stream) of the library on the tensors' device, made the current one where it is not; raises
        what it refuses."""
        stream = self._stream()
        if _current_device() == self.index:
            B._check(call(*args, stream))
        else:
            with torch.cuda.device(self.index):
                B._check(call(*args, stream))

    def _vector(self, name: str, t: torch.Tensor, dtype: torch.dtype, n: int) -> int:
        """The address of a contiguous vector of n elements."""
        if t.dtype != dtype:
            _refuse(_DTYPE, f"{name}: {t.dtype}, expected {dtype}")
        if t.shape != (n,):
            _refuse(_SHAPE, f"{name}: shape {tuple(t.shape)}, expected ({n},)")
        if not t.is_contiguous():
            _refuse(_LAYOUT_ERR, f"{name}: not contiguous")
        if t.get_device() != self.index:
            _refuse(_DEVICE, f"{name}: on {t.device}, expected {self.device}")
        return t.data_ptr()

    def _matrix(self, name: str, t: torch.Tensor, dtype: torch.dtype, rows: int, width: int) -> Tuple[int, int]:
        """The address and row stride of a [rows][width] matrix with contiguous rows."""
        if t.dtype != dtype:
            _refuse(_DTYPE, f"{name}: {t.dtype}, expected {dtype}")
        if t.shape != (rows, width):
            _refuse(_SHAPE, f"{name}: shape {tuple(t.shape)}, expected ({rows}, {width})")
        if t.get_device() != self.index:
            _refuse(_DEVICE, f"{name}: on {t.device}, expected {self.device}")
        stride, last = t.stride()
        if last != 1 and width > 1:
            _refuse(_LAYOUT_ERR, f"{name}: columns not contiguous")
        return t.data_ptr(), stride if rows > 1 else width      # that of a single row means nothing

    def status(self) -> None:
        """Wait for the current stream's work; raise MOE_ERR_DEVICE_CHECK if a call since the last status()
        met something wrong on the device (a page outside the cache, a path out of order, ...)."""
        self._launch(_LIB.moe_drafted_status, self._flags_ptr)


class Rope:
    """Rotary positions: pair j of a head at position t turns by t * freqs[j] radians.

    freqs: [pairs] 64-bit radians per position (a tensor or a list; copied to the device once).
    layout: "half" pairs dims (j, j + pairs), "interleaved" (2 j, 2 j + 1); the dims after the
    first 2 * pairs stay. magnitude: factor on cosine and sine (of a scaling method)."""

    def __init__(self, freqs, magnitude: float = 1.0, layout: str = "half", device="cuda"):
        if layout not in _LAYOUT:
            _refuse(_INVALID, f"rope layout {layout!r} (half or interleaved)")
        f = torch.as_tensor(freqs, dtype=torch.float64)
        if f.dim() != 1 or f.numel() < 1:
            _refuse(_SHAPE, f"rope freqs: shape {tuple(f.shape)}, expected (pairs,)")
        if not math.isfinite(magnitude):
            _refuse(_INVALID, "rope magnitude is not finite")
        self.freqs = (f if f.device.type == torch.device(device).type else f.to(device)).contiguous()
        self.layout, self.magnitude = layout, float(magnitude)
        self._c = B.moe_rope(self.freqs.data_ptr(), f.numel(), _LAYOUT[layout], self.magnitude)
        self._ref = ctypes.addressof(self._c)


def rope_frequencies(rotary: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained: int = 8192, fast: float = 32.0, slow: float = 1.0) -> Tuple[torch.Tensor, float]:
    """Frequencies [rotary / 2] (64-bit radians per position) and the magnitude, for Rope.

    scaling, for a context `factor` times the trained one: "linear" stretches positions; "base"
    takes a larger base, so that the slowest pair is stretched by `factor` and the fastest not; "parts"
    leaves pairs that turn `fast` times or more in the trained length, stretches those that turn
    `slow` times or less, blends between, and raises the magnitude with the log of the factor."""
    if rotary < 2 or rotary % 2:
        _refuse(_SHAPE, f"rotary {rotary}: a positive even number of dims")
    if scaling not in ("none", "linear", "base", "parts"):
        _refuse(_INVALID, f"rope scaling {scaling!r}")
    if not (factor > 0 and base > 0):
        _refuse(_INVALID, "rope base and factor must be positive")
    j = torch.arange(rotary // 2, dtype=torch.float64)
    if scaling == "base" and rotary > 2:
        base = base * factor ** (rotary / (rotary - 2))
    f = base ** (-2.0 * j / rotary)
    if scaling == "linear":
        f = f / factor
    if scaling != "parts":
        return f, 1.0
    turns = trained * f / (2 * math.pi)
    keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
    return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def tree_depths(parents: Sequence[int]) -> List[int]:
    """Depth of each row below its sequence's row 0 (parents: -1, then rows before the own)."""
    d: List[int] = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def tree_masks(parents: Sequence[int]) -> List[int]:
    """What each row of one sequence sees of the step's rows, itself and its ancestors, as signed
    64-bit masks (bit j: row j) for PagedCache.attend. At most 64 rows."""
    if len(parents) > 64:
        _refuse(_ROWS, f"{len(parents)} rows: a mask covers 64")
    m: List[int] = []
    for i, p in enumerate(parents):
        if not (p < i and (p >= 0 or i == 0)):
            _refuse(_INVALID, f"parent {p} of row {i}")
        m.append((1 << i) | (m[p] if p >= 0 else 0))
    return [v - (1 << 64) if v >> 63 else v for v in m]


class PagedCache(_Caller):
    """A paged key/value cache over tensors that the caller owns (kept alive by this object).

    k, v [pages][page][kv_heads][dim] bf16 or f16; table [seqs][width] i32, the pages of each
    sequence in order; length [seqs] i32, its cached tokens. Pages, table and lengths may change
    between calls; a call reads what they hold when it runs."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, length: torch.Tensor):
        super().__init__(k.device)
        for name, t in (("cache v", v), ("cache table", table), ("cache len", length)):
            if t.device != k.device:
                _refuse(_DEVICE, f"{name}: on {t.device}, k is on {k.device}")
        self.k, self.v, self.table, self.length = k, v, table, length
        self._c = B.moe_paged_cache(_tensor(k), _tensor(v), _tensor(table), _tensor(length), self._flags_ptr)
        self._ref = ctypes.addressof(self._c)
        B._check(_LIB.moe_paged_cache_check(self._ref))
        self.dtype = k.dtype
        self.seqs, self.kv_heads, self.dim = table.shape[0], k.shape[2], k.shape[3]

    def _heads(self, name: str, t: torch.Tensor) -> Tuple[int, int]:
        if t.dim() != 2:
            _refuse(_LAYOUT_ERR, f"{name}: rank {t.dim()}, expected 2 ([rows][heads * {self.dim}])")
        rows, width = t.shape
        if width % self.dim or not width:
            _refuse(_SHAPE, f"{name}: {width} wide, not heads of {self.dim}")
        return rows, width // self.dim

    def append(self, rope: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor,
               positions: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Rotate the queries q [rows][heads * dim] into `out` (new if None; may be q) and the keys
        k [rows][kv_heads * dim] into the cache, and copy the values v there: row i of sequence b
        becomes cached token length[b] + i. positions [rows] i32 (None: length[b] + i). The cache's
        length does not change; keep() or the caller moves it. q, k and v may be column slices
        of one projection's output."""
        rows, heads = self._heads("q", q)
        qp, qs = self._matrix("q", q, self.dtype, rows, heads * self.dim)
        kw = self.kv_heads * self.dim
        kp, ks = self._matrix("k", k, self.dtype, rows, kw)
        vp, vs = self._matrix("v", v, self.dtype, rows, kw)
        sp = self._vector("row_start", row_start, torch.int32, self.seqs + 1)
        pp = None if positions is None else self._vector("positions", positions, torch.int32, rows)
        if rope.freqs.get_device() != self.index:
            _refuse(_DEVICE, f"rope: on {rope.freqs.device}, the cache is on {self.device}")
        if out is None:
            out = torch.empty((rows, heads * self.dim), dtype=self.dtype, device=self.device)
        op, os_ = self._matrix("out", out, self.dtype, rows, heads * self.dim)
        self._launch(_LIB.moe_rope_append, self._ref, rope._ref, rows, qp, qs, heads, kp, ks, vp, vs, sp, pp, op, os_)
        return out

    def attend(self, q: torch.Tensor, row_start: torch.Tensor, mask: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of the step's rows, after append(): row i of sequence b over the cached tokens
        and, of the step's rows, those with their bit set in mask [rows] i64 (None: rows 0 to i).
        q, out [rows][heads * dim]; scale: on the scores (None: dim ** -0.5). A row that sees
        nothing gives zeros."""
        rows, heads = self._heads("q", q)
        qp, qs = self._matrix("q", q, self.dtype, rows, heads * self.dim)
        sp = self._vector("row_start", row_start, torch.int32, self.seqs + 1)
        mp = None if mask is None else self._vector("mask", mask, torch.int64, rows)
        if out is None:
            out = torch.empty((rows, heads * self.dim), dtype=self.dtype, device=self.device)
        op, os_ = self._matrix("out", out, self.dtype, rows, heads * self.dim)
        need = _LIB.moe_tree_attend_workspace(self._ref, rows, heads)
        if need < 0:
            B._check(-need)
        # from the stream's own pool each time, so that calls on several streams do not share it
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        self._launch(_LIB.moe_tree_attend, self._ref, rows, qp, qs, heads, sp, mp,
                     self.dim ** -0.5 if scale is None else scale, op, os_, ws.data_ptr() if need else None, need)
        return out

    def keep(self, row_start: torch.Tensor, n_keep: torch.Tensor, path: torch.Tensor,
             new_len: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Move the accepted path together (n_keep [seqs], path [rows] as verify() gives them): cached
        token length[b] + i becomes row path[i]'s. new_len [seqs] gets length + n_keep (None: the
        cache's own length does; where other layers' caches have the same length tensor, they would then
        find it advanced: keep_paths() serves them all)."""
        sp = self._vector("row_start", row_start, torch.int32, self.seqs + 1)
        np_ = self._vector("n_keep", n_keep, torch.int32, self.seqs)
        if path.dim() != 1:
            _refuse(_LAYOUT_ERR, f"path: rank {path.dim()}, expected 1")
        rows = path.shape[0]
        pp = self._vector("path", path, torch.int32, rows)
        if new_len is None:
            new_len = self.length
        lp = self._vector("new_len", new_len, torch.int32, self.seqs)
        self._launch(_LIB.moe_path_keep, self._ref, sp, rows, np_, pp, lp)
        return new_len


def keep_paths(caches: Sequence[PagedCache], row_start: torch.Tensor, n_keep: torch.Tensor, path: torch.Tensor) -> None:
    """PagedCache.keep() of every layer's cache. A length tensor that several of them have is advanced once, by the
    last, so that each finds the lengths of before the step."""
    last = {c.length.data_ptr(): i for i, c in enumerate(caches)}
    aside = None
    for i, c in enumerate(caches):
        new_len = None
        if last[c.length.data_ptr()] != i:
            if aside is None or aside.shape != c.length.shape or aside.device != c.device:
                aside = torch.empty_like(c.length)
            new_len = aside
        c.keep(row_start, n_keep, path, new_len=new_len)


class Verifier(_Caller):
    """Tests drafted tokens against the target's probabilities, for steps of up to max_rows rows and
    max_seqs sequences over one vocabulary."""

    def __init__(self, vocab: int, max_rows: int, max_seqs: int, device="cuda"):
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        super().__init__(device)
        need = _LIB.moe_draft_verify_workspace(max_rows, max_seqs, vocab)
        if need < 0:
            B._check(-need)
        self.vocab, self.max_rows, self.max_seqs = vocab, max_rows, max_seqs

    def verify(self, logits: torch.Tensor, tokens: torch.Tensor, row_start: torch.Tensor, u_test: Optional[torch.Tensor],
               u_pick: torch.Tensor, parent: Optional[torch.Tensor] = None, draft_probs: Optional[torch.Tensor] = None,
               temperature: Optional[torch.Tensor] = None):
        """Walk each sequence's drafted tree from row 0 (rules in include/moe_drafted.h).

        logits [rows][vocab] f32, bf16 or f16; tokens [rows] i32, the token of each row; u_test, u_pick
        [rows] f32 in [0, 1); parent [rows] i32 within the sequence (None: a chain); draft_probs
        [rows][vocab] f32, what the drafts after each row were drawn from, independently of each other (None:
        drafts chosen in any other way); temperature [seqs] f32 (None: 1; 0 or less: the largest logit).
        Returns n_keep [seqs], path [rows], tokens [rows] i32 and logprobs [rows] f32: from
        row_start[b] on, the n_keep[b] rows of the path, the tokens after each, and their log
        probabilities; -1, -1 and 0 in the places after them."""
        if logits.dim() != 2:
            _refuse(_LAYOUT_ERR, f"logits: rank {logits.dim()}, expected 2")
        rows, seqs = logits.shape[0], row_start.shape[0] - 1 if row_start.dim() == 1 else 0
        if rows > self.max_rows or not 1 <= seqs <= self.max_seqs:
            _refuse(_ROWS, f"{rows} rows of {seqs} sequences: at most {self.max_rows} of {self.max_seqs}")
        if logits.dtype not in (torch.float32, torch.bfloat16, torch.float16):
            _refuse(_DTYPE, f"logits: {logits.dtype} (float32, bfloat16 or float16)")
        zp, zs = self._matrix("logits", logits, logits.dtype, rows, self.vocab)
        z = B.make_tensor(zp, _DT[logits.dtype], (rows, self.vocab), (zs, 1))
        tp = self._vector("tokens", tokens, torch.int32, rows)
        sp = self._vector("row_start", row_start, torch.int32, seqs + 1)
        up = self._vector("u_pick", u_pick, torch.float32, rows)
        ut = None if u_test is None else self._vector("u_test", u_test, torch.float32, rows)
        pp = None if parent is None else self._vector("parent", parent, torch.int32, rows)
        qp, qs = (None, 0) if draft_probs is None else self._matrix("draft_probs", draft_probs, torch.float32, rows,
                                                                    self.vocab)
        Tp = None if temperature is None else self._vector("temperature", temperature, torch.float32, seqs)
        need = _LIB.moe_draft_verify_workspace(rows, seqs, self.vocab)
        if need < 0:
            B._check(-need)
        n_keep = torch.empty(seqs, dtype=torch.int32, device=self.device)
        path = torch.empty(rows, dtype=torch.int32, device=self.device)
        said = torch.empty(rows, dtype=torch.int32, device=self.device)
        logprobs = torch.empty(rows, dtype=torch.float32, device=self.device)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        self._launch(_LIB.moe_draft_verify, ctypes.byref(z), tp, sp, seqs, pp, ut, up, qp, qs, Tp, n_keep.data_ptr(),
                     path.data_ptr(), said.data_ptr(), logprobs.data_ptr(), self._flags_ptr,
                     ws.data_ptr() if need else None, need)
        return n_keep, path, said, logprobs
