"""Python binding of the paged-cache entry points (include/faq.h): rotary positions with the
quantized append, attention over a paged K/V cache, the cached tokens' attention weights, and
eviction by them.

Argument marshalling only.  New tokens' rows are bf16 CUDA tensors [T, H, D] whose heads are dense
(any token stride that is a multiple of 8 elements: slices of a fused projection's output pass as
they are).  Every tensor lies on the current CUDA device; the calls run on its current stream.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Sequence, Tuple

import torch

from . import _native as N
from .api import LAYOUTS, MODES, _check

_CODES = {"int8_per_head": torch.int8, "int8_per_token": torch.int8, "fp8_per_head": torch.uint8,
          "fp8_per_token": torch.uint8}
_PER_HEAD = ("int8_per_head", "fp8_per_head")


# a step of a serving loop makes several of these calls, each a few microseconds of GPU time: the checks
# below are kept to a few attribute reads per tensor
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _here() -> int:
    """The current device's current stream."""
    return _raw_stream(_current_device())


def _on_device(t: torch.Tensor, what: str):
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if d != _current_device():
        raise ValueError(f"{what} is not on the current CUDA device")


def _dense(t: torch.Tensor, dtype, what: str, shape=None) -> int:
    """The address of a contiguous tensor of that type on the current device, checked."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} CUDA tensor")
    _on_device(t, what)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _int32(x, what: str) -> int:
    """x as the C interface takes it: what does not fit would wrap there."""
    x = int(x)
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{what} must fit 32 bits, got {x}")
    return x


def _rows(t: torch.Tensor, what: str) -> N.FaRows:
    if t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{what}: expected a bf16 CUDA tensor [T, H, D]")
    _on_device(t, what)
    T, H, D = t.shape
    st = t.stride()
    if (st[2] != 1 and D > 1) or (st[1] != D and H > 1):
        raise ValueError(f"{what}: heads and elements must be dense")
    return N.FaRows(t.data_ptr(), T, H, D, st[0] if T > 1 else H * D)


@dataclass(frozen=True, eq=False, init=False)
class PagedCache:
    """Pages of quantized K and V (fa_paged_cache): codes [pages, H, page_size, D] (layout "BNSD") or
    [pages, page_size, H, D] ("BSND"), int8 or E4M3 bytes (uint8); scales fp32 [H] in the per-head
    modes, [pages, H, page_size] in the per-token ones.  Its tensors are the ones it was made with: write
    into them, or make another for other tensors."""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor
    mode: str
    layout: str = "BNSD"

    def __init__(self, k_codes, v_codes, k_scales, v_scales, mode, layout="BNSD"):
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be BNSD or BSND, got {layout!r}")
        if mode not in _CODES:
            raise ValueError(f"a paged cache's mode is one of {sorted(_CODES)}, got {mode!r}")
        s = k_codes.shape
        if len(s) != 4:
            raise ValueError("codes: expected 4 dimensions")
        pages, H, page_size, D = s if layout == "BNSD" else (s[0], s[2], s[1], s[3])
        sc = (H,) if mode in _PER_HEAD else (pages, H, page_size)
        dt = _CODES[mode]
        c = N.FaPagedCache(_dense(k_codes, dt, "k_codes"), _dense(v_codes, dt, "v_codes", s),
                           _dense(k_scales, torch.float32, "k_scales", sc), _dense(v_scales, torch.float32, "v_scales", sc),
                           MODES[mode], pages, H, page_size, D, LAYOUTS[layout])
        # (frozen: written past __setattr__, and in one go, since a serving loop may make one per call)
        self.__dict__.update(k_codes=k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales, mode=mode,
                             layout=layout, pages=pages, H=H, page_size=page_size, D=D, _c=c, _device=_current_device())

    def c(self) -> N.FaPagedCache:
        """The descriptor, for a call on the current device."""
        if self._device != _current_device():
            raise ValueError("the cache is not on the current CUDA device")
        return self._c


@dataclass(frozen=True, eq=False, init=False)
class PagedBatch:
    """The sequences of one call (fa_paged_batch): page_table int32 [B, max_pages]; seq_lens int32 [B],
    cached tokens with the new ones; cu_q int32 [B + 1], the new tokens' row offsets (None: one new
    token per sequence); max_q, a bound on a sequence's new tokens (0: all rows).  Its tensors are the ones it
    was made with: write into them (a captured graph then follows), or make another for other tensors."""
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    cu_q: Optional[torch.Tensor] = None
    max_q: int = 0

    def __init__(self, page_table, seq_lens, cu_q=None, max_q=0):
        if page_table.dim() != 2:
            raise ValueError("page_table: expected [B, max_pages]")
        B, wide = page_table.shape
        c = N.FaPagedBatch(_dense(page_table, torch.int32, "page_table"), _dense(seq_lens, torch.int32, "seq_lens", (B,)),
                           None if cu_q is None else _dense(cu_q, torch.int32, "cu_q", (B + 1,)), B, wide,
                           _int32(max_q, "max_q"))
        self.__dict__.update(page_table=page_table, seq_lens=seq_lens, cu_q=cu_q, max_q=max_q, B=B, _c=c,
                             _device=_current_device())

    def c(self) -> N.FaPagedBatch:
        """The descriptor, for a call on the current device."""
        if self._device != _current_device():
            raise ValueError("the batch is not on the current CUDA device")
        return self._c


def empty_paged_cache(pages: int, H: int, page_size: int, D: int, mode: str, layout: str = "BNSD",
                      device="cuda") -> PagedCache:
    """Allocate (with torch) the pages of a cache."""
    if mode not in _CODES:
        raise ValueError(f"a paged cache's mode is one of {sorted(_CODES)}, got {mode!r}")
    shp = (pages, H, page_size, D) if layout == "BNSD" else (pages, page_size, H, D)
    sc = (H,) if mode in _PER_HEAD else (pages, H, page_size)
    codes = [torch.empty(shp, dtype=_CODES[mode], device=device) for _ in range(2)]
    scales = [torch.empty(sc, dtype=torch.float32, device=device) for _ in range(2)]
    return PagedCache(*codes, *scales, mode, layout)


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None) -> Tuple[list, float]:
    """The pairs' rotation frequencies f_i = base^(-2 i / rotary_dim), scaled for long contexts, and
    the factor on cos and sin.  ``scaling`` is None or a dict with "type" and
      "linear": f_i / factor (S. Chen, S. Wong, L. Chen and Y. Tian, "Extending Context Window of Large
                Language Models via Positional Interpolation", 2023);
      "ntk":    the base times factor^(rotary_dim / (rotary_dim - 2)), so the slowest pair slows by
                ``factor`` and the fastest stays;
      "yarn":   f_i / factor for pairs that turn less than ``beta_slow`` (1) times in ``original``
                positions, f_i for those that turn more than ``beta_fast`` (32) times, between them a
                linear blend over the pair index; cos and sin times 0.1 ln(factor) + 1 (or
                ``attention_factor``) (B. Peng, J. Quesnelle, H. Fan and E. Shippole, "YaRN: Efficient
                Context Window Extension of Large Language Models", 2023);
      "bands":  f_i / factor for wavelengths over original / ``low`` (1), f_i below original / ``high``
                (4), between them a blend linear in original / wavelength.
    Host arithmetic in 64 bits."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    half = rotary_dim // 2
    kind = None if scaling is None else scaling["type"]
    if kind not in (None, "linear", "ntk", "yarn", "bands"):
        raise ValueError(f"unknown rotary scaling {kind!r}")
    factor = 1.0 if scaling is None else float(scaling["factor"])
    if not factor > 0.0 or not base > 0.0:
        raise ValueError("base and factor must be positive")
    if kind == "ntk":
        if rotary_dim <= 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    if kind in (None, "ntk"):
        return f, 1.0
    if kind == "linear":
        return [x / factor for x in f], 1.0
    original = float(scaling["original"])
    if kind == "yarn":
        if not base > 1.0:
            raise ValueError("yarn scaling needs base > 1")
        # the (real) pair index that turns n times in `original` positions
        at = lambda n: rotary_dim * math.log(original / (2.0 * math.pi * n)) / (2.0 * math.log(base))
        lo = max(0.0, math.floor(at(float(scaling.get("beta_fast", 32.0)))))
        hi = min(rotary_dim - 1.0, math.ceil(at(float(scaling.get("beta_slow", 1.0)))))
        width = max(hi - lo, 1e-3)
        w = [min(1.0, max(0.0, (i - lo) / width)) for i in range(half)]
        mult = float(scaling.get("attention_factor", 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0))
        return [x / factor * a + x * (1.0 - a) for x, a in zip(f, w)], mult
    low, high = float(scaling.get("low", 1.0)), float(scaling.get("high", 4.0))
    if not high > low:
        raise ValueError("bands scaling needs high > low")
    turns = [original * x / (2.0 * math.pi) for x in f]
    keep = [min(1.0, max(0.0, (n - low) / (high - low))) for n in turns]
    return [x * a + x / factor * (1.0 - a) for x, a in zip(f, keep)], 1.0


def rope_table(positions: int, rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None,
               device="cuda") -> torch.Tensor:
    """cos | sin of the rotation angles, fp32 [positions, rotary_dim] (fa_rope_table), with
    rope_frequencies' frequencies.  Made once, kept like a weight."""
    f, mult = rope_frequencies(rotary_dim, base, scaling)
    out = torch.empty((positions, rotary_dim), dtype=torch.float32, device=device)
    arr = (ctypes.c_double * len(f))(*f)
    _check(N.lib().fa_rope_table(_dense(out, torch.float32, "table"), positions, rotary_dim, arr, mult, _here()),
           "fa_rope_table")
    return out


def rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, cache: PagedCache, batch: PagedBatch,
                table: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                interleaved: bool = False, amax: Optional[Sequence[torch.Tensor]] = None,
                out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Rotate the new tokens' q and k, quantize k and v into the cache (fa_rope_append).
    ``table``: rope_table's (its width is the rotary dimension; None: no rotation).  ``positions``:
    int32 [T] (None: the tokens' cache indices).  ``amax``: per-head calibration maxima (k, v), for
    the per-head modes.  ``out`` may be q itself.  Returns the rotated q (None without q)."""
    tk, tv = _rows(k, "k"), _rows(v, "v")
    tq = to = None
    if q is not None:
        tq = _rows(q, "q")
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        to = _rows(out, "out")
    elif out is not None:
        raise ValueError("out without q")
    pt, npos, rd = None, 0, 0
    if table is not None:
        if table.dim() != 2:
            raise ValueError("table: expected [positions, rotary_dim]")
        pt = _dense(table, torch.float32, "table")
        npos, rd = table.shape
    am = (None, None)
    if amax is not None:
        am = tuple(_dense(a, torch.float32, "amax", (cache.H,)) for a in amax)
    ref = ctypes.byref
    _check(N.lib().fa_rope_append(ref(tq) if tq is not None else None, ref(tk), ref(tv), ref(cache.c()), ref(batch.c()), pt,
                                  npos, rd,
                                  None if positions is None else _dense(positions, torch.int32, "positions", (tk.T,)),
                                  1 if interleaved else 0, am[0], am[1], ref(to) if to is not None else None, _here()),
           "fa_rope_append")
    return out


def paged_attention_workspace_size(q: torch.Tensor, cache: PagedCache, batch: PagedBatch) -> int:
    tq = _rows(q, "q")
    return int(N.lib().fa_paged_attention_workspace_size(ctypes.byref(tq), ctypes.byref(cache.c()), ctypes.byref(batch.c())))


def paged_attention(q: torch.Tensor, cache: PagedCache, batch: PagedBatch, causal: bool = True,
                    softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
    """Attention of the new tokens q [T, Hq, D] over the cache (fa_paged_attention), bf16 [T, Hq, D].
    q, out, lse and the workspace must not overlap.  Returns out, or (out, lse) with return_lse (lse fp32 [T, Hq]).  ``workspace``: bytes to use where it is
    large enough (paged_attention_workspace_size), else it is allocated."""
    tq = _rows(q, "q")
    ref = ctypes.byref
    if out is None:
        out = torch.empty((tq.T, tq.H, tq.D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((tq.T, tq.H), dtype=torch.float32, device=q.device)
    c, b = ref(cache.c()), ref(batch.c())
    if workspace is not None:
        _on_device(workspace, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous tensor")
    need = N.lib().fa_paged_attention_workspace_size(ref(tq), c, b)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = q.new_empty(need, dtype=torch.uint8)
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    _check(N.lib().fa_paged_attention(ref(tq), c, b, 1 if causal else 0, float(softmax_scale),
                                      _dense(out, torch.bfloat16, "out", (tq.T, tq.H, tq.D)),
                                      None if lse is None else _dense(lse, torch.float32, "lse", (tq.T, tq.H)), ws,
                                      ws_bytes, _here()), "fa_paged_attention")
    return (out, lse) if return_lse else out


def paged_weights(q: torch.Tensor, lse: torch.Tensor, cache: PagedCache, batch: PagedBatch, acc: torch.Tensor,
                  causal: bool = True, softmax_scale: float = 0.0, accumulate: bool = True) -> torch.Tensor:
    """Add to acc (fp32 [B, Hkv, n]) the attention weight the new tokens give each cached token, or
    with accumulate=False set it (fa_paged_weights).  ``lse`` as paged_attention returned it; rows where it
    is not finite give nothing."""
    tq = _rows(q, "q")
    ref = ctypes.byref
    if acc.dim() != 3 or tuple(acc.shape[:2]) != (batch.B, cache.H):
        raise ValueError(f"acc: expected [{batch.B}, {cache.H}, n]")
    _check(N.lib().fa_paged_weights(ref(tq), _dense(lse, torch.float32, "lse", (tq.T, tq.H)), ref(cache.c()), ref(batch.c()),
                                    1 if causal else 0, float(softmax_scale), _dense(acc, torch.float32, "acc"),
                                    acc.shape[2], 1 if accumulate else 0, _here()), "fa_paged_weights")
    return acc


def paged_evict(cache: PagedCache, batch: PagedBatch, scores: torch.Tensor, budget: int, sink: int = 0, recent: int = 0,
                scores_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keep ``budget`` tokens per kv head of every sequence (the first ``sink``, the last ``recent``, the
    highest scores [B, Hkv, n] of the rest) and move their rows to the front (fa_paged_evict).
    Returns the kept cache indices int32 [B, Hkv, budget] (-1 past the kept ones) and the new lengths
    int32 [B]; scores_out receives the kept tokens' scores, then zeros."""
    if scores.dim() != 3 or tuple(scores.shape[:2]) != (batch.B, cache.H):
        raise ValueError(f"scores: expected [{batch.B}, {cache.H}, n]")
    budget, sink, recent = _int32(budget, "budget"), _int32(sink, "sink"), _int32(recent, "recent")
    if not 1 <= budget <= 2**30:
        raise ValueError("budget must be at least 1 and at most 2^30")
    ps = _dense(scores, torch.float32, "scores")
    po = None if scores_out is None else _dense(scores_out, torch.float32, "scores_out", scores.shape)
    kept = scores.new_empty((batch.B, cache.H, budget), dtype=torch.int32)
    new = scores.new_empty((batch.B,), dtype=torch.int32)
    _check(N.lib().fa_paged_evict(ctypes.byref(cache.c()), ctypes.byref(batch.c()), ps, scores.shape[2], budget, sink,
                                  recent, kept.data_ptr(), new.data_ptr(), po, _here()),
           "fa_paged_evict")
    return kept, new
