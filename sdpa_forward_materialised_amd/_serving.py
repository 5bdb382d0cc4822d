"""Binding of the serving operators (``include/sdpa_serve.h``): attention over
packed prompts without the probability map, the attention weight each key
received, and the paged 8-bit cache.

Argument marshalling only, like the rest of the binding: workspaces and default
outputs come from torch's caching allocator, the launch goes to torch's current
stream on the tensors' device, and nothing here synchronises or reads device
data. A tensor that was produced on another stream has to be ordered before the
call by the caller, as for any torch operator. There are no gradients:
``sdpa_math`` and ``bwd`` are for training.
"""

from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

import torch

from ._binding import _DTYPES, _PACK, _causal_code, _current_stream, _raise, load_library

_BYTES = {}  # workspace bytes per call signature (shapes and flags)
_PACK2, _PACK3, _PACK4 = (_PACK[n].pack for n in (2, 3, 4))

# These calls often take a few microseconds on the GPU, so the host path is
# kept short: tensors are described in one go, without the dense binding's
# right-alignment, and devices compared as indices.


def _dtype(t: torch.Tensor) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return dt


def _refuse_desc(name: str, t: torch.Tensor, n: int):
    _dtype(t)
    raise ValueError(f"{name} must have {n} dims, got {t.dim()}") from None


def _desc2(name: str, t: torch.Tensor) -> bytes:
    try:
        return _PACK2(t.data_ptr(), _DTYPES[t.dtype], 2, *t.shape, *t.stride())
    except (KeyError, struct.error):  # the item count is that of the dims
        _refuse_desc(name, t, 2)


def _desc3(name: str, t: torch.Tensor) -> bytes:
    try:
        return _PACK3(t.data_ptr(), _DTYPES[t.dtype], 3, *t.shape, *t.stride())
    except (KeyError, struct.error):
        _refuse_desc(name, t, 3)


def _device(t: torch.Tensor, *others: torch.Tensor) -> int:
    """Index of the GPU that all of the tensors are on."""
    i = t.get_device()
    if i < 0:
        raise ValueError("sdpa_math runs on the GPU only: every tensor must be a cuda tensor")
    for o in others:
        if o.get_device() != i:
            if not o.is_cuda:
                raise ValueError("sdpa_math runs on the GPU only: every tensor must be a cuda tensor")
            raise ValueError(f"tensors on different devices ({t.device} and {o.device})")
    return i


class PagedCache:
    """A pool of pages of an 8-bit key/value cache.

    ``k`` [n_pages, Hkv, page, D] and ``v`` [n_pages, Hkv, D, page] (the tokens
    of a page innermost) hold float8_e4m3fn codes; ``k_scale`` and ``v_scale``
    [n_pages, Hkv] (float32) the power of two that a page's and head's codes are
    multiplied with. The object holds these tensors for good (another pool is
    another object), and they must keep their storage.
    """

    __slots__ = ("_tensors", "_bytes")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        for name, t, nd in (("k", k, 4), ("v", v, 4), ("k_scale", k_scale, 2), ("v_scale", v_scale, 2)):
            if t.dim() != nd:
                raise ValueError(f"cache {name} must have {nd} dims, got {t.dim()}")
            if t.device != k.device:
                raise ValueError(f"cache tensors on different devices ({k.device} and {t.device})")
        self._tensors = (k, v, k_scale, v_scale)
        self._bytes = b"".join((_PACK4(k.data_ptr(), _dtype(k), 4, *k.shape, *k.stride()),
                                _PACK4(v.data_ptr(), _dtype(v), 4, *v.shape, *v.stride()),
                                _desc2("k_scale", k_scale), _desc2("v_scale", v_scale)))

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    @property
    def page_tokens(self) -> int:
        return self.k.shape[2]


def new_cache(n_pages: int, heads: int, head_dim: int, page_tokens: int = 64, device="cuda") -> PagedCache:
    """A pool of zeroed pages."""
    return PagedCache(torch.zeros((n_pages, heads, page_tokens, head_dim), dtype=torch.float8_e4m3fn, device=device),
                      torch.zeros((n_pages, heads, head_dim, page_tokens), dtype=torch.float8_e4m3fn, device=device),
                      torch.zeros((n_pages, heads), dtype=torch.float32, device=device),
                      torch.zeros((n_pages, heads), dtype=torch.float32, device=device))


# torch's current device and stream (its own raw queries when it has them:
# the tensors of a call are on the GPU already, so nothing is left to initialise)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda i: _current_stream(torch.device("cuda", i)))


def _offsets(name: str, t: torch.Tensor, n: Optional[int] = None) -> None:
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} holds {t.numel()} entries, expected {n}")


def _table(name: str, t: torch.Tensor, n_seqs: int) -> None:
    if t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D int32 tensor, contiguous in its last dim")
    if t.shape[0] != n_seqs:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {n_seqs}")


def _cu_pair(cu_q: torch.Tensor, cu_kv: torch.Tensor) -> int:
    _offsets("cu_seqlens_q", cu_q)
    n = cu_q.numel()
    if cu_kv is not cu_q:
        _offsets("cu_seqlens_kv", cu_kv)
        if cu_kv.numel() != n:
            n = 0
    if n < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_kv must hold n_seqs + 1 offsets each")
    return n - 1


def _scale(scale: Optional[float], D: int) -> float:
    if scale is not None:
        return float(scale)
    return 1.0 / math.sqrt(D) if D > 0 else 1.0


def _call(lib, fn, dev: int, *args) -> None:
    """``fn(*args, stream)`` on the tensors' device (made current only when it is not)."""
    if dev == _current_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != 0:
        _raise(rc, lib)


def _workspace(lib, fn, like: torch.Tensor, sig, *args):
    """(workspace or None, its bytes) of a call with this signature."""
    n = _BYTES.get(sig)
    if n is None:
        c = ctypes.c_size_t(0)
        rc = fn(*args, ctypes.byref(c))
        if rc != 0:
            _raise(rc, lib)
        if len(_BYTES) >= 4096:  # many distinct shapes: start over rather than grow
            _BYTES.clear()
        n = _BYTES[sig] = c.value
    return (like.new_empty(n, dtype=torch.uint8), n) if n > 0 else (None, 0)


def _outputs(q: torch.Tensor, out) -> Tuple[torch.Tensor, torch.Tensor]:
    if out is None:
        return (torch.empty_like(q) if q.is_contiguous() else q.new_empty(q.shape)), q.new_empty(q.shape[:2], dtype=torch.float32)
    O, L = out
    _device(q, O, L)
    return O, L


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     cu_seqlens_kv: torch.Tensor, max_seqlen_q: int, max_seqlen_kv: int, is_causal: bool = True,
                     scale: Optional[float] = None, enable_gqa: bool = False, causal_alignment: str = "top_left",
                     out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``sdpa_prompt_fwd``: (O [Tq, Hq, D], LSE [Tq, Hq] float32) of packed
    sequences q [Tq, Hq, D], k/v [Tkv, Hkv, D], without the probability map.
    Arguments as ``fwd_varlen``, except that it is causal by default; ``out``
    may pass (O, LSE). Tokens of no sequence are not written."""
    lib = load_library()
    dev = _device(q, k, v, cu_seqlens_q, cu_seqlens_kv)
    n = _cu_pair(cu_seqlens_q, cu_seqlens_kv)
    causal = _causal_code(is_causal, causal_alignment)
    dq, dk, dv = _desc3("q", q), _desc3("k", k), _desc3("v", v)
    O, L = _outputs(q, out)
    _call(lib, lib.sdpa_prompt_fwd, dev, dq, dk, dv, cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(), n,
          int(max_seqlen_q), int(max_seqlen_kv), causal, _scale(scale, q.shape[2]), int(bool(enable_gqa)),
          _desc3("out", O), _desc2("lse", L))
    return O, L


def key_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, cu_seqlens_q: torch.Tensor,
                cu_seqlens_kv: torch.Tensor, max_seqlen_q: int, max_seqlen_kv: int, is_causal: bool = True,
                scale: Optional[float] = None, enable_gqa: bool = False, causal_alignment: str = "top_left",
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``sdpa_key_weights``: the attention weight every key received, summed
    over its sequence's rows and its key head's query heads, float32
    [n_seqs, Hkv, max_seqlen_kv] with zeros past each sequence's keys. ``lse``
    is that of ``prompt_attention`` (or ``fwd_varlen``) on the same arguments;
    ``out`` may pass the result's tensor (last dim contiguous: a slice of the
    weights that ``cache_attention`` adds to, for instance)."""
    lib = load_library()
    dev = _device(q, k, lse, cu_seqlens_q, cu_seqlens_kv)
    n = _cu_pair(cu_seqlens_q, cu_seqlens_kv)
    causal = _causal_code(is_causal, causal_alignment)
    dq, dk = _desc3("q", q), _desc3("k", k)
    max_q, max_kv, gqa = int(max_seqlen_q), int(max_seqlen_kv), int(bool(enable_gqa))
    if out is None:
        out = q.new_empty((n, k.shape[1], max(0, max_kv)), dtype=torch.float32)
    else:
        _device(q, out)
    ws, nbytes = _workspace(lib, lib.sdpa_key_weights_workspace_bytes, q,
                            ("weights", q.shape, k.shape, q.dtype, n, max_q, max_kv), dq, dk, n, max_q, max_kv, 1)
    _call(lib, lib.sdpa_key_weights, dev, dq, dk, _desc2("lse", lse), cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(), n,
          max_q, max_kv, causal, _scale(scale, q.shape[2]), gqa, _desc3("out", out),
          None if ws is None else ws.data_ptr(), nbytes)
    return out


def cache_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                 cu_seqlens: torch.Tensor, max_new: int) -> None:
    """``sdpa_cache_append``: write new tokens k/v [T, Hkv, D] (sequence b's are
    cu_seqlens[b] .. cu_seqlens[b + 1], at most ``max_new``) behind the
    ``kv_lens`` [n_seqs] tokens that the sequences hold. ``page_table``
    [n_seqs, max_pages] lists their pages. ``kv_lens`` is not changed."""
    lib = load_library()
    dev = _device(cache.k, k, v, page_table, kv_lens, cu_seqlens)
    n = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    _offsets("kv_lens", kv_lens)
    _offsets("cu_seqlens", cu_seqlens, n + 1)
    _table("page_table", page_table, n)
    _call(lib, lib.sdpa_cache_append, dev, cache._bytes, _desc3("k", k), _desc3("v", v), page_table.data_ptr(), n,
          page_table.shape[1], page_table.stride(0), kv_lens.data_ptr(), cu_seqlens.data_ptr(), int(max_new))


def cache_attention(q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                    cu_seqlens_q: torch.Tensor, max_seqlen_q: int, max_kv: Optional[int] = None,
                    is_causal: bool = True, scale: Optional[float] = None, enable_gqa: bool = False,
                    weights: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
                    out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``sdpa_cache_attention``: (O [T, Hq, D], LSE [T, Hq] float32) of the last
    tokens of every sequence, q [T, Hq, D] packed by ``cu_seqlens_q``, over its
    ``kv_lens`` cached tokens (these tokens' own keys among them). ``max_kv``
    bounds the lengths (default: the page table's capacity). With ``weights``
    [n_seqs, Hkv, W] (float32), every key's probability, summed over its key
    head's query heads and the new tokens, is added to them, in place or into
    ``weights_out``."""
    lib = load_library()
    dev = _device(q, cache.k, page_table, kv_lens, cu_seqlens_q)
    n = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    _offsets("kv_lens", kv_lens)
    _offsets("cu_seqlens_q", cu_seqlens_q, n + 1)
    _table("page_table", page_table, n)
    dq, gqa = _desc3("q", q), int(bool(enable_gqa))
    dw = dwo = None
    if weights is not None:
        if weights_out is None:
            weights_out = weights
        _device(q, weights, weights_out)
        dw, dwo = _desc3("weights", weights), _desc3("weights_out", weights_out)
    elif weights_out is not None:
        raise ValueError("weights_out needs weights")
    max_pages, max_q, gather = page_table.shape[1], int(max_seqlen_q), int(weights is not None)
    max_kv = max_pages * cache.k.shape[2] if max_kv is None else int(max_kv)
    O, L = _outputs(q, out)
    ws, nbytes = _workspace(lib, lib.sdpa_cache_attention_workspace_bytes, q,
                            ("cache", q.shape, cache.k.shape, n, max_pages, max_q, max_kv, gqa, gather), dq,
                            cache._bytes, n, max_pages, max_q, max_kv, gqa, gather)
    _call(lib, lib.sdpa_cache_attention, dev, dq, cache._bytes, page_table.data_ptr(), n, max_pages,
          page_table.stride(0), kv_lens.data_ptr(), cu_seqlens_q.data_ptr(), max_q, max_kv, int(bool(is_causal)),
          _scale(scale, q.shape[2]), gqa, dw, dwo, _desc3("out", O), _desc2("lse", L),
          None if ws is None else ws.data_ptr(), nbytes)
    return O, L


def cache_evict(cache: PagedCache, page_table: torch.Tensor, kv_lens: torch.Tensor, weights: torch.Tensor, budget: int,
                recent: int, to_table: torch.Tensor, weights_out: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``sdpa_cache_evict``: keep at most ``budget`` tokens of every sequence and
    key head, its ``recent`` last ones and those with the largest ``weights``
    [n_seqs, Hkv, W]; they move, in order, to the pages of ``to_table``
    [n_seqs, to_pages], which must hold no token of a sequence in this call.
    The kept tokens' weights (zeros behind them) replace ``weights`` or go to
    ``weights_out``. Returns (the positions kept, int32 [n_seqs, Hkv, budget]
    with -1 behind them; the new lengths, int32 [n_seqs])."""
    lib = load_library()
    if weights_out is None:
        weights_out = weights
    dev = _device(cache.k, page_table, kv_lens, weights, weights_out, to_table)
    n = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    _offsets("kv_lens", kv_lens)
    _table("page_table", page_table, n)
    _table("to_table", to_table, n)
    budget = int(budget)
    if budget < 1:
        raise ValueError("budget must be at least 1")
    kept = kv_lens.new_empty((n, cache.k.shape[1], budget))
    lens = kv_lens.new_empty((n,))
    _call(lib, lib.sdpa_cache_evict, dev, cache._bytes, page_table.data_ptr(), n, page_table.shape[1],
          page_table.stride(0), kv_lens.data_ptr(), _desc3("weights", weights), _desc3("weights_out", weights_out), budget, int(recent),
          to_table.data_ptr(), to_table.shape[1], to_table.stride(0), kept.data_ptr(), lens.data_ptr())
    return kept, lens
