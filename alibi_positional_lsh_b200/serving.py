"""Serving with Positional-LSH attention: packed prompts, a paged cache and attention against it.

PlshServing keeps what all sequences share, the table's windows and masks for positions
0 .. max_len - 1, and runs T~ (causal) over
  attend_packed   whole prompts of different lengths, packed without padding  (plsh_packed_fwd)
  attend_paged    new tokens of every sequence against a paged cache          (plsh_paged_fwd)
PagedCache holds the pages and moves rows in and out of them
  append          new tokens' K and V, quantised to e4m3 or copied            (plsh_cache_append)
  read            a range of every sequence as packed tensors                 (plsh_cache_read)
Every call is asynchronous on `stream` (default: the current stream of the tensors' device), makes no
host copies and can be captured into a CUDA graph. Data errors (a malformed sequence, a page
outside the pool) are reported by check().
"""
from __future__ import annotations

from struct import Struct
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import (PLSH_BF16, PLSH_F32, PLSH_MAX_S, PLSH_TILE, PlshError, _check, _lib, decode_device_error,
               plsh_draw_table_heads, plsh_near_counts, plsh_window_from_table)

_CODES = {torch.bfloat16: PLSH_BF16, torch.float32: PLSH_F32}


# the calls' arguments as arrays: ctypes takes longer to pass them one by one than the library to check and launch
_PACKED, _APPEND, _READ, _PAGED = (Struct(f"={len(f.argtypes)}q") for f in (_lib.plsh_packed_fwd, _lib.plsh_cache_append, _lib.plsh_cache_read,
                                                                          _lib.plsh_paged_fwd))
_EMPTY = (0, 0, 0)
_FEW = 8  # plsh_paged_fwd may need scratch for more new tokens than this


def _stream(stream: Optional[torch.cuda.Stream], device: torch.device) -> int:
    # the handle without the Stream object around it, which takes longer to make than the rest of a call's checks
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _rows(t: torch.Tensor, name: str, T: Optional[int], heads: int, d: int, dtype: torch.dtype, device: torch.device) -> Tuple[int, int, int]:
    """(pointer, token stride, head stride) of t, which must be [T][heads][d] of dtype on `device`, with rows that the kernels can
    load 16 bytes at a time. T None: any."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or (T is not None and shape[0] != T):
        raise ValueError(f"{name} must have shape {('T' if T is None else T, heads, d)}, got {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    n = shape[0]
    if n == 0:
        return _EMPTY
    p = t.data_ptr()
    if t.is_contiguous():
        if p % 16 == 0:
            return p, heads * d, d
    else:
        # the stride of a dimension of one element says nothing: torch leaves any number there
        token, head, one = t.stride()
        if heads == 1:
            head = d
        if n == 1:
            token = heads * head
        step = 16 // t.element_size()
        if one == 1 and p % 16 == 0 and token % step == 0 and head % step == 0 and token >= d and head >= d:
            return p, token, head
    raise ValueError(f"{name} must have contiguous, 16-byte aligned rows that do not overlap")


def _ints(t: torch.Tensor, name: str, dims: int, device: torch.device) -> int:
    if t.dtype is not torch.int32 or t.dim() != dims or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dims} dimension(s) on {device}")
    return t.data_ptr()


def _sequences(cu_seqlens: torch.Tensor, device: torch.device) -> Tuple[int, int]:
    p = _ints(cu_seqlens, "cu_seqlens", 1, device)
    S = cu_seqlens.shape[0] - 1
    if S < 0:
        raise ValueError("cu_seqlens must hold one entry more than there are sequences")
    return p, S


def _cached(start: torch.Tensor, page_table: torch.Tensor, S: int, device: torch.device) -> Tuple[int, int, int]:
    """Pointers of start and the page table, and the table's width."""
    ps, pt = _ints(start, "start", 1, device), _ints(page_table, "page_table", 2, device)
    if start.shape[0] != S:
        raise ValueError(f"start must hold one entry per sequence ({S})")
    if page_table.shape[0] != S or page_table.shape[1] < 1:
        raise ValueError(f"page_table must be [{S}][pages] with at least one page per sequence")
    return ps, pt, page_table.shape[1]


class _On:
    """The current device for the launches of a call: `device`, without work where it is current already (the usual case, which
    torch.cuda.device's own steps would make up a good part of a decoding step's host time)."""

    __slots__ = ("index", "back")

    def __init__(self, index: int):
        self.index, self.back = index, -1

    def __enter__(self) -> None:
        now = torch._C._cuda_getDevice()
        if now != self.index:
            self.back = now
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc) -> None:
        if self.back >= 0:
            torch.cuda.set_device(self.back)


def _empty(like: torch.Tensor, stream: Optional[torch.cuda.Stream], *shape: int) -> torch.Tensor:
    """A new tensor of like's type and device for work on `stream` (None: the current one)."""
    if stream is None:
        return like.new_empty(*shape)
    with torch.cuda.stream(stream):
        return like.new_empty(*shape)


class _Kept:
    """An object whose calls pass addresses and sizes that were looked up once: its attributes cannot be exchanged (memory that a
    call still reads would be freed), and a copy looks its own up. Also the device error word of the calls."""

    err: torch.Tensor

    def _keep(self) -> dict:
        """What the calls need of the object's tensors, by attribute."""
        raise NotImplementedError

    def _fix(self) -> None:
        self.__dict__.update(self._keep())
        self.__dict__.setdefault("_fixed", frozenset(self.__dict__) | {"_fixed"})  # not what a caller adds later

    def __setattr__(self, name: str, value) -> None:
        if name in self.__dict__.get("_fixed", ()):
            raise AttributeError(f"{name} cannot be exchanged: the calls go on with what the object was made of")
        super().__setattr__(name, value)

    def __delattr__(self, name: str) -> None:
        if name in self.__dict__.get("_fixed", ()):
            raise AttributeError(f"{name} cannot be taken out: the calls go on with what the object was made of")
        super().__delattr__(name)

    def __setstate__(self, state: dict) -> None:  # copies and pickles: other tensors, other addresses
        self.__dict__.update(state)
        self._fix()

    def reset_errors(self) -> None:
        self.err.zero_()

    def device_errors(self) -> list:
        """Synchronises and decodes the device error word."""
        torch.cuda.synchronize(self.err.device)
        return decode_device_error(int(self.err[0].item()) & 0xFFFFFFFF)

    def check(self) -> None:
        errs = self.device_errors()
        if errs:
            raise PlshError(-1, "device reported " + ",".join(errs))


class PagedCache(_Kept):
    """K and V of many sequences in pages [num_pages][H_kv][page_size][d].

    dtype torch.float8_e4m3fn: each row is held as e4m3 values times a power of two, whose exponent is in
    k_exp, v_exp (int8 [num_pages][H_kv][page_size]); torch.bfloat16 or torch.float32: rows as they are.
    Which page holds which positions is the caller's: every call takes a page table int32 [S][pages].
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_exp: Optional[torch.Tensor] = None,
                 v_exp: Optional[torch.Tensor] = None):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages must be alike: [num_pages][H_kv][page_size][d]")
        self.num_pages, self.H_kv, self.page_size, self.d = k_pages.shape
        self.dtype, self.device = k_pages.dtype, k_pages.device
        if self.dtype not in (torch.float8_e4m3fn, torch.bfloat16, torch.float32):
            raise ValueError("pages must be float8_e4m3fn, bfloat16 or float32")
        if self.page_size not in (16, 32, 64, 128, 256) or self.d not in (64, 128) or self.num_pages < 1 or self.H_kv < 1:
            raise ValueError("need pages of 16, 32, 64, 128 or 256 rows of 64 or 128 elements")
        self.quantised = self.dtype == torch.float8_e4m3fn
        if (k_exp is not None) != self.quantised or (v_exp is not None) != self.quantised:
            raise ValueError("e4m3 pages need k_exp and v_exp, other pages take none")
        for t, nm in ((k_pages, "k_pages"), (v_pages, "v_pages"), (k_exp, "k_exp"), (v_exp, "v_exp")):
            if t is None:
                continue
            if not t.is_cuda or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{nm} must be a contiguous CUDA tensor on {self.device}")
            if nm.endswith("exp") and (t.dtype != torch.int8 or t.shape != k_pages.shape[:3]):
                raise ValueError(f"{nm} must be int8 [num_pages][H_kv][page_size]")
        self._tensors = k_pages, v_pages, k_exp, v_exp
        self.err = torch.zeros((4,), dtype=torch.int32, device=self.device)
        self._like = {t: torch.empty((0,), dtype=t, device=self.device) for t in _CODES}  # what new tensors are made from
        self._fix()

    def _keep(self) -> dict:
        return {"_pages": tuple(0 if x is None else x.data_ptr() for x in self._tensors)}

    # the cache's own tensors
    k_pages = property(lambda self: self._tensors[0])
    v_pages = property(lambda self: self._tensors[1])
    k_exp = property(lambda self: self._tensors[2])
    v_exp = property(lambda self: self._tensors[3])

    @classmethod
    def empty(cls, num_pages: int, H_kv: int, page_size: int, d: int, dtype: torch.dtype = torch.float8_e4m3fn,
              device: str = "cuda") -> "PagedCache":
        """A cache with nothing in it (the pages' contents are not set)."""
        shape = (num_pages, H_kv, page_size, d)
        exps = [torch.empty(shape[:3], dtype=torch.int8, device=device) for _ in range(2)] if dtype == torch.float8_e4m3fn else [None] * 2
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device), *exps)

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, cu_seqlens: torch.Tensor,
               start: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Writes rows [cu[s], cu[s + 1]) of k, v [T][H_kv][d] to positions start[s] .. of sequence s."""
        dtype = k.dtype
        if dtype not in _CODES or (not self.quantised and dtype is not self.dtype):
            raise ValueError(f"k of {dtype} cannot go into {self.dtype} pages")
        T, dev = k.shape[0], self.device
        kr = _rows(k, "k", None, self.H_kv, self.d, dtype, dev)
        vr = _rows(v, "v", T, self.H_kv, self.d, dtype, dev)
        cu, S = _sequences(cu_seqlens, dev)
        st, pt, width = _cached(start, page_table, S, dev)
        if S == 0 or T == 0:
            return
        with _On(dev.index):
            _check(_lib.plsh_cache_append_args(_APPEND.pack(*kr, *vr, _CODES[dtype], T, S, cu, st, self.H_kv, self.d, *self._pages, pt, width,
                                                            self.num_pages, self.page_size, self.err.data_ptr(), _stream(stream, dev)), _APPEND.size))

    def read(self, page_table: torch.Tensor, cu_seqlens: torch.Tensor, start: torch.Tensor, total: int,
             dtype: Optional[torch.dtype] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
             stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Positions start[s] .. of every sequence as packed K, V [total][H_kv][d], sequence s in rows [cu[s], cu[s + 1]).

        total is the rows of the result, at least cu[S] (cu_seqlens stays on the device); rows of no sequence are left as
        they are. dtype: bfloat16 (default) or float32 for e4m3 pages, the pages' own else. out: tensors to fill."""
        dtype = dtype if dtype is not None else (out[0].dtype if out is not None else torch.bfloat16 if self.quantised else self.dtype)
        if dtype not in (tuple(_CODES) if self.quantised else (self.dtype,)):
            raise ValueError(f"cannot read {self.dtype} pages as {dtype}")
        dev = self.device
        cu, S = _sequences(cu_seqlens, dev)
        st, pt, width = _cached(start, page_table, S, dev)
        if total < 0:
            raise ValueError("total must be >= 0")
        with _On(dev.index):
            if out is None:
                like = self._like[dtype]
                K, V = _empty(like, stream, total, self.H_kv, self.d), _empty(like, stream, total, self.H_kv, self.d)
            else:
                K, V = out
                for x, nm in ((K, "K"), (V, "V")):
                    _rows(x, nm, total, self.H_kv, self.d, dtype, dev)
                    if not x.is_contiguous():
                        raise ValueError(f"{nm} must be contiguous")
            if S and total:
                _check(_lib.plsh_cache_read_args(_READ.pack(*self._pages, pt, width, self.num_pages, self.page_size, total, S, cu, st, self.H_kv,
                                            self.d, _CODES[dtype], K.data_ptr(), V.data_ptr(), self.err.data_ptr(), _stream(stream, dev)), _READ.size))
        return K, V


class PlshServing(_Kept):
    """T~ (causal) for sequences of up to max_len positions, all with one table."""

    def __init__(self, H: int, H_kv: int, max_len: int, d: int, s: int, sigma: Sequence[float], seed: int = 0,
                 dtype: torch.dtype = torch.bfloat16, device: str = "cuda", head_offset: int = 0,
                 table: Optional[np.ndarray] = None):
        """sigma, seed, head_offset, table: as PlshForward's (table: float64 [H][s][2] instead of a drawn one)."""
        if dtype not in _CODES:
            raise ValueError("dtype must be torch.bfloat16 or torch.float32")
        if H < 1 or H_kv < 1 or H % H_kv or max_len < 1 or d not in (64, 128) or not 1 <= s <= PLSH_MAX_S:
            raise ValueError(f"need H_kv dividing H, max_len >= 1, d 64 or 128 and 1 <= s <= {PLSH_MAX_S}")
        self.H, self.H_kv, self.max_len, self.d, self.s = H, H_kv, max_len, d, s
        self.dtype, self.device = dtype, torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("device must be a CUDA device")
        torch.cuda.init()
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.sigma_host = np.ascontiguousarray(sigma, dtype=np.float64)
        if self.sigma_host.shape != (H,):
            raise ValueError("sigma must hold one value per query head")
        self.table_host = np.empty((H, s, 2), dtype=np.float64)
        if table is None:
            plsh_draw_table_heads(int(seed), int(head_offset), H, s, self.sigma_host, self.table_host)
        else:
            t = np.ascontiguousarray(table, dtype=np.float64)
            if t.shape != (H, s, 2):
                raise ValueError("table must be float64 [H][s][2]")
            self.table_host[...] = t
        with torch.cuda.device(self.device):
            self.err = torch.zeros((4,), dtype=torch.int32, device=self.device)
            self.table_dev = torch.from_numpy(self.table_host).to(self.device)
            self.bmax = torch.empty((H,), dtype=torch.int32, device=self.device)
            self.spans = torch.empty((H, -(-max_len // PLSH_TILE), 2), dtype=torch.int32, device=self.device)
            self.bmask = torch.empty((H, max_len), dtype=torch.int32 if s <= 32 else torch.int64, device=self.device)
            plsh_window_from_table(self.table_dev, H, s, max_len, 1, self.bmax, self.spans, self.bmask, self.err)
            self.near = torch.empty((H, max_len, 64), dtype=torch.uint8, device=self.device)  # each position's counts in its own key tile
            plsh_near_counts(self.bmask, H, s, max_len, self.near)
            self.check()  # waits for the plan, so that any stream may use it from here on
            self.windows_host = self.bmax.cpu().numpy()  # the heads' longest blocks
        self.max_window = int(self.windows_host.max())
        self._like = tuple(torch.empty((0,), dtype=t, device=self.device) for t in (dtype, torch.float32, torch.uint8))
        self._code = _CODES[dtype]
        self._fix()

    def _keep(self) -> dict:
        self.windows_host.flags.writeable = False
        return {"_windows": self.windows_host.ctypes.data, "_err": self.err.data_ptr(), "_table": self.table_dev.data_ptr(),
                "_plan": (self.spans.data_ptr(), self.bmask.data_ptr(), self.near.data_ptr())}

    def _outputs(self, T: int, out, stream) -> Tuple[torch.Tensor, torch.Tensor]:
        if out is None:
            return _empty(self._like[0], stream, T, self.H, self.d), _empty(self._like[1], stream, T, self.H)
        O, row_sum = out
        _rows(O, "O", T, self.H, self.d, self.dtype, self.device)
        if row_sum.shape != (T, self.H) or row_sum.dtype != torch.float32 or row_sum.device != self.device \
                or not row_sum.is_contiguous() or not O.is_contiguous():
            raise ValueError(f"out must be contiguous {self.dtype} [T][H][d] and float32 [T][H] on {self.device}")
        return O, row_sum

    def attend_packed(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                      out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """T~ of whole prompts: q [T][H][d], k, v [T][H_kv][d], sequence s in tokens [cu[s], cu[s + 1]).

        Returns new tensors O [T][H][d] and row_sum [T][H] (float32), or fills `out`; tokens of no sequence (behind the
        last) are left as they are. Views with contiguous rows, as a fused QKV projection gives, need no copy."""
        T, dev, dtype = q.shape[0], self.device, self.dtype
        qr = _rows(q, "q", None, self.H, self.d, dtype, dev)
        kr = _rows(k, "k", T, self.H_kv, self.d, dtype, dev)
        vr = _rows(v, "v", T, self.H_kv, self.d, dtype, dev)
        cu, S = _sequences(cu_seqlens, dev)
        with _On(dev.index):
            O, row_sum = self._outputs(T, out, stream)
            if S and T:
                _check(_lib.plsh_packed_fwd_args(_PACKED.pack(*qr, *kr, *vr, self._code, T, S, cu, self.H, self.H_kv, self.d, self.s, self.max_len,
                                            *self._plan, O.data_ptr(), row_sum.data_ptr(), self._err, _stream(stream, dev)), _PACKED.size))
        return O, row_sum

    def attend_paged(self, q: torch.Tensor, cache: PagedCache, page_table: torch.Tensor, cu_seqlens: torch.Tensor,
                     start: torch.Tensor, max_new: Optional[int] = None,
                     out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """T~ of new tokens against the cache: q [T][H][d], token t of sequence s at position start[s] + t - cu[s].

        The cache holds the new tokens' own K and V already (append first); pages that the first new token's window no longer
        reaches may be in another's use. max_new: the most new tokens of a sequence where the caller knows it (1 when
        decoding); it chooses the kernels. Without it any sequence may be a chunk of T tokens, and a decoding step of more
        than 16 pays for the chunks' kernels (16/8 heads, d 128, e4m3 pages: 32 sequences 60 us instead of 19, 128 sequences 91
        instead of 41; 12 sequences 18 instead of 15). Returns as attend_packed."""
        T, dev = q.shape[0], self.device
        qr = _rows(q, "q", None, self.H, self.d, self.dtype, dev)
        if cache.device != dev or cache.H_kv != self.H_kv or cache.d != self.d or \
                (not cache.quantised and cache.dtype != self.dtype):
            raise ValueError("the cache's device, heads, head dim or type do not match the plan")
        cu, S = _sequences(cu_seqlens, dev)
        st, pt, width = _cached(start, page_table, S, dev)
        if max_new is not None and max_new < 1:
            raise ValueError("max_new must be >= 1")
        most = T if max_new is None else min(max_new, T)
        with _On(dev.index):
            O, row_sum = self._outputs(T, out, stream)
            if S and T:
                scratch, need = None, 0
                if most > _FEW and cache.quantised and self.dtype == torch.bfloat16:
                    need = _lib.plsh_paged_scratch_bytes(T, S, most, self.H_kv, self.d, self.max_window)
                    if need:
                        scratch = _empty(self._like[2], stream, need)
                _check(_lib.plsh_paged_fwd_args(_PAGED.pack(*qr, self._code, T, S, cu, st, most, self.H, self.H_kv, self.d, *cache._pages, pt, width,
                                           cache.num_pages, cache.page_size, self.s, self.max_len, self._table, *self._plan, self._windows,
                                           scratch.data_ptr() if need else 0, need, O.data_ptr(), row_sum.data_ptr(), self._err,
                                           _stream(stream, dev)), _PAGED.size))
        return O, row_sum
