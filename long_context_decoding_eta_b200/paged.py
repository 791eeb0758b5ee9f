"""Paged KV cache and the decode over it (include/eta.h, "Paged caches").

`PagedKVCache` owns the page pools and their bookkeeping and changes them on the
device: append, fork, free, compact, copy_pages.  `PagedEtaDecoder` is the decoder of
such a cache: the ETA step of `EtaDecoder` (metadata, thresholds, screening, gated
decode over the admitted blocks) with the blocks behind the page table, and
`shared_decode`, which reads a prefix that many rows share once for all of them.

    cache = PagedKVCache(B=64, Hkv=4, d=128, blk=64, max_pages=2048, n_pages=20000)
    cache.append(k, v, cu)                  # a prompt of row 0
    cache.fork([0] * 7, range(1, 8))        # seven more continuations of it
    dec = PagedEtaDecoder(cache, Hq=16, T=None)
    o, lse = dec.shared_decode(q, [0, 8, 64], [prompt_len, 0])

Every change of the bookkeeping is asynchronous on the current stream; nothing is
read back to the host except by `check_status` and the read-only helpers that say so.
Rows, pages, offsets and lengths are whole numbers: int32 device tensors go to the kernels
as they are (a captured call takes no others), lists and host tensors are copied behind
what the stream still runs, at some 10 us of host time each.
Every step runs in libeta.so's kernels; this module only allocates and marshals.
"""
from __future__ import annotations

import math
import operator
from typing import Optional

import torch

from . import _lib as L


_INT32 = torch.iinfo(torch.int32)
_INDEX_TYPES = (torch.int32, torch.int64, torch.int16, torch.int8, torch.uint8)


def _whole(v) -> int:
    if isinstance(v, bool) or (isinstance(v, torch.Tensor) and v.dtype not in _INDEX_TYPES):
        raise ValueError(f"a whole number is wanted, not {v!r}")
    try:
        return operator.index(v)
    except TypeError:
        raise ValueError(f"a whole number is wanted, not {v!r}") from None


def _index_tensor(x, device) -> torch.Tensor:
    """int32 device tensor of a list, range or tensor of whole numbers.  A mask is none.
    Numbers of an int64 tensor that do not fit become the ends of the int32 range, which
    no row, page or length reaches, so that a call reports them and does not wrap them."""
    if isinstance(x, torch.Tensor):
        if x.dtype is torch.int32 and x.device == device and x.is_contiguous():
            return x
        if x.dtype not in _INDEX_TYPES:
            raise ValueError(f"rows, pages and lengths are whole numbers, not {x.dtype}")
        if x.dtype is torch.int64:
            x = x.clamp(_INT32.min, _INT32.max)
        x = x.to(torch.int32).contiguous()
    else:
        x = list(x)
        if not set(map(type, x)) <= {int}:
            x = [_whole(v) for v in x]
        if x and not (_INT32.min <= min(x) and max(x) <= _INT32.max):
            raise ValueError("a number does not fit 32 bits")
        x = torch.tensor(x, dtype=torch.int32)
    if x.device.type != "cpu" or device.type == "cpu":
        return x.to(device)
    if torch.cuda.is_current_stream_capturing():
        raise ValueError("a captured call takes its rows, pages and lengths as device tensors: "
                         "a copy of host numbers cannot be captured")
    # from pinned memory, so that the copy does not wait for what the stream still runs; the
    # pinned block is not used again before the copy is over
    return x.pin_memory().to(device, non_blocking=True)


def _on(device, stream, fn, *args):
    """Calls fn with `device` and, if one is given, `stream` current: what fn makes of its
    arguments (index tensors from lists, say) then belongs to the stream that reads it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return fn(*args)
    if device.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


class PagedKVCache:
    """Pools of `n_pages` pages (blk tokens of every KV head each) and the page table of
    `B` rows of up to `max_pages` pages.  K, V: bf16 [n_pages, Hkv, blk, d], allocated
    here when not given.

    state       int32, the whole bookkeeping; its sections are the views below.  A copy
                of it is a snapshot that can be copied back.
    lengths     int32 [B];  table int32 [B, max_pages] (-1: no page)
    ref         int32 [n_pages], rows that hold the page;  free_list int32 [n_pages]
    n_free      int32 [1], free pages (device)
    """

    def __init__(self, B: int, Hkv: int, d: int, blk: int, max_pages: int, n_pages: int, *,
                 K: Optional[torch.Tensor] = None, V: Optional[torch.Tensor] = None,
                 device="cuda"):
        if (K is None) != (V is None):
            raise ValueError("K and V pools come together")
        shape = (n_pages, Hkv, blk, d)
        if K is None:
            K = torch.zeros(shape, dtype=torch.bfloat16, device=device)
            V = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        for t in (K, V):
            if not t.is_cuda:
                raise ValueError("K/V must be CUDA tensors")
            if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"K/V pools must be contiguous bf16 {shape}")
        if K.device != V.device:
            raise ValueError("K and V pools must be on one device")
        self.K, self.V, self.device = K, V, K.device
        self.B, self.Hkv, self.d, self.blk = B, Hkv, d, blk
        self.max_pages, self.n_pages = max_pages, n_pages
        self.dims = L.Dims.of(B, Hkv, Hkv, d, blk, max_pages * blk)
        words = L.eta_page_state_words(self.dims, n_pages)
        # raises the library's own error for dims that it refuses
        at = L.eta_page_state_offsets(self.dims, n_pages)
        self.state = torch.zeros(words, dtype=torch.int32, device=self.device)
        self.n_free = self.state[at[0]:at[0] + 1]
        self.lengths = self.state[at[1]:at[1] + B]
        self.table = self.state[at[2]:at[2] + B * max_pages].view(B, max_pages)
        self.ref = self.state[at[3]:at[3] + n_pages]
        self.free_list = self.state[at[4]:at[4] + n_pages]
        # holds a bitmap that every call leaves cleared: zeroed once
        self.ws = torch.zeros(L.eta_page_workspace_size(self.dims, n_pages), dtype=torch.uint8,
                              device=self.device)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._cu_one = torch.arange(B + 1, dtype=torch.int32, device=self.device)
        self.init()

    def init(self, stream=None):
        """Empties every row and frees every page."""
        _on(self.device, stream, L.eta_page_init, self.dims, self.n_pages, self.state)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, cu_new=None, stream=None):
        """Writes new tokens behind every row's last one: k_new, v_new bf16
        [n_new, Hkv, d]; row b gets tokens cu_new[b] .. cu_new[b + 1] - 1 (int32
        [B + 1]; None: one token for every row)."""
        n_new = int(k_new.shape[0])
        for t in (k_new, v_new):
            if (t.dtype is not torch.bfloat16 or t.shape != (n_new, self.Hkv, self.d)
                    or not t.is_contiguous() or t.device != self.device):
                raise ValueError(f"k_new/v_new must be contiguous bf16 [n_new, {self.Hkv}, "
                                 f"{self.d}] on {self.device}")
        if cu_new is None:
            if n_new != self.B:
                raise ValueError("without cu_new there is one token for every row")
            cu_new = self._cu_one

        def call():
            cu = _index_tensor(cu_new, self.device)
            if cu.numel() != self.B + 1:
                raise ValueError("cu_new has B + 1 entries")
            L.eta_page_append(self.dims, self.n_pages, self.state, self.K, self.V, k_new, v_new,
                              cu, n_new, self.ws, self.dev_status)
        _on(self.device, stream, call)

    def _pairs(self, src, dst):
        src, dst = _index_tensor(src, self.device), _index_tensor(dst, self.device)
        if src.numel() != dst.numel():
            raise ValueError("src and dst differ in length")
        return src, dst, src.numel()

    def fork(self, src, dst, stream=None):
        """Row dst[i] (empty) becomes a copy of row src[i]: whole pages are shared, the
        partly filled last one is copied."""
        def call():
            s, t, n = self._pairs(src, dst)
            L.eta_page_fork(self.dims, self.n_pages, self.state, self.K, self.V, s, t, n, self.ws,
                            self.dev_status)
        _on(self.device, stream, call)

    def free(self, rows, stream=None):
        """Empties rows; pages that no row holds any more become free."""
        def call():
            r = _index_tensor(rows, self.device)
            L.eta_page_free(self.dims, self.n_pages, self.state, r, r.numel(), self.ws,
                            self.dev_status)
        _on(self.device, stream, call)

    def compact(self, stream=None):
        """Moves the pages in use to the numbers below n_live = n_pages - n_free."""
        _on(self.device, stream, L.eta_page_compact, self.dims, self.n_pages, self.state, self.K,
            self.V, self.ws, self.dev_status)

    def copy_pages(self, src, dst, stream=None):
        """Copies the contents of pages src[i] to pages dst[i]."""
        def call():
            s, t, n = self._pairs(src, dst)
            L.eta_page_copy(self.dims, self.n_pages, self.K, self.V, s, t, n, self.ws,
                            self.dev_status)
        _on(self.device, stream, call)

    def check_status(self):
        """Synchronizes, reads the device status word, raises on any error bit."""
        _raise_status(self.dev_status)


def _raise_status(word_t: torch.Tensor):
    word = int(word_t.item())
    if word:
        code = L.eta_status_from_device(word)
        word_t.zero_()
        raise L.EtaError(f"device status 0x{word:x}", code)


class PagedEtaDecoder:
    """The decode of a paged cache for Hq query heads.  T: temperature of the gate (0 =
    hard), None = no gate.  out_dtype: torch.float32 or torch.bfloat16 outputs.  The
    other arguments as EtaDecoder; the block metadata are allocated when build_meta is
    first called, so that a decoder that never screens holds none."""

    def __init__(self, cache: PagedKVCache, Hq: int, *, bound: str = "exact", z: float = 3.0,
                 T: Optional[float] = 0.0, scale: float = 0.0, prune: str = "skip",
                 cent_format: str = "f32", out_dtype: torch.dtype = torch.float32):
        if cent_format not in ("f32", "bf16"):
            raise ValueError(cent_format)
        if out_dtype not in L.OUT:
            raise ValueError("out_dtype is torch.float32 or torch.bfloat16")
        c = self.cache = cache
        dev = self.device = c.device
        self.dims = L.Dims.of(c.B, Hq, c.Hkv, c.d, c.blk, c.max_pages * c.blk)
        self.B, self.Hq, self.Hkv, self.d, self.blk, self.NB = (c.B, Hq, c.Hkv, c.d, c.blk,
                                                                c.max_pages)
        self.bound, self.z, self.T, self.prune = bound, float(z), T, prune
        self.scale = float(scale) if scale else 1.0 / math.sqrt(c.d)
        self.cent_format = cent_format
        f32, i32 = torch.float32, torch.int32
        ws_decode = L.eta_decode_workspace_size(self.dims)
        if ws_decode == 0:
            raise ValueError(f"unsupported {self.dims}")
        self.ws_decode = torch.empty(ws_decode, dtype=torch.uint8, device=dev)
        self.ws_screen = torch.empty(max(L.eta_screen_workspace_size(self.dims), 256),
                                     dtype=torch.uint8, device=dev)
        self.ws_shared = None
        self.tau = torch.zeros(self.B, Hq, dtype=f32, device=dev)
        self.head_mask = torch.zeros(self.B, Hq, (self.NB + 31) // 32, dtype=i32, device=dev)
        self.union_idx = torch.zeros(self.B, self.Hkv, self.NB, dtype=i32, device=dev)
        self.union_cnt = torch.zeros(self.B, self.Hkv, dtype=i32, device=dev)
        self.head_cnt = torch.zeros(self.B, Hq, dtype=i32, device=dev)
        self.o = torch.zeros(self.B, Hq, self.d, dtype=out_dtype, device=dev)
        self.lse = torch.zeros(self.B, Hq, dtype=f32, device=dev)
        self.cent = self.rmax = self.var = self.cnt = self.vsum = self.vardim = None
        self.dev_status = torch.zeros(1, dtype=i32, device=dev)

    # -- metadata, thresholds, screening -----------------------------------------------
    def _alloc_meta(self):
        B, Hkv, NB, d, dev = self.B, self.Hkv, self.NB, self.d, self.device
        f32 = torch.float32
        self.cent = torch.zeros(B, Hkv, d, NB, device=dev,
                                dtype=torch.bfloat16 if self.cent_format == "bf16" else f32)
        self.rmax = torch.zeros(B, Hkv, NB, dtype=f32, device=dev)
        self.var = torch.zeros(B, Hkv, NB, dtype=f32, device=dev)
        self.cnt = torch.zeros(B, Hkv, NB, dtype=torch.int32, device=dev)
        if self.prune == "floor":
            self.vsum = torch.zeros(B, Hkv, NB, d, dtype=f32, device=dev)
        if self.bound == "prob_dim":
            self.vardim = torch.zeros(B, Hkv, d, NB, dtype=f32, device=dev)

    def build_meta(self, blk_begin: int = 0, blk_end: int = -1, stream=None):
        """Block metadata of blocks [blk_begin, blk_end) of every row.  Screening knows
        these alone, not the lengths or the table: call it after an append of more than
        one token, a fork or a free, over the blocks that changed (append_update after a
        decode step's append).  It reads every key of those blocks."""
        c = self.cache

        def call():
            if self.cent is None:
                if torch.cuda.is_current_stream_capturing():
                    raise ValueError("call build_meta once before it is captured")
                self._alloc_meta()
            L.eta_paged_build_block_meta(self.dims, c.n_pages, c.K, c.V, c.table, c.lengths,
                                         blk_begin, blk_end, self.cent, self.rmax, self.var,
                                         self.cnt, self.vsum, self.dev_status,
                                         vardim=self.vardim)
        _on(self.device, stream, call)

    def append_update(self, stream=None):
        """Recompute the tail block of every row (call after appending a token)."""
        self.build_meta(L.TAIL_BLOCK, -1, stream)

    def predict_tau(self, q, W=None, bias=None, tau_const=None, stream=None):
        self._check_q(q)
        if W is None and tau_const is None:
            raise ValueError("W or tau_const")
        for name, t, shape in (("W", W, (self.Hq * self.d, self.Hq)), ("bias", bias, (self.Hq,)),
                               ("tau_const", tau_const, (self.Hq,))):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape
                                  or not t.is_contiguous() or t.device != self.device):
                raise ValueError(f"{name} must be contiguous fp32 {shape} on {self.device}")
        _on(self.device, stream, L.eta_predict_tau, self.dims, q, W, bias, tau_const, self.tau,
            self.dev_status)
        return self.tau

    def screen(self, q, tau=None, stream=None):
        self._check_q(q)
        if self.cent is None:
            raise ValueError("screen needs build_meta first")
        tau = self.tau if tau is None else self._check_tau(tau)

        def call():
            L.eta_screen(self.dims, q, tau, self.cent, self.rmax, self.var, self.cnt, self.bound,
                         self.z, self.scale, self.head_mask, self.union_idx, self.union_cnt, None,
                         self.head_cnt, self.ws_screen, self.dev_status, vardim=self.vardim)
        _on(self.device, stream, call)

    # -- attention ----------------------------------------------------------------------
    def _check_q(self, q):
        if (q.dtype is not torch.bfloat16 or q.shape != (self.B, self.Hq, self.d)
                or not q.is_contiguous() or q.device != self.device):
            raise ValueError(f"q must be contiguous bf16 [{self.B}, {self.Hq}, {self.d}] on "
                             f"{self.device}")

    def _check_tau(self, tau):
        if (tau.dtype is not torch.float32 or tau.shape != (self.B, self.Hq)
                or not tau.is_contiguous() or tau.device != self.device):
            raise ValueError(f"tau must be contiguous fp32 [{self.B}, {self.Hq}] on "
                             f"{self.device}")
        return tau

    def _gate(self, tau):
        """(thresholds or None, temperature) of a call."""
        if self.T is None:
            return None, 0.0
        return (self.tau if tau is None else self._check_tau(tau)), self.T

    def decode(self, q, tau=None, stream=None, all_blocks: bool = False):
        """Attention over the admitted blocks that screen() left (all_blocks: over every
        block of the row), gated by tau (default: the thresholds of predict_tau)."""
        self._check_q(q)
        tau, T = self._gate(tau)
        c = self.cache
        if all_blocks:
            idx = cnt = None
            prune = "skip"
        else:
            idx, cnt, prune = self.union_idx, self.union_cnt, self.prune
        _on(self.device, stream, L.eta_paged_decode, self.dims, c.n_pages, q, tau, c.K, c.V, c.table,
            c.lengths, idx, cnt, T, self.scale, prune, self.vsum, self.cnt, self.o, self.lse,
            self.ws_decode, self.dev_status)
        return self.o, self.lse

    def dense_decode(self, q, stream=None):
        """Standard softmax attention over every key of every row (no gate)."""
        self._check_q(q)
        c = self.cache
        _on(self.device, stream, L.eta_paged_decode, self.dims, c.n_pages, q, None, c.K, c.V, c.table,
            c.lengths, None, None, 0.0, self.scale, "skip", None, None, self.o, self.lse,
            self.ws_decode, self.dev_status)
        return self.o, self.lse

    def shared_decode(self, q, group_off, prefix_len, tau=None, stream=None):
        """Attention over every key of every row (gated by tau unless T is None), each
        group's shared prefix read once: rows group_off[k] .. group_off[k + 1] - 1 hold
        the same pages for their first prefix_len[k] tokens.  group_off int32
        [n_groups + 1], prefix_len int32 [n_groups] (lists are copied to the device)."""
        self._check_q(q)
        tau, T = self._gate(tau)
        c = self.cache

        def call():
            off, pre = _index_tensor(group_off, self.device), _index_tensor(prefix_len, self.device)
            n = pre.numel()
            if not 1 <= n <= self.B:
                raise ValueError("between 1 and B groups")
            if off.numel() != n + 1:
                raise ValueError("group_off has one entry more than prefix_len")
            if self.ws_shared is None:
                # for any number of groups: a captured call keeps its address
                size = L.eta_shared_decode_workspace_size(self.dims, self.B)
                self.ws_shared = torch.empty(size, dtype=torch.uint8, device=self.device)
            L.eta_shared_decode(self.dims, c.n_pages, n, q, tau, c.K, c.V, c.table, c.lengths, off,
                                pre, T, self.scale, self.o, self.lse, self.ws_shared,
                                self.dev_status)
        _on(self.device, stream, call)
        return self.o, self.lse

    def step(self, q, W=None, bias=None, tau_const=None, stream=None, append: bool = True):
        """One ETA decode step after cache.append: tail-block metadata (on append),
        thresholds, screening, gated decode over the admitted blocks."""
        if append:
            self.append_update(stream)
        self.predict_tau(q, W, bias, tau_const, stream)
        self.screen(q, stream=stream)
        return self.decode(q, stream=stream)

    def check_status(self):
        """Synchronizes, reads the device status word, raises on any error bit."""
        _raise_status(self.dev_status)
