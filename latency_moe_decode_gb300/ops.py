"""Operators beside the engine, torch tensors in: the paged 4-bit KV cache with its attention, and
log-probabilities (the dec_kvq_* and dec_logprobs entry points of include/dec.h, which define them).

Every call is queued on the current stream of the tensors' device (or on `stream`, a torch stream or
a cudaStream_t) and returns without waiting; none reads device memory on the host, so all may be
captured into CUDA graphs. Outputs and workspaces come from torch's allocator unless they are given;
rows that belong to no sequence are not written (a fresh output holds anything there). What a kernel finds wrong
in device data (a page id, a length) is recorded in the cache's status word: KvqCache.check().
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple

import torch

from . import capi
from .capi import (DEC_BF16, DEC_F32, DecError, DecKvqAppendArgs, DecKvqAttentionArgs, DecKvqCache, DecKvqSeqs,
                   DecLogprobsArgs, DecRows)

_DTYPES = {torch.bfloat16: DEC_BF16, torch.float32: DEC_F32}


def _raise(st: int, where: str):
    raise DecError(st, where, capi.lib().dec_op_error().decode())


def _stream(device) -> int:
    """cudaStream_t of the device's current torch stream (0: the legacy stream)."""
    return torch.cuda.current_stream(device).cuda_stream


def _on_stream(f):
    """Give f a `stream` argument (a torch stream or a cudaStream_t): the whole call, its outputs and
    the copies it makes included, then belongs to that stream."""
    @functools.wraps(f)
    def call(*a, stream=None, **kw):
        if stream is None:
            return f(*a, **kw)
        with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))):
            return f(*a, **kw)
    return call


class _on:
    """The tensors' device as the current one for the call."""

    def __init__(self, device):
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)


def _ints(t: Optional[torch.Tensor], n: int, name: str, device) -> Optional[int]:
    """Address of a contiguous int32 vector of at least n entries."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.device != device or t.dim() != 1 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous int32 vector of {n} entries on {device}")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, n: int, heads: Optional[int], hd: int, device) -> torch.Tensor:
    """A [n, heads, hd] tensor whose rows the kernels can read as they lie, copied if they cannot."""
    if t.dim() != 3 or t.shape[0] != n or t.shape[2] != hd or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{n}, {'heads' if heads is None else heads}, {hd}], got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    per = 16 // t.element_size()
    s0, s1, s2 = t.stride()
    if s2 != 1 or s0 % per or s1 % per or t.data_ptr() % 16:
        t = t.contiguous() if not t.is_contiguous() else t.clone()
    return t


def _rows(t: Optional[torch.Tensor]) -> DecRows:
    if t is None:
        return DecRows(None, 0, 0)
    s = t.stride()
    return DecRows(t.data_ptr(), s[0], s[1])


def _out_rows(t: torch.Tensor, name: str, shape, device) -> torch.Tensor:
    """A bf16 output given by the caller: written as it lies, so its layout has to fit."""
    if list(t.shape) != list(shape) or t.dtype != torch.bfloat16 or t.device != device:
        raise ValueError(f"{name} must be bfloat16 {list(shape)} on {device}")
    if t.stride(2) != 1 or t.stride(0) % 8 or t.stride(1) % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: heads contiguous, rows and strides multiples of 16 bytes")
    return t


def rope_table(n: int, rotary_dim: int, theta: float, device="cuda") -> torch.Tensor:
    """fp32 [n, rotary_dim / 2, 2]: cosine and sine of position p's angles p * theta^(-2i / rotary_dim),
    computed in double (the angles of far positions lose their low bits in fp32)."""
    inv = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    a = torch.arange(n, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


class KvqCache:
    """A paged KV cache of one layer held in 4 bits (dec_kvq_cache): pages shared by any number of
    sequences, which the caller hands out through page tables.

    In every call, lengths (int32 [batch]) is the position of each sequence's first row, table (int32
    [batch, max_pages]) its pages, and cu_tokens (int32 [batch + 1]) the bounds of its rows; without
    cu_tokens every sequence has one row."""

    def __init__(self, n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda",
                 pages: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
        """pages: uint8 memory of n_pages pages to use (one layer's share of a larger buffer, say)."""
        self.lib = capi.lib()
        each = self.lib.dec_kvq_page_bytes(page_tokens, n_kv_heads, head_dim)
        if each == 0 or n_pages < 1:
            raise DecError(-5, "KvqCache", f"page_tokens {page_tokens}, n_kv_heads {n_kv_heads}, head_dim {head_dim}")
        self.page_bytes, self.n_kv_heads, self.head_dim, self.page_tokens = each, n_kv_heads, head_dim, page_tokens
        self.n_pages = n_pages
        if pages is None:
            pages = torch.empty(n_pages * each, dtype=torch.uint8, device=device)
        if (pages.dtype != torch.uint8 or not pages.is_cuda or not pages.is_contiguous() or
                pages.numel() < n_pages * each or pages.data_ptr() % 16):
            raise ValueError(f"pages must be {n_pages * each} contiguous, 16-byte aligned bytes on a CUDA device")
        self.pages, self.device = pages, pages.device
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device) if status is None else status
        if self.status.dtype != torch.int32 or self.status.device != self.device:
            raise ValueError("status must be int32 on the pages' device")
        self.c = DecKvqCache(pages.data_ptr(), n_pages, page_tokens, n_kv_heads, head_dim, self.status.data_ptr())
        self._ws = {}

    def check(self):
        """Wait for the device and raise what the kernels found wrong (and forget it)."""
        torch.cuda.synchronize(self.device)
        st = int(self.status.item())
        if st != 0:
            self.status.zero_()
            raise DecError(st, "KvqCache", "a page id, a length or cu_tokens reached out of its range")

    def _seqs(self, lengths, table, cu, n_tokens) -> DecKvqSeqs:
        batch = lengths.shape[0] if lengths.dim() == 1 else -1
        dev = self.device
        if (lengths.dtype != torch.int32 or table.dtype != torch.int32 or batch < 0 or not lengths.is_contiguous() or
                lengths.device != dev or table.device != dev or table.dim() != 2 or table.shape[0] != batch or
                (table.stride(1) != 1 and table.shape[1] > 1)):
            raise ValueError(f"lengths must be int32 [batch] and table int32 [batch, max_pages] on {dev}")
        if cu is None:
            if n_tokens != batch:
                raise ValueError("without cu_tokens every sequence has one row")
            cu_ptr = None
        else:
            cu_ptr = _ints(cu, batch + 1, "cu_tokens", dev)
        return DecKvqSeqs(batch, n_tokens, cu_ptr, lengths.data_ptr(), table.data_ptr(), table.shape[1], table.stride(0))

    @_on_stream
    def append(self, k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
               cu_tokens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
               q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
               rope: Optional[torch.Tensor] = None, interleaved: bool = False,
               q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Append k, v ([n, n_kv_heads, head_dim], bf16 or fp32) at the sequences' positions; with q
        ([n, n_heads, head_dim], of the same type) return it normalised and rotated, in bf16. rope: a
        rope_table() of rotary_dim = 2 * rope.shape[1]."""
        dev, n, hd = self.device, k.shape[0], self.head_dim
        dt = _DTYPES.get(k.dtype)
        if dt is None or v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
            raise ValueError("q, k and v must be bfloat16 or float32, all of one type")
        k = _heads(k, "k", n, self.n_kv_heads, hd, dev)
        v = _heads(v, "v", n, self.n_kv_heads, hd, dev)
        if q is not None:
            q = _heads(q, "q", n, None, hd, dev)
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
            else:
                _out_rows(q_out, "q_out", q.shape, dev)
        for w, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if w is not None and (w.dtype != torch.bfloat16 or w.shape != (hd,) or not w.is_contiguous() or w.device != dev):
                raise ValueError(f"{name} must be contiguous bfloat16 [{hd}] on {dev}")
        rot = rope_len = 0
        if rope is not None:
            if rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[2] != 2 or not rope.is_contiguous() or rope.device != dev:
                raise ValueError(f"rope must be contiguous float32 [positions, rotary_dim / 2, 2] on {dev}")
            rope_len, rot = rope.shape[0], 2 * rope.shape[1]
        a = DecKvqAppendArgs(dt, 0 if q is None else q.shape[1], _rows(q), _rows(k), _rows(v), _rows(q_out if q is not None else None),
                             None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(), eps,
                             None if not rot else rope.data_ptr(), rope_len, rot, interleaved)
        s = self._seqs(lengths, table, cu_tokens, n)
        with _on(dev):
            st = self.lib.dec_kvq_append(self.c, s, a, _stream(dev))
        if st:
            _raise(st, "dec_kvq_append")
        return q_out if q is not None else None

    @_on_stream
    def gather(self, lengths: torch.Tensor, table: torch.Tensor, n_tokens: int, cu_tokens: Optional[torch.Tensor] = None,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The values the cache holds at the sequences' positions: k, v bf16 [n_tokens, n_kv_heads, head_dim]."""
        dev, shape = self.device, (n_tokens, self.n_kv_heads, self.head_dim)
        if out is None:
            k, v = (torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        else:
            k, v = _out_rows(out[0], "k", shape, dev), _out_rows(out[1], "v", shape, dev)
        s = self._seqs(lengths, table, cu_tokens, n_tokens)
        with _on(dev):
            st = self.lib.dec_kvq_gather(self.c, s, _rows(k), _rows(v), _stream(dev))
        if st:
            _raise(st, "dec_kvq_gather")
        return k, v

    @_on_stream
    def attention(self, q: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                  cu_tokens: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None, causal: bool = True,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False):
        """Attention of q (bf16 [n, n_heads, head_dim]) over the cache: row j of a sequence attends to
        positions 0 .. lengths + j (causal) or 0 .. lengths - 1. max_tokens: an upper bound of the rows
        of one sequence (default: n with cu_tokens, 1 without). Returns out (bf16, shaped as q), or
        (out, lse) with lse fp32 [n, n_heads]."""
        dev, n, hd = self.device, q.shape[0], self.head_dim
        if q.dtype != torch.bfloat16:
            raise ValueError("q must be bfloat16")
        q = _heads(q, "q", n, None, hd, dev)
        hq = q.shape[1]
        if out is None:
            out = torch.empty((n, hq, hd), dtype=torch.bfloat16, device=dev)
        else:
            _out_rows(out, "out", (n, hq, hd), dev)
        lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if return_lse else None
        if max_tokens is None:
            max_tokens = 1 if cu_tokens is None else n
        s = self._seqs(lengths, table, cu_tokens, n)
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        with _on(dev):
            key = (hq, s.batch, max_tokens)
            need = self._ws.get(key)
            if need is None:
                need = self._ws[key] = self.lib.dec_kvq_attention_workspace(self.c, hq, s.batch, max_tokens)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
            a = DecKvqAttentionArgs(hq, _rows(q), _rows(out), None if lse is None else lse.data_ptr(),
                                    0.0 if scale is None else scale, causal, max_tokens,
                                    None if ws is None else ws.data_ptr(), max(need, 0))
            st = self.lib.dec_kvq_attention(self.c, s, a, _stream(dev))
        if st:
            _raise(st, "dec_kvq_attention")
        return (out, lse) if return_lse else out


class LogProbs(NamedTuple):
    logprob: Optional[torch.Tensor]       # fp32 [rows]
    rank: Optional[torch.Tensor]          # int32 [rows]
    entropy: torch.Tensor                 # fp32 [rows], nats
    top_ids: Optional[torch.Tensor]       # int32 [rows, top_n]
    top_logprobs: Optional[torch.Tensor]  # fp32 [rows, top_n]


@_on_stream
def logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top_n: int = 0) -> LogProbs:
    """Log-probabilities of `targets` (int32 [rows]) under logits (fp32 or bf16 [rows, vocab]), their
    ranks, the rows' entropies and the top_n likeliest ids with their log-probabilities."""
    dt = _DTYPES.get(logits.dtype)
    if dt is None or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be bfloat16 or float32 [rows, vocab] on a CUDA device")
    if logits.stride(1) != 1 and logits.shape[1] > 1:
        logits = logits.contiguous()
    rows, vocab = logits.shape
    dev = logits.device
    tp = _ints(targets, rows, "targets", dev)
    f32 = dict(dtype=torch.float32, device=dev)
    lp = torch.empty(rows, **f32) if targets is not None else None
    rank = torch.empty(rows, dtype=torch.int32, device=dev) if targets is not None else None
    ent = torch.empty(rows, **f32)
    ids = torch.empty(rows, top_n, dtype=torch.int32, device=dev) if top_n > 0 else None
    tlp = torch.empty(rows, top_n, **f32) if top_n > 0 else None
    a = DecLogprobsArgs(logits.data_ptr(), dt, rows, vocab, logits.stride(0), tp, None if lp is None else lp.data_ptr(),
                        None if rank is None else rank.data_ptr(), ent.data_ptr(), top_n,
                        None if ids is None else ids.data_ptr(), None if tlp is None else tlp.data_ptr())
    with _on(dev):
        st = capi.lib().dec_logprobs(a, _stream(dev))
    if st:
        _raise(st, "dec_logprobs")
    return LogProbs(lp, rank, ent, ids, tlp)
