"""Operators beside the engine, torch tensors in: the paged 4-bit KV cache with its attention and what keeps
it within a bound, trees of drafted tokens and their verification, and log-probabilities (the dec_kvq_*,
dec_draft_tree, dec_verify_drafts and dec_logprobs entry points of include/dec.h, which define them).

Every call is queued on the current stream of the tensors' device (or on `stream`, a torch stream or
a cudaStream_t) and returns without waiting; none reads device memory on the host, so all may be
captured into CUDA graphs. Outputs and workspaces come from torch's allocator unless they are given;
rows that belong to no sequence are not written (a fresh output holds anything there). What a kernel finds wrong
in device data (a page id, a length) is recorded in the cache's status word: KvqCache.check().
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import capi
from .capi import (DEC_BF16, DEC_F32, DEC_MAX_TREE, DecDraftTreeArgs, DecError, DecKvqAppendArgs, DecKvqAttentionArgs,
                   DecKvqCache, DecKvqHeaviestArgs, DecKvqMassArgs, DecKvqMoveArgs, DecKvqSeqs, DecLogprobsArgs, DecRows,
                   DecVerifyDraftsArgs)

_DTYPES = {torch.bfloat16: DEC_BF16, torch.float32: DEC_F32}


def _raise(st: int, where: str):
    raise DecError(st, where, capi.lib().dec_op_error().decode())


def _current_raw_stream(index: int) -> int:
    """The raw handle of a device's current torch stream (0: the legacy stream)."""
    return torch.cuda.current_stream(index).cuda_stream


# (torch's own short cut to it takes a microsecond less; a torch without CUDA does not have it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream)


def _on_stream(stream, device: torch.device):
    """A torch stream, or a cudaStream_t, of the tensors' device as its current stream: the whole call,
    its outputs and the copies it makes included, then belongs to it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _call(f, index: int, *args) -> int:
    """f(*args, current stream) with the tensors' device as the current one."""
    if torch.cuda.current_device() == index:
        return f(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return f(*args, _raw_stream(index))


def _readable(t: torch.Tensor) -> torch.Tensor:
    """Rows of heads that the kernels can read as they lie, copied if they cannot."""
    per = 16 // t.element_size()
    s0, s1, s2 = t.stride()
    if s2 != 1 or s0 % per or s1 % per or t.data_ptr() % 16:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _out(t: torch.Tensor, name: str, shape, index: int) -> torch.Tensor:
    """A bf16 output given by the caller: written as it lies, so its layout has to fit."""
    if t.shape != shape or t.dtype != torch.bfloat16 or t.get_device() != index:
        raise ValueError(f"{name} must be bfloat16 {list(shape)} on cuda:{index}")
    if t.stride(2) != 1 or t.stride(0) % 8 or t.stride(1) % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: heads contiguous, rows and strides multiples of 16 bytes")
    return t


def _ints(t: torch.Tensor, name: str, n: int, index: int) -> int:
    """The address of a contiguous int32 vector of n on the tensors' device."""
    if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be contiguous int32 [{n}] on cuda:{index}")
    return t.data_ptr()


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
        self._index = pages.get_device()
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
        i, shape = self._index, table.shape
        batch = lengths.numel()
        if (lengths.dtype is not torch.int32 or table.dtype is not torch.int32 or lengths.get_device() != i or
                table.get_device() != i or lengths.dim() != 1 or len(shape) != 2 or shape[0] != batch or
                not lengths.is_contiguous()):
            raise ValueError(f"lengths must be int32 [batch] and table int32 [batch, max_pages] on {self.device}")
        s0, s1 = table.stride()
        if s1 != 1 and shape[1] > 1:
            raise ValueError("table: the pages of a sequence must lie next to each other")
        if cu is None:
            if n_tokens != batch:
                raise ValueError("without cu_tokens every sequence has one row")
            return DecKvqSeqs(batch, n_tokens, None, lengths.data_ptr(), table.data_ptr(), shape[1], s0)
        if cu.dtype is not torch.int32 or cu.get_device() != i or cu.dim() != 1 or cu.numel() != batch + 1 or not cu.is_contiguous():
            raise ValueError(f"cu_tokens must be contiguous int32 [{batch + 1}] on {self.device}")
        return DecKvqSeqs(batch, n_tokens, cu.data_ptr(), lengths.data_ptr(), table.data_ptr(), shape[1], s0)

    def append(self, k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
               cu_tokens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
               q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
               rope: Optional[torch.Tensor] = None, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
               stream=None, positions: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """Append k, v ([n, n_kv_heads, head_dim], bf16 or fp32) at the sequences' positions; with q
        ([n, n_heads, head_dim], of the same type) return it normalised and rotated, in bf16. rope: a
        rope_table() of rotary_dim = 2 * rope.shape[1]. positions (int32 [n]): the rows' rotary positions,
        where those are not their places in the cache (a tree's tokens, a sequence that positions were taken from)."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.append(k, v, lengths, table, cu_tokens, q, q_norm, k_norm, eps, rope, interleaved, q_out,
                                   positions=positions)
        index, hd, hkv, dtype = self._index, self.head_dim, self.n_kv_heads, k.dtype
        shape = k.shape
        dt = _DTYPES.get(dtype)
        if dt is None or v.dtype is not dtype:
            raise ValueError("q, k and v must be bfloat16 or float32, all of one type")
        if (len(shape) != 3 or shape[1] != hkv or shape[2] != hd or v.shape != shape or k.get_device() != index or
                v.get_device() != index):
            raise ValueError(f"k and v must be [n, {hkv}, {hd}] on {self.device}")
        n = shape[0]
        k, v = _readable(k), _readable(v)
        (k0, k1, _), (v0, v1, _) = k.stride(), v.stride()
        hq = qp = q0 = q1 = op = o0 = o1 = 0
        if q is not None:
            shape = q.shape
            if q.dtype is not dtype or len(shape) != 3 or shape[0] != n or shape[2] != hd or q.get_device() != index:
                raise ValueError(f"q must be [{n}, n_heads, {hd}] of k's type on {self.device}")
            hq = shape[1]
            q = _readable(q)
            q_out = torch.empty(shape, dtype=torch.bfloat16, device=self.device) if q_out is None else _out(q_out, "q_out", shape, index)
            qp, op = q.data_ptr(), q_out.data_ptr()
            (q0, q1, _), (o0, o1, _) = q.stride(), q_out.stride()
        for w in (q_norm, k_norm):
            if w is not None and (w.dtype is not torch.bfloat16 or w.shape != (hd,) or not w.is_contiguous() or w.get_device() != index):
                raise ValueError(f"q_norm and k_norm must be contiguous bfloat16 [{hd}] on {self.device}")
        rot = rope_len = 0
        if rope is not None:
            shape = rope.shape
            if rope.dtype is not torch.float32 or len(shape) != 3 or shape[2] != 2 or not rope.is_contiguous() or rope.get_device() != index:
                raise ValueError(f"rope must be contiguous float32 [positions, rotary_dim / 2, 2] on {self.device}")
            rope_len, rot = shape[0], 2 * shape[1]
        a = DecKvqAppendArgs(dt, hq, qp, q0, q1, k.data_ptr(), k0, k1, v.data_ptr(), v0, v1, op, o0, o1,
                             None if q_norm is None else q_norm.data_ptr(), None if k_norm is None else k_norm.data_ptr(),
                             eps, rope.data_ptr() if rot else None, rope_len, rot, interleaved,
                             None if positions is None else _ints(positions, "positions", n, index))
        st = _call(self.lib.dec_kvq_append, index, self.c, self._seqs(lengths, table, cu_tokens, n), a)
        if st:
            _raise(st, "dec_kvq_append")
        return q_out if q is not None else None

    def gather(self, lengths: torch.Tensor, table: torch.Tensor, n_tokens: int, cu_tokens: Optional[torch.Tensor] = None,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The values the cache holds at the sequences' positions: k, v bf16 [n_tokens, n_kv_heads, head_dim]."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.gather(lengths, table, n_tokens, cu_tokens, out)
        hkv, hd = self.n_kv_heads, self.head_dim
        shape = (n_tokens, hkv, hd)
        if out is None:
            k = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            v = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            kr, vr = DecRows(k.data_ptr(), hkv * hd, hd), DecRows(v.data_ptr(), hkv * hd, hd)
        else:
            k, v = _out(out[0], "k", shape, self._index), _out(out[1], "v", shape, self._index)
            kr, vr = DecRows(k.data_ptr(), *k.stride()[:2]), DecRows(v.data_ptr(), *v.stride()[:2])
        st = _call(self.lib.dec_kvq_gather, self._index, self.c, self._seqs(lengths, table, cu_tokens, n_tokens), kr, vr)
        if st:
            _raise(st, "dec_kvq_gather")
        return k, v

    def attention(self, q: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                  cu_tokens: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None, causal: bool = True,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False, stream=None,
                  tree_mask: Optional[torch.Tensor] = None):
        """Attention of q (bf16 [n, n_heads, head_dim]) over the cache: row j of a sequence attends to
        positions 0 .. lengths + j (causal) or 0 .. lengths - 1. max_tokens: an upper bound of the rows
        of one sequence, which also chooses the kernel (default: 1 without cu_tokens; with them n, and the kernel
        that suits the sequences' mean). tree_mask (int32 [n, words], draft_tree's): each row attends to positions
        0 .. lengths - 1 and, of its sequence's rows, to those whose bits are set. Returns out (bf16, shaped as q), or
        (out, lse) with lse fp32 [n, n_heads]."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.attention(q, lengths, table, cu_tokens, max_tokens, causal, scale, out, return_lse,
                                      tree_mask=tree_mask)
        index, hd, shape = self._index, self.head_dim, q.shape
        if q.dtype is not torch.bfloat16 or len(shape) != 3 or shape[2] != hd or q.get_device() != index:
            raise ValueError(f"q must be bfloat16 [n, n_heads, {hd}] on {self.device}")
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        n, hq, _ = shape
        q = _readable(q)
        mask = None
        mask_stride = words = 0
        if tree_mask is not None:
            if not causal:
                raise ValueError("a tree's rows stand in the cache: causal")
            if (tree_mask.dtype not in (torch.int32, torch.uint32) or tree_mask.dim() != 2 or tree_mask.shape[0] != n or
                    tree_mask.shape[1] < 1 or (tree_mask.stride(1) != 1 and tree_mask.shape[1] > 1) or
                    tree_mask.get_device() != index):
                raise ValueError(f"tree_mask must be int32 [{n}, words] with adjacent words on {self.device}")
            mask, mask_stride, words = tree_mask.data_ptr(), tree_mask.stride(0), tree_mask.shape[1]
        out = torch.empty(shape, dtype=torch.bfloat16, device=self.device) if out is None else _out(out, "out", shape, index)
        lse = torch.empty((n, hq), dtype=torch.float32, device=self.device) if return_lse else None
        # The bound of n rows says nothing about single sequences: their mean does, unless most of them are empty.
        # Mean against bound, us (32 query, 8 KV heads of 128, all on 2 k): 64 sequences of 1 row 43 / 112, of 2
        # 46 / 113; one of 128 and 63 of 1 87 / 121, one of 256 and 63 of 1 127 / 127, of none 83 / 33.
        likely = 0
        if max_tokens is None:
            max_tokens = 1 if cu_tokens is None else n
            likely = -(-n // max(1, lengths.numel()))
        s = self._seqs(lengths, table, cu_tokens, n)
        key = (hq, max_tokens)  # (what its size goes by; a batch of 1 or many is alike)
        need = self._ws.get(key)
        if need is None:
            with torch.cuda.device(index):
                need = self._ws[key] = max(0, self.lib.dec_kvq_attention_workspace(self.c, hq, s.batch, max_tokens))
        # (its own workspace: calls on several streams, or in several captured graphs, may run at once)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        (q0, q1, _), (o0, o1, _) = q.stride(), out.stride()
        a = DecKvqAttentionArgs(hq, q.data_ptr(), q0, q1, out.data_ptr(), o0, o1, None if lse is None else lse.data_ptr(),
                                0.0 if scale is None else scale, causal, max_tokens, ws.data_ptr(), need, likely, mask, mask_stride, words)
        st = _call(self.lib.dec_kvq_attention, index, self.c, s, a)
        if st:
            _raise(st, "dec_kvq_attention")
        return (out, lse) if return_lse else out

    def new_mass(self) -> torch.Tensor:
        """fp32 zeros laid out as the pages: what attention_mass adds up, one number a position and KV head."""
        return torch.zeros((self.n_pages, self.n_kv_heads, self.page_tokens), dtype=torch.float32, device=self.device)

    def _mass(self, t: torch.Tensor, name: str) -> int:
        if (t.dtype is not torch.float32 or t.shape != (self.n_pages, self.n_kv_heads, self.page_tokens) or
                not t.is_contiguous() or t.get_device() != self._index or t.data_ptr() % 16):
            raise ValueError(f"{name} must be contiguous, 16-byte aligned float32 [{self.n_pages}, {self.n_kv_heads}, {self.page_tokens}] on "
                             f"{self.device}")
        return t.data_ptr()

    def attention_mass(self, q: torch.Tensor, lse: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                       mass: torch.Tensor, cu_tokens: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None,
                       causal: bool = True, scale: Optional[float] = None, decay: float = 1.0,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Add the attention weight that cached positions receive from q (with the lse that attention() returned
        for it) to what they have: out = decay * mass + weights, over all rows and the heads of each KV head
        (dec_kvq_mass). mass and out (default: mass itself) are as new_mass() makes them; positions that the
        rows stand at begin anew. A tree's rows go in when their path is accepted and moved into place, as a chain:
        those rows' q and lse at the same lengths. max_tokens: an upper bound of the rows of one sequence, which also chooses the kernel
        (default: 1 without cu_tokens; with them n). Sequences that share pages take calls of their own, one after the
        other: within one call their order on such a page is not fixed."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.attention_mass(q, lse, lengths, table, mass, cu_tokens, max_tokens, causal, scale, decay, out)
        index, hd, shape = self._index, self.head_dim, q.shape
        if q.dtype is not torch.bfloat16 or len(shape) != 3 or shape[2] != hd or q.get_device() != index:
            raise ValueError(f"q must be bfloat16 [n, n_heads, {hd}] on {self.device}")
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        n, hq, _ = shape
        if lse.dtype is not torch.float32 or lse.shape != (n, hq) or not lse.is_contiguous() or lse.get_device() != index:
            raise ValueError(f"lse must be contiguous float32 [{n}, {hq}] on {self.device}")
        out = mass if out is None else out
        q = _readable(q)
        if max_tokens is None:
            max_tokens = 1 if cu_tokens is None else n
        a = DecKvqMassArgs(hq, q.data_ptr(), q.stride(0), q.stride(1), lse.data_ptr(), 0.0 if scale is None else scale, causal,
                           max_tokens, decay, self._mass(mass, "mass"), self._mass(out, "out"))
        st = _call(self.lib.dec_kvq_mass, index, self.c, self._seqs(lengths, table, cu_tokens, n), a)
        if st:
            _raise(st, "dec_kvq_mass")
        return out

    def heaviest(self, mass: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor, budget: int, sinks: int = 0,
                 recent: int = 0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Which positions a cache of `budget` positions a sequence keeps: the first `sinks`, the last `recent` and,
        between them, the heaviest (dec_kvq_heaviest). Returns (kept int32 [batch, n_kv_heads, budget], ascending,
        -1 behind the last; count int32 [batch])."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.heaviest(mass, lengths, table, budget, sinks, recent)
        batch = lengths.numel()
        s = self._seqs(lengths, table, None, batch)
        if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
            raise ValueError("budget must be positive and hold the sinks and the recent positions")
        kept = torch.empty((batch, self.n_kv_heads, budget), dtype=torch.int32, device=self.device)
        count = torch.empty(batch, dtype=torch.int32, device=self.device)
        a = DecKvqHeaviestArgs(self._mass(mass, "mass"), budget, sinks, recent, kept.data_ptr(), count.data_ptr())
        st = _call(self.lib.dec_kvq_heaviest, self._index, self.c, s, a)
        if st:
            _raise(st, "dec_kvq_heaviest")
        return kept, count

    def move(self, index: torch.Tensor, count: torch.Tensor, table: torch.Tensor, start: Optional[torch.Tensor] = None,
             to: Optional[torch.Tensor] = None, mass: Optional[torch.Tensor] = None, stream=None):
        """Move positions as they are held: position start + i of every sequence receives position start + index[.., i]
        (dec_kvq_move). index: int32 [batch, n] for all heads alike (verify_drafts' path) or [batch, n_kv_heads, n]
        (heaviest's kept), ascending, index[i] >= i; count int32 [batch]; start int32 [batch] (default: 0); to: a page
        table to write to (default: in place); mass: weights to move alongside."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.move(index, count, table, start, to, mass)
        i, batch = self._index, count.numel()
        shape = index.shape
        if (index.dtype is not torch.int32 or len(shape) not in (2, 3) or shape[0] != batch or index.get_device() != i or
                (len(shape) == 3 and shape[1] != self.n_kv_heads) or (shape[-1] > 1 and index.stride(-1) != 1)):
            raise ValueError(f"index must be int32 [{batch}, n] or [{batch}, {self.n_kv_heads}, n] with adjacent entries on "
                             f"{self.device}")
        s = self._seqs(count if start is None else start, table, None, batch)
        if start is None:
            s.lengths = None
        tp = pages = stride = 0
        if to is not None:
            if (to.dtype is not torch.int32 or to.dim() != 2 or to.shape[0] != batch or to.get_device() != i or
                    (to.shape[1] > 1 and to.stride(1) != 1)):
                raise ValueError(f"to must be a page table, int32 [{batch}, pages] on {self.device}")
            tp, pages, stride = to.data_ptr(), to.shape[1], to.stride(0)
            if pages == 0 and shape[-1] > 0:
                raise ValueError("to: no pages")
        a = DecKvqMoveArgs(index.data_ptr(), index.stride(0), index.stride(1) if len(shape) == 3 else 0,
                           _ints(count, "count", batch, i), shape[-1], tp, pages, stride,
                           None if mass is None else self._mass(mass, "mass"))
        st = _call(self.lib.dec_kvq_move, i, self.c, s, a)
        if st:
            _raise(st, "dec_kvq_move")

    def evict(self, mass: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor, budget: int, sinks: int = 0,
              recent: int = 0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Bring every sequence down to `budget` positions, in place, its weights with them: heaviest() and move().
        Returns (kept, count); count holds the new lengths. Rows appended later stand there, and keep their rotary
        positions by append(positions=): the engine's steps turn rows by their place and must not follow
        (Engine.step_kvq, kvq_load). Pages in which positions move belong to one sequence."""
        if stream is not None:
            with _on_stream(stream, self.device):
                return self.evict(mass, lengths, table, budget, sinks, recent)
        kept, count = self.heaviest(mass, lengths, table, budget, sinks, recent)
        self.move(kept, count, table, mass=mass)
        return kept, count


class DraftTree(NamedTuple):
    mask: torch.Tensor                 # int32 [n, words]: bit i of a row: row i of its sequence is itself or above it
    positions: Optional[torch.Tensor]  # int32 [n]: rotary positions


def draft_tree(parents: torch.Tensor, lengths: Optional[torch.Tensor], cu_tokens: torch.Tensor,
               max_tokens: Optional[int] = None, stream=None) -> DraftTree:
    """What attention(tree_mask=) and append(positions=) take for trees of drafted tokens (dec_draft_tree): parents
    (int32 [n]) is each row's parent, an earlier row of its sequence. max_tokens: an upper bound of the rows of one
    sequence (default: n, at most 1024)."""
    if stream is not None and parents.is_cuda:
        with _on_stream(stream, parents.device):
            return draft_tree(parents, lengths, cu_tokens, max_tokens)
    if not parents.is_cuda:
        raise ValueError("parents must be int32 [n] on a CUDA device")
    n, index, batch = parents.numel(), parents.get_device(), cu_tokens.numel() - 1
    max_tokens = min(n, DEC_MAX_TREE) if max_tokens is None else max_tokens
    words = max(1, (max_tokens + 31) // 32)
    mask = torch.empty((n, words), dtype=torch.int32, device=parents.device)
    positions = None if lengths is None else torch.empty(n, dtype=torch.int32, device=parents.device)
    a = DecDraftTreeArgs(batch, n, _ints(cu_tokens, "cu_tokens", batch + 1, index), _ints(parents, "parents", n, index),
                         None if lengths is None else _ints(lengths, "lengths", batch, index), max_tokens, mask.data_ptr(),
                         words, None if lengths is None else positions.data_ptr())
    st = _call(capi.lib().dec_draft_tree, index, a)
    if st:
        _raise(st, "dec_draft_tree")
    return DraftTree(mask, positions)


class Verified(NamedTuple):
    path: torch.Tensor         # int32 [batch, max_tokens]: the accepted rows, 0 first; -1 behind the last
    count: torch.Tensor        # int32 [batch]: how many
    next_tokens: torch.Tensor  # int32 [batch]


def verify_drafts(logits: torch.Tensor, tokens: torch.Tensor, uniforms: torch.Tensor, cu_tokens: torch.Tensor,
                  parents: Optional[torch.Tensor] = None, draft_probs: Optional[torch.Tensor] = None,
                  temperature: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None, stream=None) -> Verified:
    """Which path of each sequence's tree (parents None: chain) of drafted tokens the target's probabilities accept,
    and the token that follows it, from given random numbers (dec_verify_drafts). logits: fp32 or bf16 [n, vocab],
    each row the target's after that token; tokens int32 [n], row 0 of a sequence its last known one; uniforms fp32
    [n] in [0, 1); draft_probs fp32 [n, vocab], what each row's children were drawn from (None: certainty);
    temperature fp32 [batch] (None: 1; 0: greedy). max_tokens: an upper bound of the rows of one sequence (default: n,
    at most 1024). path and count are what KvqCache.move takes."""
    if stream is not None and logits.is_cuda:
        with _on_stream(stream, logits.device):
            return verify_drafts(logits, tokens, uniforms, cu_tokens, parents, draft_probs, temperature, max_tokens)
    dt = _DTYPES.get(logits.dtype)
    shape = logits.shape
    if dt is None or len(shape) != 2 or not logits.is_cuda:
        raise ValueError("logits must be bfloat16 or float32 [rows, vocab] on a CUDA device")
    n, vocab = shape
    if n >= 2 ** 31 or vocab >= 2 ** 31:
        raise ValueError("logits: 2^31 rows or ids")
    dev, index, batch = logits.device, logits.get_device(), cu_tokens.numel() - 1
    if logits.stride(1) != 1 and vocab > 1:
        logits = logits.contiguous()
    qp = qs = 0
    if draft_probs is not None:
        if draft_probs.dtype is not torch.float32 or draft_probs.shape != shape or draft_probs.get_device() != index:
            raise ValueError(f"draft_probs must be float32 {list(shape)} on {dev}")
        if draft_probs.stride(1) != 1 and vocab > 1:
            draft_probs = draft_probs.contiguous()
        qp, qs = draft_probs.data_ptr(), draft_probs.stride(0)
    for name, t, size in (("uniforms", uniforms, n), ("temperature", temperature, batch)):
        if t is not None and (t.dtype is not torch.float32 or t.dim() != 1 or t.numel() != size or not t.is_contiguous() or
                              t.get_device() != index):
            raise ValueError(f"{name} must be contiguous float32 [{size}] on {dev}")
    max_tokens = min(n, DEC_MAX_TREE) if max_tokens is None else max_tokens
    path = torch.empty((batch, max(0, max_tokens)), dtype=torch.int32, device=dev)
    count = torch.empty(batch, dtype=torch.int32, device=dev)
    nxt = torch.empty(batch, dtype=torch.int32, device=dev)
    lib = capi.lib()
    need = lib.dec_verify_drafts_workspace(n)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    a = DecVerifyDraftsArgs(logits.data_ptr(), dt, vocab, logits.stride(0), qp, qs, batch, n,
                            _ints(cu_tokens, "cu_tokens", batch + 1, index), _ints(tokens, "tokens", n, index),
                            None if parents is None else _ints(parents, "parents", n, index), uniforms.data_ptr(),
                            None if temperature is None else temperature.data_ptr(), max_tokens, path.data_ptr(),
                            count.data_ptr(), nxt.data_ptr(), ws.data_ptr(), need)
    st = _call(lib.dec_verify_drafts, index, a)
    if st:
        _raise(st, "dec_verify_drafts")
    return Verified(path, count, nxt)


class LogProbs(NamedTuple):
    logprob: Optional[torch.Tensor]       # fp32 [rows]
    rank: Optional[torch.Tensor]          # int32 [rows]
    entropy: torch.Tensor                 # fp32 [rows], nats
    top_ids: Optional[torch.Tensor]       # int32 [rows, top_n]
    top_logprobs: Optional[torch.Tensor]  # fp32 [rows, top_n]


def logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top_n: int = 0, stream=None) -> LogProbs:
    """Log-probabilities of `targets` (int32 [rows]) under logits (fp32 or bf16 [rows, vocab]), their
    ranks, the rows' entropies and the top_n likeliest ids with their log-probabilities."""
    if stream is not None and logits.is_cuda:
        with _on_stream(stream, logits.device):
            return logprobs(logits, targets, top_n)
    dt = _DTYPES.get(logits.dtype)
    shape = logits.shape
    if dt is None or len(shape) != 2 or not logits.is_cuda:
        raise ValueError("logits must be bfloat16 or float32 [rows, vocab] on a CUDA device")
    rows, vocab = shape
    if rows >= 2 ** 31 or vocab >= 2 ** 31:
        raise ValueError("logits: 2^31 rows or ids")
    s0, s1 = logits.stride()
    if s1 != 1 and vocab > 1:
        logits = logits.contiguous()
        s0 = vocab
    dev, index = logits.device, logits.get_device()
    lp = rank = ids = tlp = lpp = rankp = tp = idp = tlpp = None
    if targets is not None:
        if (targets.dtype is not torch.int32 or targets.get_device() != index or targets.dim() != 1 or
                targets.numel() != rows or not targets.is_contiguous()):
            raise ValueError(f"targets must be contiguous int32 [{rows}] on {dev}")
        lp = torch.empty(rows, dtype=torch.float32, device=dev)
        rank = torch.empty(rows, dtype=torch.int32, device=dev)
        tp, lpp, rankp = targets.data_ptr(), lp.data_ptr(), rank.data_ptr()
    ent = torch.empty(rows, dtype=torch.float32, device=dev)
    if top_n > 0:
        ids = torch.empty((rows, top_n), dtype=torch.int32, device=dev)
        tlp = torch.empty((rows, top_n), dtype=torch.float32, device=dev)
        idp, tlpp = ids.data_ptr(), tlp.data_ptr()
    a = DecLogprobsArgs(logits.data_ptr(), dt, rows, vocab, s0, tp, lpp, rankp, ent.data_ptr(), top_n, idp, tlpp)
    st = _call(capi.lib().dec_logprobs, index, a)
    if st:
        _raise(st, "dec_logprobs")
    return LogProbs(lp, rank, ent, ids, tlp)
