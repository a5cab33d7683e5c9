"""The serving operators around the draft head (include/nanospec_ops.h).

* ``norm_rotate``     norms of queries and keys for each head, and their
                      rotation by position;
* ``attend_prompt``   causal attention over whole packed prompts;
* ``attend_paged``    attention of a sequence's new tokens (one, or the nodes
                      of a draft tree) over a paged key-value cache;
* ``attend_shared``   the same for sequences that share a long prefix, which
                      is read once for all of them;
* ``KvPages``         the paged cache, of 16 or 8 bits: truncate, fork, extend,
                      write, read, compact, copy;
* ``token_logprobs``  log probabilities of given tokens, entropy, alternatives;
* ``ops_error``       the sticky device flags of these calls.

This module holds the names, defaults and documentation; the argument checks
and calls are native (csrc/ns_binding.cpp), because the small calls take less
time than Python would need for them.  Everything is computed in the library's
kernels, asynchronously on ``stream`` (the current stream when it is None).
Outputs and workspaces come from torch's caching allocator unless they are
passed in; with ``stream`` they are made on that stream, so they are never
memory that work still queued on another one uses.  Tensors used on a stream
other than the one they were made on (inputs, and outputs that are read
elsewhere) must be ordered by the caller, as with any torch op.  None of the
operators has a gradient: outside ``torch.no_grad()`` tensors that require one
are refused.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from .nanospec import NanoSpecError, _check, load_library

FLAG_NO_PAGES = 0x10
FLAG_BAD_SEQ = 0x20
FLAG_SHARED_PAGE = 0x40
MAX_NEW = 64
MAX_ATTEND_SEQS = 4096
MAX_ALTERNATIVES = 32
MAX_PAGE_SEQS = 8192

_binding = None


def _native():
    """The native binding (loaded once; raises when it is not built)."""
    global _binding
    if _binding is None:
        load_library()
        try:
            from . import _serving
        except ImportError as e:
            raise ImportError("the serving operators' binding is missing or does not fit this torch: build.build() "
                              "compiles it with g++ against torch's and Python's headers") from e

        _serving.set_error(NanoSpecError)
        _binding = _serving
    return _binding


def _other(stream):
    """The stream as a torch stream, None where it is the current one."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return None if stream.cuda_stream == torch.cuda.current_stream().cuda_stream else stream


def _on(stream, call):
    """call() with `stream` as the current one, so that what it allocates belongs to that stream: a block that the
    caller's stream has freed may be in use by kernels still queued there, which nothing orders before `stream`.
    The tensors it returns are not reused before both streams are done with them."""
    caller = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        r = call()
    for t in r or ():
        if t is not None:
            t.record_stream(stream)
            t.record_stream(caller)
    return r


def norm_rotate(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, *,
                q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                eps: Optional[float] = None, neighbours: bool = False, q_out: Optional[torch.Tensor] = None,
                k_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norms of queries and keys for each head and their rotation by position, in one pass: q [T, Hq, D] and k
    [T, Hkv, D] or None (bf16 or fp16, D 64 or 128; token and head strides are free multiples of 8 elements).  With
    eps each row x becomes x * weight / sqrt(mean(x^2) + eps), weights [D] of q's type (None: ones); without, it stays.
    Then the pairs i of the first 2 len(inv_freq) columns turn by positions * inv_freq[i]: pairs are halves (i, i +
    len(inv_freq)) or, with neighbours, (2i, 2i + 1); positions int32 [T], inv_freq fp64 (a multiple of 8 of them, up
    to D / 2).  Returns (q, k) rotated, in q_out and k_out where they are given: rows that lie apart, which may be q
    and k themselves but may not overlap them otherwise."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: norm_rotate(q, k, positions, inv_freq, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                          neighbours=neighbours, q_out=q_out, k_out=k_out))
    return _native().norm_rotate(q, k, positions, inv_freq, q_weight, k_weight, eps, neighbours, q_out, k_out)


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, max_len: int, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention over packed prompts: q [T, Hq, D], k and v [T, Hkv, D] (bf16 or fp16, D 64 or 128; token
    and head strides are free positive multiples of 8 elements), cu int32 [B + 1] the sequences' bounds, max_len the
    longest.  Returns (out [T, Hq, D], lse fp32 [T, Hq]).  scale: 1 / sqrt(D) by default.  bf16 values of 2^113 / (a
    sequence's length / 64) and more may overflow in the sums."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: attend_prompt(q, k, v, cu, max_len, scale=scale, out=out, lse=lse))
    return _native().attend_prompt(q, k, v, cu, max_len, scale, out, lse)


def attend_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                 lengths: torch.Tensor, seqs: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, max_len: int = 0, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of n new tokens per sequence over one layer of a paged cache: q [B, n, Hq, D]; k_pages and
    v_pages [pages, Hkv, page_size, D] (strides free); table int32 [max_seqs, pages per sequence], lengths int32
    [max_seqs] (the new tokens included), seqs int32 [B] the cache sequences; mask int64 [B, n]: bit j of word i
    set where new token i sees new token j (None: j <= i).  max_len, a bound on the lengths, takes part in how
    the keys are split: results of another bound may differ by their rounding.  With more than 16 rows (n * Hq / Hkv)
    a q off a 16-byte boundary, or with strides other than positive multiples of 8 elements, takes about three times
    as long, and bf16 values may overflow as in attend_prompt (up to 16 rows: of 2^128 / length).  With k_exp and
    v_exp, uint8 [pages, Hkv, page_size], the pages are a cache of 8 bits (KvPages): codes in e4m3 and the exponent of
    each row (more than 16 rows in fp16 see at most 65504 of what bf16 rows have written).  Returns (out [B, n, Hq, D],
    lse fp32 [B, n, Hq])."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: attend_paged(q, k_pages, v_pages, table, lengths, seqs, mask=mask, scale=scale,
                                           max_len=max_len, out=out, lse=lse, workspace=workspace, k_exp=k_exp,
                                           v_exp=v_exp))
    return _native().attend_paged(q, k_pages, v_pages, table, lengths, seqs, mask, scale, max_len, out, lse,
                                  workspace, k_exp, v_exp, None)


def attend_shared(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                  lengths: torch.Tensor, seqs: torch.Tensor, groups: torch.Tensor, *,
                  mask: Optional[torch.Tensor] = None, scale: Optional[float] = None, max_len: int = 0,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, k_exp: Optional[torch.Tensor] = None,
                  v_exp: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """attend_paged for groups of sequences that begin with the same pages, as samples of one prompt do after
    KvPages.fork: seqs[groups[g]] .. seqs[groups[g + 1] - 1] are a group (groups int32 [G + 1], at most 512 groups, 0
    first and B last).  What the members of a group share is found in the table, in whole tiles of 128 positions, and
    read once for all of them; the rest of each sequence as in attend_paged, from whose results these differ by their
    rounding alone (and bf16 values may overflow as there with more than 16 rows).  q [B, n, Hq, D]: sequences follow
    one another as their tokens do (stride(0) is n * stride(1)), on a 16-byte boundary, with strides that are positive
    multiples of 8.  It pays where a group's members are many, what they share is long and their new tokens are few;
    where it would not (more than 128 rows, n * Hq / Hkv; up to 192 MB of keys and values by max_len, with more than 16
    rows counted as of 16 bits; no fewer groups than sequences, or by max_len less than 128 positions of context), the
    call is attend_paged's.  k_exp and v_exp: as there.  Returns (out [B, n, Hq, D], lse fp32 [B, n, Hq])."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: attend_shared(q, k_pages, v_pages, table, lengths, seqs, groups, mask=mask, scale=scale,
                                            max_len=max_len, out=out, lse=lse, workspace=workspace, k_exp=k_exp,
                                            v_exp=v_exp))
    return _native().attend_paged(q, k_pages, v_pages, table, lengths, seqs, mask, scale, max_len, out, lse,
                                  workspace, k_exp, v_exp, groups)


class KvPages:
    """A paged key-value cache over the caller's tensors: k and v [layers, pages, heads, page_size, dim] (any element
    type; rows of dim consecutive elements, a multiple of 16 bytes; other strides free), table int32 [max_seqs,
    pages per sequence] (-1 past a sequence's last page), lengths int32 [max_seqs], refs int32 [pages] (how many
    sequences hold a page).  Their contents may be changed, but not which tensors they are: the cache works on the
    memory that it was made over.  Its device must be the current one in every call.  ``KvPages.new`` makes an empty
    one.

    A cache of 8 bits: k and v of torch.float8_e4m3fn (64 or 128 columns, pages of a multiple of 8) with k_exp and
    v_exp, uint8 [layers, pages, heads, page_size].  A row stands for its codes times 2^(exponent - 127), and for NaN
    where the byte is 255.  ``write`` rounds bf16 or fp16 rows to it, by the smallest power of two by which the row
    fits (within 2^-40 and 2^40; a row that holds an infinity or NaN gets 255), ``read`` gives rows back, ``attend``
    works on them as they are, and every call that moves rows moves their exponents too."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                 refs: torch.Tensor, k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None):
        self._b = _native()
        self._c = self._b.cache(k, v, table, lengths, refs, k_exp, v_exp)
        # kept alive: the native record has their addresses
        self._over = k, v, table, lengths, refs, k_exp, v_exp

    k = property(lambda self: self._over[0])
    v = property(lambda self: self._over[1])
    table = property(lambda self: self._over[2])
    lengths = property(lambda self: self._over[3])
    refs = property(lambda self: self._over[4])
    k_exp = property(lambda self: self._over[5])
    v_exp = property(lambda self: self._over[6])

    @classmethod
    def new(cls, layers: int, pages: int, kv_heads: int, page_size: int, dim: int, max_seqs: int, max_pages: int,
            dtype=torch.bfloat16, device=None, scaled: bool = False) -> "KvPages":
        """An empty cache of `pages` pages for up to max_seqs sequences of up to max_pages pages each;
        scaled: one of 8 bits, with exponents, whatever dtype says."""
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        k = torch.empty((layers, pages, kv_heads, page_size, dim), dtype=torch.float8_e4m3fn if scaled else dtype,
                        device=device)
        i32 = {"dtype": torch.int32, "device": device}
        exps = [None, None]
        if scaled:
            exps = [torch.zeros(k.shape[:4], dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(k, torch.empty_like(k), torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(pages, **i32), *exps)

    @staticmethod
    def _handle(stream):
        return None if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def truncate(self, seqs: torch.Tensor, new_len: Optional[torch.Tensor] = None, stream=None) -> None:
        """Shortens sequences to new_len [n] positions (None: frees them)."""
        self._b.truncate(self._c, seqs, new_len, self._handle(stream))

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """The empty sequences dst [n] come to hold the pages of src [n]."""
        self._b.fork(self._c, src, dst, self._handle(stream))

    def extend(self, seqs: torch.Tensor, n_new: torch.Tensor, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """Lengthens sequences by n_new [n] positions; a partly filled last page that others hold too is copied."""
        s = None if stream is None else _other(stream)
        if s is not None:
            _on(s, lambda: self.extend(seqs, n_new, workspace))
        else:
            self._b.extend(self._c, seqs, n_new, workspace)

    def write(self, layer: int, seqs: torch.Tensor, cu: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
              stream=None) -> None:
        """Writes k_new and v_new [tokens, heads, dim] as the last positions of the sequences in one layer; tokens
        cu[i] .. cu[i + 1] - 1 are sequence seqs[i]'s (cu int32 [n + 1]).  Into a cache of 8 bits: bf16 or fp16."""
        self._b.write(self._c, layer, seqs, cu, k_new, v_new, self._handle(stream))

    def read(self, layer: int, seqs: torch.Tensor, cu: torch.Tensor, tokens: int, *, dtype=None,
             k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The other way round: the last cu[i + 1] - cu[i] positions of each sequence seqs[i] in one layer, as rows
        cu[i] .. cu[i + 1] - 1 of (k, v) [tokens, heads, dim]; of a cache of 8 bits what the codes stand for, in dtype
        (bf16, which holds every value, or fp16), otherwise the elements as they are.  Rows of no sequence, or of an
        invalid one, are not written."""
        s = None if stream is None else _other(stream)
        if s is not None:
            return _on(s, lambda: self.read(layer, seqs, cu, tokens, dtype=dtype, k_out=k_out, v_out=v_out))
        scaled = self.k_exp is not None
        if dtype not in ((None, torch.bfloat16, torch.float16) if scaled else (None, self.k.dtype)):
            raise ValueError(f"a cache of {self.k.dtype} does not give rows of {dtype}")
        return self._b.read(self._c, layer, seqs, cu, tokens, scaled and dtype == torch.float16, k_out, v_out)

    def compact(self, seqs: torch.Tensor, base: torch.Tensor, keep: torch.Tensor, n_keep: torch.Tensor,
                stream=None) -> None:
        """From position base [n] on, keeps the positions base + keep [n, m] (the first n_keep [n] of each row,
        strictly increasing) in every layer, and drops the rest."""
        self._b.compact(self._c, seqs, base, keep, n_keep, self._handle(stream))

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies pages src [n] onto pages dst [n] in every layer."""
        self._b.copy(self._c, src, dst, self._handle(stream))

    def attend(self, layer: int, q: torch.Tensor, seqs: torch.Tensor, groups: Optional[torch.Tensor] = None,
               **kw) -> Tuple[torch.Tensor, torch.Tensor]:
        """attend_paged over one layer of this cache; with groups, attend_shared."""
        if self.k_exp is not None:
            kw = dict(kw, k_exp=self.k_exp[layer], v_exp=self.v_exp[layer])
        if groups is not None:
            return attend_shared(q, self.k[layer], self.v[layer], self.table, self.lengths, seqs, groups, **kw)
        return attend_paged(q, self.k[layer], self.v[layer], self.table, self.lengths, seqs, **kw)


class TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor      # fp32 [rows, m]
    entropy: torch.Tensor       # fp32 [rows]
    lse: torch.Tensor           # fp32 [rows]
    top_ids: torch.Tensor       # int32 [rows, k]
    top_logprobs: torch.Tensor  # fp32 [rows, k]


def token_logprobs(logits: torch.Tensor, ids: Optional[torch.Tensor] = None, k: int = 0, *, temperature: float = 1.0,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of ids int32 [rows, m] (-1: an empty place, NaN) under softmax(logits / temperature),
    logits [rows, V] fp32, bf16 or fp16 with a free row stride; the distribution's entropy and log-sum-exp, and
    the k most probable tokens (ties to the smaller id)."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: token_logprobs(logits, ids, k, temperature=temperature))
    return TokenLogprobs._make(_native().token_logprobs(logits, ids, k, temperature))


def ops_error(clear: bool = False) -> int:
    """The sticky NS_FLAG_* mask of these calls on the current device (synchronises it)."""
    f = ctypes.c_uint32()
    _check(load_library().ns_ops_get_error(ctypes.byref(f), int(clear)), "ns_ops_get_error")
    return int(f.value)
