"""The serving operators around the draft head (include/nanospec_ops.h).

* ``attend_prompt``   causal attention over whole packed prompts;
* ``attend_paged``    attention of a sequence's new tokens (one, or the nodes
                      of a draft tree) over a paged key-value cache;
* ``KvPages``         the paged cache: truncate, fork, extend, write, compact, copy;
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
        t.record_stream(stream)
        t.record_stream(caller)
    return r


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, max_len: int, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention over packed prompts: q [T, Hq, D], k and v [T, Hkv, D] (bf16 or fp16, D 64 or 128; token
    and head strides are free positive multiples of 8 elements), cu int32 [B + 1] the sequences' bounds, max_len the
    longest.  Returns (out [T, Hq, D], lse fp32 [T, Hq]).  scale: 1 / sqrt(D) by default."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: attend_prompt(q, k, v, cu, max_len, scale=scale, out=out, lse=lse))
    return _native().attend_prompt(q, k, v, cu, max_len, scale, out, lse)


def attend_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                 lengths: torch.Tensor, seqs: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, max_len: int = 0, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of n new tokens per sequence over one layer of a paged cache: q [B, n, Hq, D]; k_pages and
    v_pages [pages, Hkv, page_size, D] (strides free); table int32 [max_seqs, pages per sequence], lengths int32
    [max_seqs] (the new tokens included), seqs int32 [B] the cache sequences; mask int64 [B, n]: bit j of word i
    set where new token i sees new token j (None: j <= i).  max_len, a bound on the lengths, takes part in how
    the keys are split: results of another bound may differ by their rounding.  With more than 16 rows (n * Hq / Hkv)
    a q off a 16-byte boundary, or with strides other than positive multiples of 8 elements, takes about three times
    as long.  Returns (out [B, n, Hq, D], lse fp32 [B, n, Hq])."""
    s = None if stream is None else _other(stream)
    if s is not None:
        return _on(s, lambda: attend_paged(q, k_pages, v_pages, table, lengths, seqs, mask=mask, scale=scale,
                                           max_len=max_len, out=out, lse=lse, workspace=workspace))
    return _native().attend_paged(q, k_pages, v_pages, table, lengths, seqs, mask, scale, max_len, out, lse,
                                  workspace)


class KvPages:
    """A paged key-value cache over the caller's tensors: k and v [layers, pages, heads, page_size, dim] (any element
    type; rows of dim consecutive elements, a multiple of 16 bytes; other strides free), table int32 [max_seqs,
    pages per sequence] (-1 past a sequence's last page), lengths int32 [max_seqs], refs int32 [pages] (how many
    sequences hold a page).  Their contents may be changed, but not which tensors they are: the cache works on the
    memory that it was made over.  Its device must be the current one in every call.  ``KvPages.new`` makes an empty
    one."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                 refs: torch.Tensor):
        self._b = _native()
        self._c = self._b.cache(k, v, table, lengths, refs)
        self._over = k, v, table, lengths, refs  # kept alive: the native record has their addresses

    k = property(lambda self: self._over[0])
    v = property(lambda self: self._over[1])
    table = property(lambda self: self._over[2])
    lengths = property(lambda self: self._over[3])
    refs = property(lambda self: self._over[4])

    @classmethod
    def new(cls, layers: int, pages: int, kv_heads: int, page_size: int, dim: int, max_seqs: int, max_pages: int,
            dtype=torch.bfloat16, device=None) -> "KvPages":
        """An empty cache of `pages` pages for up to max_seqs sequences of up to max_pages pages each."""
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        k = torch.empty((layers, pages, kv_heads, page_size, dim), dtype=dtype, device=device)
        i32 = {"dtype": torch.int32, "device": device}
        return cls(k, torch.empty_like(k), torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(pages, **i32))

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
        cu[i] .. cu[i + 1] - 1 are sequence seqs[i]'s (cu int32 [n + 1])."""
        self._b.write(self._c, layer, seqs, cu, k_new, v_new, self._handle(stream))

    def compact(self, seqs: torch.Tensor, base: torch.Tensor, keep: torch.Tensor, n_keep: torch.Tensor,
                stream=None) -> None:
        """From position base [n] on, keeps the positions base + keep [n, m] (the first n_keep [n] of each row,
        strictly increasing) in every layer, and drops the rest."""
        self._b.compact(self._c, seqs, base, keep, n_keep, self._handle(stream))

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies pages src [n] onto pages dst [n] in every layer."""
        self._b.copy(self._c, src, dst, self._handle(stream))

    def attend(self, layer: int, q: torch.Tensor, seqs: torch.Tensor, **kw) -> Tuple[torch.Tensor, torch.Tensor]:
        """attend_paged over one layer of this cache."""
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
