"""The serving operators around the draft head (include/nanospec_ops.h).

* ``attend_prompt``   causal attention over whole packed prompts;
* ``attend_paged``    attention of a sequence's new tokens (one, or the nodes
                      of a draft tree) over a paged key-value cache;
* ``KvPages``         the paged cache: truncate, fork, extend, write, compact, copy;
* ``token_logprobs``  log probabilities of given tokens, entropy, alternatives;
* ``ops_error``       the sticky device flags of these calls.

As in ``nanospec``, this module only checks and marshals arguments; everything
is computed in the library's kernels, asynchronously on ``stream`` (the current
stream when it is None).  Outputs and workspaces come from torch's caching
allocator unless they are passed in.  Inputs used on a stream other than the
one they were made on must be ordered by the caller, as with any torch op.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from .nanospec import _check, load_library

FLAG_NO_PAGES = 0x10
FLAG_BAD_SEQ = 0x20
FLAG_SHARED_PAGE = 0x40
MAX_NEW = 64
MAX_ATTEND_SEQS = 4096
MAX_ALTERNATIVES = 32
MAX_PAGE_SEQS = 8192

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class ns_kv_pages(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v")] +
                [(f"{t}_{n}", ctypes.c_int64) for t in "kv" for n in ("layer", "page", "head", "token")] +
                [(n, ctypes.c_int32) for n in ("layers", "pages", "heads", "page_size", "row_bytes", "max_seqs",
                                               "table_ld")] +
                [(n, ctypes.c_void_p) for n in ("table", "lengths", "refs")])


def _need(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _on_device(what: str, t: torch.Tensor, device: torch.device) -> None:
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, not {t.device}")


def _device(t: torch.Tensor, what: str) -> torch.device:
    d = t.device
    if d.type != "cuda" or d.index != torch.cuda.current_device():
        raise ValueError(f"{what} must be on the current CUDA device, not {d}")
    return d


def _i32(what: str, t: torch.Tensor, device: torch.device, *shape) -> int:
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor on {device}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {shape}")
    return t.data_ptr()


def _rows(what: str, t: torch.Tensor, device: torch.device, dtype: torch.dtype) -> None:
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what} must be {dtype} on {device}, not {t.dtype} on {t.device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must have consecutive elements in its last dimension")


def _stream(stream, device, *made) -> int:
    """The stream's handle; tensors made here and used on another stream are recorded there."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.cuda_stream != torch.cuda.current_stream(device).cuda_stream:
        for t in made:
            t.record_stream(stream)
    return stream.cuda_stream


def _output(what: str, t: Optional[torch.Tensor], shape, dtype, device, made: list) -> torch.Tensor:
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        made.append(t)
    elif t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, max_len: int, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention over packed prompts: q [T, Hq, D], k and v [T, Hkv, D] (bf16 or fp16, D 64 or 128; token
    and head strides are free multiples of 8 elements), cu int32 [B + 1] the sequences' bounds, max_len the
    longest.  Returns (out [T, Hq, D], lse fp32 [T, Hq]).  scale: 1 / sqrt(D) by default."""
    lib = load_library()
    dev = _device(q, "q")
    _need(q.dtype in (torch.bfloat16, torch.float16), "q must be bf16 or fp16")
    _need(q.dim() == 3 and k.dim() == 3 and v.dim() == 3, "q, k and v must be [tokens, heads, dim]")
    T, hq, d = q.shape
    hkv = k.shape[1]
    _need(tuple(k.shape) == (T, hkv, d) and k.shape == v.shape, "k and v must be [tokens, kv_heads, dim]")
    _need(hkv > 0 and hq % hkv == 0, "q_heads must be a multiple of kv_heads")
    for what, t in (("q", q), ("k", k), ("v", v)):
        _rows(what, t, dev, q.dtype)
    cu_ptr = _i32("cu", cu, dev, None)
    _need(cu.shape[0] >= 1, "cu must have one more entry than there are sequences")
    made = []
    out = _output("out", out, (T, hq, d), q.dtype, dev, made)
    lse = _output("lse", lse, (T, hq), torch.float32, dev, made)
    _check(lib.ns_attend_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPES[q.dtype], T, hq, hkv, d,
                                q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), cu_ptr,
                                cu.shape[0] - 1, max_len, d ** -0.5 if scale is None else scale, out.data_ptr(),
                                lse.data_ptr(), _stream(stream, dev, *made)), "ns_attend_prompt")
    return out, lse


def attend_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                 lengths: torch.Tensor, seqs: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, max_len: int = 0, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of n new tokens per sequence over one layer of a paged cache: q [B, n, Hq, D]; k_pages and
    v_pages [pages, Hkv, page_size, D] (strides free); table int32 [max_seqs, pages per sequence], lengths int32
    [max_seqs] (the new tokens included), seqs int32 [B] the cache sequences; mask int64 [B, n]: bit j of word i
    set where new token i sees new token j (None: j <= i).  max_len, a bound on the lengths, only sizes the
    launch.  Returns (out [B, n, Hq, D], lse fp32 [B, n, Hq])."""
    lib = load_library()
    dev = _device(q, "q")
    _need(q.dtype in (torch.bfloat16, torch.float16), "q must be bf16 or fp16")
    _need(q.dim() == 4 and k_pages.dim() == 4, "q must be [B, n, heads, dim], the cache [pages, heads, page_size, dim]")
    B, n, hq, d = q.shape
    pages, hkv, page, _ = k_pages.shape
    _need(k_pages.shape[3] == d and k_pages.shape == v_pages.shape, "k_pages and v_pages must have q's dim")
    _need(hkv > 0 and hq % hkv == 0, "q_heads must be a multiple of kv_heads")
    _need(1 <= n <= MAX_NEW and B <= MAX_ATTEND_SEQS, f"at most {MAX_NEW} new tokens and {MAX_ATTEND_SEQS} sequences")
    for what, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages)):
        _rows(what, t, dev, q.dtype)
    t_ptr, l_ptr = _i32("table", table, dev, None, None), _i32("lengths", lengths, dev, table.shape[0])
    s_ptr = _i32("seqs", seqs, dev, B)
    if mask is not None:
        _need(mask.dtype == torch.int64 and mask.is_contiguous() and tuple(mask.shape) == (B, n) and
              mask.device == dev, f"mask must be a contiguous int64 tensor of shape {(B, n)} on {dev}")
    made = []
    out = _output("out", out, (B, n, hq, d), q.dtype, dev, made)
    lse = _output("lse", lse, (B, n, hq), torch.float32, dev, made)
    need = lib.ns_attend_paged_workspace(B, n, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        made.append(workspace)
    else:
        _on_device("workspace", workspace, dev)
        _need(workspace.is_contiguous(), "workspace must be contiguous")
    _check(lib.ns_attend_paged(q.data_ptr(), _DTYPES[q.dtype], B, n, hq, hkv, d, q.stride(0), q.stride(1),
                               q.stride(2), k_pages.data_ptr(), v_pages.data_ptr(), pages, page, k_pages.stride(0),
                               k_pages.stride(1), k_pages.stride(2), v_pages.stride(0), v_pages.stride(1),
                               v_pages.stride(2), t_ptr, table.shape[1], table.shape[0], l_ptr, s_ptr,
                               None if mask is None else mask.data_ptr(), d ** -0.5 if scale is None else scale,
                               max_len, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(stream, dev, *made)),
           "ns_attend_paged")
    return out, lse


class KvPages:
    """A paged key-value cache over the caller's tensors: k and v [layers, pages, heads, page_size, dim] (any element
    type; rows of dim consecutive elements, a multiple of 16 bytes; other strides free), table int32 [max_seqs,
    pages per sequence] (-1 past a sequence's last page), lengths int32 [max_seqs], refs int32 [pages] (how many
    sequences hold a page).  ``KvPages.new`` makes an empty one."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                 refs: torch.Tensor):
        self._lib = load_library()
        self.device = dev = _device(k, "k")
        _need(k.dim() == 5 and k.shape == v.shape, "k and v must be [layers, pages, heads, page_size, dim]")
        _need(k.dtype == v.dtype, "k and v must have one type")
        _rows("k", k, dev, k.dtype)
        _rows("v", v, dev, v.dtype)
        self.k, self.v, self.table, self.lengths, self.refs = k, v, table, lengths, refs
        e = k.element_size()
        L, pages, heads, page, d = k.shape
        s, t = k.stride(), v.stride()
        c = ns_kv_pages()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.k_layer, c.k_page, c.k_head, c.k_token = s[0] * e, s[1] * e, s[2] * e, s[3] * e
        c.v_layer, c.v_page, c.v_head, c.v_token = t[0] * e, t[1] * e, t[2] * e, t[3] * e
        c.layers, c.pages, c.heads, c.page_size, c.row_bytes = L, pages, heads, page, d * e
        c.table = _i32("table", table, dev, None, None)
        c.max_seqs, c.table_ld = table.shape
        c.lengths = _i32("lengths", lengths, dev, c.max_seqs)
        c.refs = _i32("refs", refs, dev, pages)
        self._c = c
        self._p = ctypes.byref(c)

    @classmethod
    def new(cls, layers: int, pages: int, kv_heads: int, page_size: int, dim: int, max_seqs: int, max_pages: int,
            dtype=torch.bfloat16, device=None) -> "KvPages":
        """An empty cache of `pages` pages for up to max_seqs sequences of up to max_pages pages each."""
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        k = torch.empty((layers, pages, kv_heads, page_size, dim), dtype=dtype, device=device)
        i32 = {"dtype": torch.int32, "device": device}
        return cls(k, torch.empty_like(k), torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(pages, **i32))

    def truncate(self, seqs: torch.Tensor, new_len: Optional[torch.Tensor] = None, stream=None) -> None:
        """Shortens sequences to new_len [n] positions (None: frees them)."""
        n = seqs.shape[0]
        _check(self._lib.ns_pages_truncate(self._p, _i32("seqs", seqs, self.device, n),
                                           None if new_len is None else _i32("new_len", new_len, self.device, n), n,
                                           _stream(stream, self.device)), "ns_pages_truncate")

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """The empty sequences dst [n] come to hold the pages of src [n]."""
        n = src.shape[0]
        _check(self._lib.ns_pages_fork(self._p, _i32("src", src, self.device, n), _i32("dst", dst, self.device, n), n,
                                       _stream(stream, self.device)), "ns_pages_fork")

    def extend(self, seqs: torch.Tensor, n_new: torch.Tensor, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """Lengthens sequences by n_new [n] positions; a partly filled last page that others hold too is copied."""
        n = seqs.shape[0]
        ps, pn = _i32("seqs", seqs, self.device, n), _i32("n_new", n_new, self.device, n)
        made = []
        if workspace is None:
            need = self._lib.ns_pages_workspace(self._p, n)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=self.device)
            made.append(workspace)
        else:
            _on_device("workspace", workspace, self.device)
            _need(workspace.is_contiguous(), "workspace must be contiguous")
        _check(self._lib.ns_pages_extend(self._p, ps, pn, n, workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream, self.device, *made)), "ns_pages_extend")

    def write(self, layer: int, seqs: torch.Tensor, cu: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
              stream=None) -> None:
        """Writes k_new and v_new [tokens, heads, dim] as the last positions of the sequences in one layer; tokens
        cu[i] .. cu[i + 1] - 1 are sequence seqs[i]'s (cu int32 [n + 1])."""
        n = seqs.shape[0]
        T = k_new.shape[0]
        want = (T, self.k.shape[2], self.k.shape[4])
        for what, t in (("k_new", k_new), ("v_new", v_new)):
            _rows(what, t, self.device, self.k.dtype)
            _need(tuple(t.shape) == want, f"{what} must be [tokens, heads, dim] = {want}")
        e = k_new.element_size()
        _check(self._lib.ns_pages_write(self._p, layer, _i32("seqs", seqs, self.device, n),
                                        _i32("cu", cu, self.device, n + 1), n, k_new.data_ptr(), v_new.data_ptr(),
                                        k_new.stride(0) * e, k_new.stride(1) * e, v_new.stride(0) * e,
                                        v_new.stride(1) * e, T, _stream(stream, self.device)), "ns_pages_write")

    def compact(self, seqs: torch.Tensor, base: torch.Tensor, keep: torch.Tensor, n_keep: torch.Tensor,
                stream=None) -> None:
        """From position base [n] on, keeps the positions base + keep [n, m] (the first n_keep [n] of each row,
        strictly increasing) in every layer, and drops the rest."""
        n = seqs.shape[0]
        _check(self._lib.ns_pages_compact(self._p, _i32("seqs", seqs, self.device, n),
                                          _i32("base", base, self.device, n), _i32("keep", keep, self.device, n, None),
                                          keep.shape[1], _i32("n_keep", n_keep, self.device, n), n,
                                          _stream(stream, self.device)), "ns_pages_compact")

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies pages src [n] onto pages dst [n] in every layer."""
        n = src.shape[0]
        _check(self._lib.ns_pages_copy(self._p, _i32("src", src, self.device, n), _i32("dst", dst, self.device, n), n,
                                       _stream(stream, self.device)), "ns_pages_copy")

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
    lib = load_library()
    dev = _device(logits, "logits")
    _need(logits.dtype in _DTYPES and logits.dim() == 2, "logits must be [rows, V] of fp32, bf16 or fp16")
    _rows("logits", logits, dev, logits.dtype)
    _need(0 <= k <= MAX_ALTERNATIVES, f"k must be from 0 to {MAX_ALTERNATIVES}")
    rows, V = logits.shape
    m = 0 if ids is None else ids.shape[-1]
    ids_ptr = None if ids is None else _i32("ids", ids, dev, rows, None)
    ld = logits.stride(0) if rows > 1 else max(logits.stride(0), V)
    f32 = {"dtype": torch.float32, "device": dev}
    r = TokenLogprobs(torch.empty((rows, m), **f32), torch.empty(rows, **f32), torch.empty(rows, **f32),
                      torch.empty((rows, k), dtype=torch.int32, device=dev), torch.empty((rows, k), **f32))
    _check(lib.ns_token_logprobs(logits.data_ptr(), _DTYPES[logits.dtype], rows, V, ld, temperature, ids_ptr, m, k,
                                 r.logprobs.data_ptr(), r.entropy.data_ptr(), r.lse.data_ptr(), r.top_ids.data_ptr(),
                                 r.top_logprobs.data_ptr(), _stream(stream, dev, *r)), "ns_token_logprobs")
    return r


def ops_error(clear: bool = False) -> int:
    """The sticky NS_FLAG_* mask of these calls on the current device (synchronises it)."""
    f = ctypes.c_uint32()
    _check(load_library().ns_ops_get_error(ctypes.byref(f), int(clear)), "ns_ops_get_error")
    return int(f.value)
