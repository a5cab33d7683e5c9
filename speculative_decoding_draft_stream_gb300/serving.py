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


# Every call's host time is part of its latency (a kernel here may take less
# than its launch), so the checks below are plain comparisons on the path that
# passes, and messages are only made when one fails.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream

_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_empty = torch.empty


def _device(t: torch.Tensor, what: str) -> torch.device:
    d = t.device
    if d.type != "cuda" or d.index != torch.cuda.current_device():
        raise ValueError(f"{what} must be on the current CUDA device, not {d}")
    return d


def _i32(what: str, t: torch.Tensor, device: torch.device, shape) -> int:
    if t.dtype is not _I32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor on {device}")
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _i32_2d(what: str, t: torch.Tensor, device: torch.device) -> int:
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    return _i32(what, t, device, t.shape)


def _rows(what: str, t: torch.Tensor, device: torch.device, dtype: torch.dtype):
    """The strides of a tensor whose last dimension has consecutive elements."""
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what} must be {dtype} on {device}, not {t.dtype} on {t.device}")
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must have consecutive elements in its last dimension")
    return st


def _stream(stream, device, *made) -> int:
    """The stream's handle; tensors made here and used on another stream are recorded there."""
    now = _raw_stream(device.index)
    if stream is None:
        return now
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.cuda_stream != now:
        for t in made:
            t.record_stream(stream)
    return stream.cuda_stream


def _given(what: str, t: torch.Tensor, shape, dtype, device) -> None:
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _workspace(workspace: Optional[torch.Tensor], need: int, device, made: list):
    """The workspace (made here when it is None), its address and size."""
    if workspace is None:
        workspace = _empty(need if need > 16 else 16, dtype=_U8, device=device)
        made.append(workspace)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, max_len: int, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention over packed prompts: q [T, Hq, D], k and v [T, Hkv, D] (bf16 or fp16, D 64 or 128; token
    and head strides are free multiples of 8 elements), cu int32 [B + 1] the sequences' bounds, max_len the
    longest.  Returns (out [T, Hq, D], lse fp32 [T, Hq]).  scale: 1 / sqrt(D) by default."""
    lib = load_library()
    dev = _device(q, "q")
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("q must be bf16 or fp16")
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, dim]")
    T, hq, d = q.shape
    ks = k.shape
    hkv = ks[1]
    if ks[0] != T or ks[2] != d or v.shape != ks:
        raise ValueError("k and v must be [tokens, kv_heads, dim]")
    if hkv == 0 or hq % hkv:
        raise ValueError("q_heads must be a multiple of kv_heads")
    qst, kst, vst = _rows("q", q, dev, dtype), _rows("k", k, dev, dtype), _rows("v", v, dev, dtype)
    n = cu.shape[0] if cu.dim() == 1 else 0
    cu_ptr = _i32("cu", cu, dev, (n,))
    if n < 1:
        raise ValueError("cu must have one more entry than there are sequences")
    made = []
    if out is None:
        out = _empty((T, hq, d), dtype=dtype, device=dev)
        made.append(out)
    else:
        _given("out", out, (T, hq, d), dtype, dev)
    if lse is None:
        lse = _empty((T, hq), dtype=_F32, device=dev)
        made.append(lse)
    else:
        _given("lse", lse, (T, hq), _F32, dev)
    _check(lib.ns_attend_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPES[dtype], T, hq, hkv, d, qst[0],
                                qst[1], kst[0], kst[1], vst[0], vst[1], cu_ptr, n - 1, max_len,
                                d ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(),
                                _stream(stream, dev, *made)), "ns_attend_prompt")
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
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("q must be bf16 or fp16")
    if q.dim() != 4 or k_pages.dim() != 4:
        raise ValueError("q must be [B, n, heads, dim], the cache [pages, heads, page_size, dim]")
    B, n, hq, d = shape = q.shape
    ks = k_pages.shape
    pages, hkv, page, kd = ks
    if kd != d or v_pages.shape != ks:
        raise ValueError("k_pages and v_pages must have q's dim")
    if hkv == 0 or hq % hkv:
        raise ValueError("q_heads must be a multiple of kv_heads")
    if not (1 <= n <= MAX_NEW and B <= MAX_ATTEND_SEQS):
        raise ValueError(f"at most {MAX_NEW} new tokens and {MAX_ATTEND_SEQS} sequences")
    qst = _rows("q", q, dev, dtype)
    kst, vst = _rows("k_pages", k_pages, dev, dtype), _rows("v_pages", v_pages, dev, dtype)
    t_ptr = _i32_2d("table", table, dev)
    rows, ld = table.shape
    l_ptr, s_ptr = _i32("lengths", lengths, dev, (rows,)), _i32("seqs", seqs, dev, (B,))
    if mask is not None:
        _given("mask", mask, (B, n), torch.int64, dev)
    made = []
    if out is None:
        out = _empty(shape, dtype=dtype, device=dev)
        made.append(out)
    else:
        _given("out", out, shape, dtype, dev)
    if lse is None:
        lse = _empty((B, n, hq), dtype=_F32, device=dev)
        made.append(lse)
    else:
        _given("lse", lse, (B, n, hq), _F32, dev)
    ws, ws_bytes = _workspace(workspace, lib.ns_attend_paged_workspace(B, n, hq, hkv, d), dev, made)
    _check(lib.ns_attend_paged(q.data_ptr(), _DTYPES[dtype], B, n, hq, hkv, d, qst[0], qst[1], qst[2],
                               k_pages.data_ptr(), v_pages.data_ptr(), pages, page, kst[0], kst[1], kst[2], vst[0],
                               vst[1], vst[2], t_ptr, ld, rows, l_ptr, s_ptr,
                               None if mask is None else mask.data_ptr(), d ** -0.5 if scale is None else scale,
                               max_len, out.data_ptr(), lse.data_ptr(), ws, ws_bytes, _stream(stream, dev, *made)),
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
        shape, dtype = k.shape, k.dtype
        if len(shape) != 5 or v.shape != shape:
            raise ValueError("k and v must be [layers, pages, heads, page_size, dim]")
        s, t = _rows("k", k, dev, dtype), _rows("v", v, dev, dtype)
        self.k, self.v, self.table, self.lengths, self.refs = k, v, table, lengths, refs
        e = k.element_size()
        L, pages, heads, page, d = shape
        t_ptr = _i32_2d("table", table, dev)
        rows, ld = table.shape
        self._c = ns_kv_pages(k.data_ptr(), v.data_ptr(), s[0] * e, s[1] * e, s[2] * e, s[3] * e, t[0] * e, t[1] * e,
                              t[2] * e, t[3] * e, L, pages, heads, page, d * e, rows, ld, t_ptr,
                              _i32("lengths", lengths, dev, (rows,)), _i32("refs", refs, dev, (pages,)))
        self._p = ctypes.byref(self._c)

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
        dev, n = self.device, (len(seqs),)
        _check(self._lib.ns_pages_truncate(self._p, _i32("seqs", seqs, dev, n),
                                           None if new_len is None else _i32("new_len", new_len, dev, n), n[0],
                                           _stream(stream, dev)), "ns_pages_truncate")

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """The empty sequences dst [n] come to hold the pages of src [n]."""
        dev, n = self.device, (len(src),)
        _check(self._lib.ns_pages_fork(self._p, _i32("src", src, dev, n), _i32("dst", dst, dev, n), n[0],
                                       _stream(stream, dev)), "ns_pages_fork")

    def extend(self, seqs: torch.Tensor, n_new: torch.Tensor, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """Lengthens sequences by n_new [n] positions; a partly filled last page that others hold too is copied."""
        dev, n = self.device, (len(seqs),)
        ps, pn = _i32("seqs", seqs, dev, n), _i32("n_new", n_new, dev, n)
        made = []
        ws, ws_bytes = _workspace(workspace, self._lib.ns_pages_workspace(self._p, n[0]), dev, made)
        _check(self._lib.ns_pages_extend(self._p, ps, pn, n[0], ws, ws_bytes, _stream(stream, dev, *made)),
               "ns_pages_extend")

    def write(self, layer: int, seqs: torch.Tensor, cu: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
              stream=None) -> None:
        """Writes k_new and v_new [tokens, heads, dim] as the last positions of the sequences in one layer; tokens
        cu[i] .. cu[i + 1] - 1 are sequence seqs[i]'s (cu int32 [n + 1])."""
        dev, n, c = self.device, len(seqs), self._c
        kst, vst = _rows("k_new", k_new, dev, self.k.dtype), _rows("v_new", v_new, dev, self.k.dtype)
        e = k_new.element_size()
        T, heads, dim = k_new.shape if k_new.dim() == 3 else (0, 0, 0)
        if heads != c.heads or dim * e != c.row_bytes or v_new.shape != k_new.shape:
            raise ValueError(f"k_new and v_new must be [tokens, {c.heads}, {c.row_bytes // e}]")
        _check(self._lib.ns_pages_write(self._p, layer, _i32("seqs", seqs, dev, (n,)), _i32("cu", cu, dev, (n + 1,)), n,
                                        k_new.data_ptr(), v_new.data_ptr(), kst[0] * e, kst[1] * e, vst[0] * e,
                                        vst[1] * e, T, _stream(stream, dev)), "ns_pages_write")

    def compact(self, seqs: torch.Tensor, base: torch.Tensor, keep: torch.Tensor, n_keep: torch.Tensor,
                stream=None) -> None:
        """From position base [n] on, keeps the positions base + keep [n, m] (the first n_keep [n] of each row,
        strictly increasing) in every layer, and drops the rest."""
        dev, n = self.device, (len(seqs),)
        k_ptr = _i32_2d("keep", keep, dev)
        if keep.shape[0] != n[0]:
            raise ValueError(f"keep has shape {tuple(keep.shape)}, expected ({n[0]}, any)")
        _check(self._lib.ns_pages_compact(self._p, _i32("seqs", seqs, dev, n), _i32("base", base, dev, n), k_ptr,
                                          keep.shape[1], _i32("n_keep", n_keep, dev, n), n[0], _stream(stream, dev)),
               "ns_pages_compact")

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Copies pages src [n] onto pages dst [n] in every layer."""
        dev, n = self.device, (len(src),)
        _check(self._lib.ns_pages_copy(self._p, _i32("src", src, dev, n), _i32("dst", dst, dev, n), n[0],
                                       _stream(stream, dev)), "ns_pages_copy")

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
    code = _DTYPES.get(logits.dtype)
    if code is None or logits.dim() != 2:
        raise ValueError("logits must be [rows, V] of fp32, bf16 or fp16")
    st = _rows("logits", logits, dev, logits.dtype)
    if not 0 <= k <= MAX_ALTERNATIVES:
        raise ValueError(f"k must be from 0 to {MAX_ALTERNATIVES}")
    rows, V = logits.shape
    m, ids_ptr = 0, None
    if ids is not None:
        ids_ptr = _i32_2d("ids", ids, dev)
        if ids.shape[0] != rows:
            raise ValueError(f"ids has shape {tuple(ids.shape)}, expected ({rows}, any)")
        m = ids.shape[1]
    lp, ent = _empty((rows, m), dtype=_F32, device=dev), _empty(rows, dtype=_F32, device=dev)
    lse, tid = _empty(rows, dtype=_F32, device=dev), _empty((rows, k), dtype=_I32, device=dev)
    tlp = _empty((rows, k), dtype=_F32, device=dev)
    _check(lib.ns_token_logprobs(logits.data_ptr(), code, rows, V, st[0] if rows > 1 else max(st[0], V), temperature,
                                 ids_ptr, m, k, lp.data_ptr(), ent.data_ptr(), lse.data_ptr(), tid.data_ptr(),
                                 tlp.data_ptr(), _stream(stream, dev, lp, ent, lse, tid, tlp)), "ns_token_logprobs")
    return TokenLogprobs(lp, ent, lse, tid, tlp)


def ops_error(clear: bool = False) -> int:
    """The sticky NS_FLAG_* mask of these calls on the current device (synchronises it)."""
    f = ctypes.c_uint32()
    _check(load_library().ns_ops_get_error(ctypes.byref(f), int(clear)), "ns_ops_get_error")
    return int(f.value)
