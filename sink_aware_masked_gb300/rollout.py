"""The rollout side: a 4-bit paged key/value cache, attention over it, and token sampling.

As in ``api``, this is argument marshalling only: every step runs in the CUDA
kernels of libsinkattn.so (the formats and contracts are in
include/sinkattn.h).  Calls are asynchronous on the current stream of the
tensors' device and allocate nothing but outputs that are not passed in, so a
step can be captured into a CUDA graph.

One rollout step of B sequences::

    done = kv4_reserve(cache, slots, ones)               # room for the new tokens
    kv4_append(cache, slots, k, v)                       # k, v [B, Hkv, 64] bf16
    o, lse = kv4_decode_fwd(cache, slots, q, sink, q_per_seq=1, workspace=ws)
    ...
    tokens, logp, logq = sample_tokens(logits, u, temperature=t, top_p=p)
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _lib
from .api import HEAD_DIM, WINDOW_INF, _check, _on_gpu, _ptr

BLOCK_TOKENS = 16
TOKEN_BYTES = 72  # per token and kv head: 2 x 32 bytes of codes, 2 x 4 scales

_SCALE = 1.0 / math.sqrt(HEAD_DIM)
_LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


# The current device and a device's current stream as plain integers: a small
# step's time is its calls' time on the host, and torch.cuda.current_stream()
# makes a Stream object on the way.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_functions = {}


def _call(name: str, dev: torch.device, *args) -> None:
    """Call the library on ``dev``'s current stream (the last argument of every entry point)."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    index = dev.index
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        _lib.check(name, st)


def _tensor(name: str, t, dtype: torch.dtype, shape, dev) -> int:
    """Checks a tensor as ``api._check`` does, which words the refusal, and returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _check(name, t, dtype, shape, dev)
    return t.data_ptr()


def _output(name: str, t, make, dtype: torch.dtype, shape, dev):
    """A caller's output, checked, or a new one made like ``make``: the tensor and its address."""
    if t is None:
        t = torch.empty_like(make)
        return t, t.data_ptr()
    return t, _tensor(name, t, dtype, shape, dev)


def _vector(name: str, t, dtype: torch.dtype, dev) -> int:
    """The length of a 1-D tensor that is checked like any other."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 1):
        _check(name, t, dtype, (None,), dev)
    return t.shape[0]


class KV4Cache:
    """One layer's keys and values of up to ``num_slots`` sequences in 4 bits, in shared pages.

    pages uint8 [num_pages, Hkv, page_size * 72], page_table int32
    [num_slots, max_pages], seqlens int32 [num_slots], refcount int32
    [num_pages], k_scale and v_scale float32 [Hkv] (2^-100 to 2^100: a value
    is code * e4m3 scale * its head's factor).  The cache keeps these tensors
    and works on them in place; ``empty`` makes the tensors of a new one.
    Calls that change a cache follow one another, and the calls that read it,
    on one stream or by events.
    """

    _FIXED = frozenset(("pages", "page_table", "seqlens", "refcount", "k_scale", "v_scale", "device", "num_pages",
                        "num_heads_kv", "page_size", "num_slots", "max_pages"))

    def __setattr__(self, name, value):
        # The library holds the tensors' addresses: another tensor in their place would not be seen, and the one
        # that is used would be freed.
        if name in self._FIXED and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} of a KV4Cache cannot be replaced: write into the tensor it was made with")
        super().__setattr__(name, value)

    def __init__(self, pages, page_table, seqlens, refcount, k_scale, v_scale):
        dev = pages.device if isinstance(pages, torch.Tensor) else None
        _check("pages", pages, torch.uint8, (None, None, None), dev)
        num_pages, heads, page_bytes = (int(x) for x in pages.shape)
        if page_bytes % (BLOCK_TOKENS * TOKEN_BYTES) != 0:
            raise ValueError(f"pages holds {page_bytes} bytes per page and head, expected a multiple of "
                             f"{BLOCK_TOKENS * TOKEN_BYTES}")
        _check("page_table", page_table, torch.int32, (None, None), dev)
        _check("seqlens", seqlens, torch.int32, (page_table.shape[0],), dev)
        _check("refcount", refcount, torch.int32, (num_pages,), dev)
        _check("k_scale", k_scale, torch.float32, (heads,), dev)
        _check("v_scale", v_scale, torch.float32, (heads,), dev)
        _on_gpu("pages", pages)
        self.pages, self.page_table, self.seqlens, self.refcount = pages, page_table, seqlens, refcount
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device = pages.device
        self.num_pages, self.num_heads_kv = num_pages, heads
        self.page_size = page_bytes // TOKEN_BYTES
        self.num_slots, self.max_pages = (int(x) for x in page_table.shape)
        self._struct = _lib.Kv4Cache(
            pages=_ptr(pages), page_table=_ptr(page_table), seqlens=_ptr(seqlens), refcount=_ptr(refcount),
            k_scale=_ptr(k_scale), v_scale=_ptr(v_scale), num_pages=num_pages, page_size=self.page_size,
            num_heads_kv=heads, num_slots=self.num_slots, max_pages=self.max_pages)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, num_pages: int, num_slots: int, max_pages: int, num_heads_kv: int, *, page_size: int = 64,
              k_scale=None, v_scale=None, device="cuda") -> "KV4Cache":
        """A cache whose slots are empty and whose pages are free (factors 1 unless given)."""
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError(f"page_size must be 16, 32, 64, 128 or 256, not {page_size}")
        one = lambda s: torch.ones(num_heads_kv, dtype=torch.float32, device=device) if s is None else s  # noqa: E731
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((num_pages, num_heads_kv, page_size * TOKEN_BYTES), dtype=torch.uint8, device=device),
                   torch.full((num_slots, max_pages), -1, **i32), torch.zeros(num_slots, **i32),
                   torch.zeros(num_pages, **i32), one(k_scale), one(v_scale))


def kv4_reserve(cache: KV4Cache, slots, new_tokens, *, done=None):
    """Slot slots[i] grows by new_tokens[i] tokens (int32 [n], on the device); returns done int32 [n].

    A request that finds no room gets done = 0 and stays as it was, and so
    does every later one that needs a page.
    """
    dev, i32 = cache.device, torch.int32
    n = _vector("slots", slots, i32, dev)
    sp, np_ = _tensor("slots", slots, i32, (n,), dev), _tensor("new_tokens", new_tokens, i32, (n,), dev)
    done, op = _output("done", done, slots, i32, (n,), dev)
    _call("sinkattn_kv4_reserve", dev, cache._ref, sp, np_, n, op)
    return done


def kv4_fork(cache: KV4Cache, src, dst, *, done=None):
    """The empty slots dst[i] become copies of src[i], sharing its full pages; returns done int32 [n]."""
    dev, i32 = cache.device, torch.int32
    n = _vector("src", src, i32, dev)
    sp, dp = _tensor("src", src, i32, (n,), dev), _tensor("dst", dst, i32, (n,), dev)
    done, op = _output("done", done, src, i32, (n,), dev)
    _call("sinkattn_kv4_fork", dev, cache._ref, sp, dp, n, op)
    return done


def kv4_free(cache: KV4Cache, slots) -> None:
    """Empties the slots; pages that no other slot holds become free."""
    dev = cache.device
    n = _vector("slots", slots, torch.int32, dev)
    _call("sinkattn_kv4_free", dev, cache._ref, _tensor("slots", slots, torch.int32, (n,), dev), n)


def kv4_compact(cache: KV4Cache, to: KV4Cache, *, count=None, workspace=None):
    """Moves the pages in use to the front of another cache's pool; returns their number, int32 [1].

    ``to`` has the same page size, heads, slots and table width and memory of
    its own; if it is too small it is left as it was (compare the count).
    """
    dev = cache.device
    if to.device != dev:
        raise ValueError(f"to is on {to.device}, expected {dev}")
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=dev)
    cp = _tensor("count", count, torch.int32, (1,), dev)
    if workspace is None:
        size = int(_lib.load().sinkattn_kv4_compact_workspace_size(cache._ref))
        workspace = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    wn = _vector("workspace", workspace, torch.uint8, dev)
    _call("sinkattn_kv4_compact", dev, cache._ref, to._ref, cp, _tensor("workspace", workspace, torch.uint8, (wn,), dev),
          wn)
    return count


def kv4_append(cache: KV4Cache, slots, k, v, *, cu_new=None) -> None:
    """Writes k and v (bf16 [T, Hkv, 64]) as the last positions of the slots, in 4 bits.

    Slot slots[b] takes rows cu_new[b] .. cu_new[b + 1] - 1 (int32
    [len(slots) + 1], on the device), or T / len(slots) rows each without
    cu_new; its length counts them already (kv4_reserve).  No slot is named
    twice in a call.
    """
    dev, bf16 = cache.device, torch.bfloat16
    n = _vector("slots", slots, torch.int32, dev)
    sp = _tensor("slots", slots, torch.int32, (n,), dev)
    if not (isinstance(k, torch.Tensor) and k.dim() == 3):
        _check("k", k, bf16, (None, cache.num_heads_kv, HEAD_DIM), dev)
    shape = (k.shape[0], cache.num_heads_kv, HEAD_DIM)
    kp, vp = _tensor("k", k, bf16, shape, dev), _tensor("v", v, bf16, shape, dev)
    cp = None if cu_new is None else _tensor("cu_new", cu_new, torch.int32, (n + 1,), dev)
    _call("sinkattn_kv4_append", dev, cache._ref, sp, n, cp, shape[0], kp, vp)


def kv4_read(cache: KV4Cache, slots, total: int, *, cu=None, k=None, v=None):
    """The last rows of the slots as bf16: returns (k, v) [total, Hkv, 64].

    Slot slots[b] gives rows cu[b] .. cu[b + 1] - 1 (or total / len(slots)
    each): with cu the offsets of whole lengths, the sequences as sinkattn_fwd
    takes them.  Rows before a sequence's begin are zero; rows behind cu[-1]
    are not written.
    """
    dev, bf16 = cache.device, torch.bfloat16
    n = _vector("slots", slots, torch.int32, dev)
    sp = _tensor("slots", slots, torch.int32, (n,), dev)
    shape = (int(total), cache.num_heads_kv, HEAD_DIM)
    cp = None if cu is None else _tensor("cu", cu, torch.int32, (n + 1,), dev)
    k = torch.empty(shape, dtype=bf16, device=dev) if k is None else k
    kp = _tensor("k", k, bf16, shape, dev)
    v, vp = _output("v", v, k, bf16, shape, dev)
    _call("sinkattn_kv4_read", dev, cache._ref, sp, n, cp, shape[0], kp, vp)
    return k, v


def kv4_decode_workspace(cache: KV4Cache, q) -> torch.Tensor:
    """A zero-filled workspace for kv4_decode_fwd with queries shaped like q."""
    with torch.cuda.device(cache.device):  # the size goes by that device's number of SMs
        size = int(_lib.load().sinkattn_kv4_decode_workspace_size(int(q.shape[0]), int(q.shape[1])))
    if size == 0:
        raise ValueError(f"kv4_decode_workspace: no workspace for queries of shape {list(q.shape)}")
    return torch.zeros(size, dtype=torch.uint8, device=cache.device)


def kv4_decode_fwd(cache: KV4Cache, slots, q, sink, *, q_per_seq: int, window: int = WINDOW_INF, prefix: int = 0,
                   scale: Optional[float] = None, o=None, lse=None, workspace=None):
    """Decode forward over the cache: returns (o, lse) for the last q_per_seq positions of each slot.

    q, o [len(slots) * q_per_seq, Hq, 64] bf16, sink [Hq] fp32, lse [Hq, rows]
    fp32; mask, sink and lse as in sinkattn_decode_fwd.  The new positions'
    keys and values are in the cache already.  Rows of idle slots and rows
    before a sequence's begin get o = 0 and lse = -inf.  A workspace
    (kv4_decode_workspace) can be kept for calls that follow one another, of any
    shape it is large enough for; without one a zero-filled one is made per
    call.
    """
    dev = cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D tensor [rows, heads, head_dim]")
    _, hq, d = q.shape
    if d != HEAD_DIM:
        raise ValueError(f"head_dim must be {HEAD_DIM} (q: {d})")
    if hq % cache.num_heads_kv != 0 or hq == 0:
        raise ValueError(f"query heads ({hq}) must be a multiple of key/value heads ({cache.num_heads_kv})")
    n = _vector("slots", slots, torch.int32, dev)
    sp = _tensor("slots", slots, torch.int32, (n,), dev)
    q_per_seq, window, prefix = int(q_per_seq), int(window), int(prefix)
    rows = n * q_per_seq
    shape = (rows, hq, HEAD_DIM)
    qp, kp = _tensor("q", q, torch.bfloat16, shape, dev), _tensor("sink", sink, torch.float32, (hq,), dev)
    o, op = _output("o", o, q, torch.bfloat16, shape, dev)
    if lse is None:
        lse = torch.empty((hq, rows), dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _tensor("lse", lse, torch.float32, (hq, rows), dev)
    if workspace is None:
        workspace = kv4_decode_workspace(cache, q)
    wn = _vector("workspace", workspace, torch.uint8, dev)
    _call("sinkattn_kv4_decode_fwd", dev, cache._ref, sp, n, q_per_seq, hq, window, prefix,
          _SCALE if scale is None else scale, qp, kp, op, lp, _tensor("workspace", workspace, torch.uint8, (wn,), dev), wn)
    return o, lse


def sample_tokens(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logp=None,
                  logq=None):
    """Samples one token per row: returns (tokens int32 [B], logp fp32 [B], logq fp32 [B]).

    logits [B, V] fp32, bf16 or fp16, rows contiguous (any row stride); u fp32
    [B] random numbers in [0, 1); temperature, top_p, min_p fp32 [B] and top_k
    int32 [B] (default 1, off, off and off).  logp is the token's
    log-probability at the temperature over the whole vocabulary (grpo_loss's
    logp_old), logq the one among the kept tokens.  temperature 0 takes the
    largest logit (the lowest index of equal ones).  A row without an allowed
    token gives -1 and -inf, an invalid row -1 and NaN.
    """
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a 2-D tensor [rows, vocab]")
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits has dtype {logits.dtype}, expected float32, bfloat16 or float16")
    B, V = logits.shape
    if (V > 1 and logits.stride(1) != 1) or (B > 1 and logits.stride(0) < V):
        raise ValueError("logits must have contiguous rows that do not overlap")
    dev = logits.device
    f32, i32, one = torch.float32, torch.int32, (B,)
    up = _tensor("u", u, f32, one, dev)
    temperature = torch.ones_like(u) if temperature is None else temperature
    top_k = torch.zeros(B, dtype=i32, device=dev) if top_k is None else top_k
    top_p = torch.ones_like(u) if top_p is None else top_p
    min_p = torch.zeros_like(u) if min_p is None else min_p
    tp, kp = _tensor("temperature", temperature, f32, one, dev), _tensor("top_k", top_k, i32, one, dev)
    pp, mp = _tensor("top_p", top_p, f32, one, dev), _tensor("min_p", min_p, f32, one, dev)
    tokens, to = _output("tokens", tokens, top_k, i32, one, dev)
    logp, lp = _output("logp", logp, u, f32, one, dev)
    logq, lq = _output("logq", logq, u, f32, one, dev)
    _on_gpu("logits", logits)
    _call("sinkattn_sample_tokens", dev, logits.data_ptr(), kind, B, V, logits.stride(0) if B > 1 else V, up, tp, kp, pp,
          mp, to, lp, lq)
    return tokens, logp, logq
