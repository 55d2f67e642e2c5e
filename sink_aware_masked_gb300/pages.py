"""The rollout side in the trainer's precision: pages of bf16 keys and values, and attention over them.

As in ``rollout``, this is argument marshalling only: every step runs in the
CUDA kernels of libsinkattn.so (the contracts are in include/sinkattn.h).
Calls are asynchronous on the current stream of the tensors' device and
allocate nothing but outputs that are not passed in, so a step can be captured
into a CUDA graph.

One rollout step of B sequences, each with its last token and some drafts
behind it::

    live, cu, slot_map, positions = kv_plan(pages, slots, new, total, drop=rejected)
    kv_write(pages, slot_map, k, v)                      # k, v [total, Hkv, 64] bf16
    o, lse = kv_decode_fwd(pages, live, q, sink, q_per_seq=most, cu_rows=cu, workspace=ws)
    ...
    tokens, logp, accepted, rejected = verify_tokens(logits, drafts, u, cu, draft_logits=..., live=live)

A request that found no page (live -1) has its rows in cu all the same, but not
in the pages; with ``live`` the verification rejects nothing of it, and the slot
keeps what it holds until a later plan serves it.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .api import HEAD_DIM, WINDOW_INF, _check, _on_gpu, _ptr
from .rollout import _SCALE, _call, _output, _tensor, _vector


class KVPages:
    """One layer's keys and values of up to ``num_slots`` sequences in bf16 pages.

    k_pages and v_pages bf16 [num_pages, page_size, Hkv, 64], block_table int32
    [num_slots, max_pages], seqlens int32 [num_slots], owner int32 [num_pages]
    (the slot that holds a page, -1 where it is free).  The tensors are kept and
    worked on in place; ``empty`` makes those of new pages.  Layers whose slots
    grow alike can share one table: a KVPages each with pages of its own and the
    same block_table, seqlens and owner, and one ``kv_plan`` for all.
    Calls that change pages follow one another, and the calls that read them, on
    one stream or by events.
    """

    _FIXED = frozenset(("k_pages", "v_pages", "block_table", "seqlens", "owner", "device", "num_pages", "num_heads_kv",
                        "page_size", "num_slots", "max_pages"))

    def __setattr__(self, name, value):
        # The library holds the tensors' addresses: another tensor in their place would not be seen, and the one
        # that is used would be freed.
        if name in self._FIXED and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} of a KVPages cannot be replaced: write into the tensor it was made with")
        super().__setattr__(name, value)

    def __init__(self, k_pages, v_pages, block_table, seqlens, owner):
        dev = k_pages.device if isinstance(k_pages, torch.Tensor) else None
        _check("k_pages", k_pages, torch.bfloat16, (None, None, None, HEAD_DIM), dev)
        num_pages, page_size, heads = (int(x) for x in k_pages.shape[:3])
        _check("v_pages", v_pages, torch.bfloat16, tuple(k_pages.shape), dev)
        _check("block_table", block_table, torch.int32, (None, None), dev)
        _check("seqlens", seqlens, torch.int32, (block_table.shape[0],), dev)
        _check("owner", owner, torch.int32, (num_pages,), dev)
        _on_gpu("k_pages", k_pages)
        self.k_pages, self.v_pages = k_pages, v_pages
        self.block_table, self.seqlens, self.owner = block_table, seqlens, owner
        self.device = k_pages.device
        self.num_pages, self.page_size, self.num_heads_kv = num_pages, page_size, heads
        self.num_slots, self.max_pages = (int(x) for x in block_table.shape)
        self._struct = _lib.KvPages(
            k_pages=_ptr(k_pages), v_pages=_ptr(v_pages), block_table=_ptr(block_table), seqlens=_ptr(seqlens),
            owner=_ptr(owner), num_pages=num_pages, page_size=page_size, num_heads_kv=heads, num_slots=self.num_slots,
            max_pages=self.max_pages)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, num_pages: int, num_slots: int, max_pages: int, num_heads_kv: int, *, page_size: int = 64,
              device="cuda") -> "KVPages":
        """Pages that are free, of slots that are empty."""
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError(f"page_size must be 16, 32, 64, 128 or 256, not {page_size}")
        i32, shape = dict(dtype=torch.int32, device=device), (num_pages, page_size, num_heads_kv, HEAD_DIM)
        return cls(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                   torch.zeros(shape, dtype=torch.bfloat16, device=device), torch.full((num_slots, max_pages), -1, **i32),
                   torch.zeros(num_slots, **i32), torch.full((num_pages,), -1, **i32))


def kv_plan(pages: KVPages, slots, new_tokens, total: int, *, drop=None, live=None, cu=None, slot_map=None,
            positions=None):
    """Slot slots[i] drops its last drop[i] tokens and gets new_tokens[i] new ones (int32 [n], on the device).

    Returns (live int32 [n], cu int32 [n + 1], slot_map int32 [total],
    positions int32 [total]): the slot, or -1 where a request was not served;
    the offsets of the requests' rows; each row's place in the pages and its
    position in the sequence, -1 behind the last row and where a request was
    not served.  ``total`` is at least the number of new tokens (more: a padded
    batch).  A slot that drops all it has is freed.
    """
    dev, i32, total = pages.device, torch.int32, int(total)
    if total < 0:
        raise ValueError(f"total must not be negative ({total})")
    n = _vector("slots", slots, i32, dev)
    sp, np_ = _tensor("slots", slots, i32, (n,), dev), _tensor("new_tokens", new_tokens, i32, (n,), dev)
    dp = None if drop is None else _tensor("drop", drop, i32, (n,), dev)
    live, lp = _output("live", live, slots, i32, (n,), dev)
    cu = torch.empty(n + 1, dtype=i32, device=dev) if cu is None else cu
    slot_map = torch.empty(total, dtype=i32, device=dev) if slot_map is None else slot_map
    cp, mp = _tensor("cu", cu, i32, (n + 1,), dev), _tensor("slot_map", slot_map, i32, (total,), dev)
    positions, pp = _output("positions", positions, slot_map, i32, (total,), dev)
    _call("sinkattn_kv_plan", dev, pages._ref, sp, dp, np_, n, lp, cp, mp, pp, total)
    return live, cu, slot_map, positions


def _rows(name: str, t, rows: int, heads: int, dev):
    """The address and row stride of a bf16 [rows, heads, 64] tensor whose rows are contiguous each."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 3 and t.dtype is torch.bfloat16 and t.device == dev
            and t.shape == (rows, heads, HEAD_DIM)):
        _check(name, t, torch.bfloat16, (rows, heads, HEAD_DIM), dev)
    stride = t.stride(0) if rows > 1 else heads * HEAD_DIM
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != HEAD_DIM) or stride < heads * HEAD_DIM:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), stride


def kv_write(pages: KVPages, slot_map, k, v) -> None:
    """Writes rows of k and v (bf16 [T, Hkv, 64]) to places slot_map (int32 [T], from ``kv_plan``); -1 is skipped.

    The rows may lie apart, as views of a fused projection do (a stride of a
    multiple of 8 values).
    """
    dev = pages.device
    T = _vector("slot_map", slot_map, torch.int32, dev)
    mp = _tensor("slot_map", slot_map, torch.int32, (T,), dev)
    kp, ks = _rows("k", k, T, pages.num_heads_kv, dev)
    vp, vs = _rows("v", v, T, pages.num_heads_kv, dev)
    _call("sinkattn_kv_write", dev, pages._ref, mp, T, kp, ks, vp, vs)


def kv_decode_workspace(pages: KVPages) -> torch.Tensor:
    """A zero-filled workspace for kv_decode_fwd over these pages, of any shape."""
    with torch.cuda.device(pages.device):  # the size goes by that device's number of SMs
        size = int(_lib.load().sinkattn_kv_decode_workspace_size(pages.num_heads_kv))
    if size == 0:
        raise ValueError(f"kv_decode_workspace: no workspace for {pages.num_heads_kv} kv heads")
    return torch.zeros(size, dtype=torch.uint8, device=pages.device)


def kv_decode_fwd(pages: KVPages, slots, q, sink, *, q_per_seq: int, cu_rows=None, window: int = WINDOW_INF,
                  prefix: int = 0, scale: Optional[float] = None, o=None, lse=None, workspace=None):
    """Decode forward over the pages: returns (o, lse) for the last positions of each slot.

    q, o [rows, Hq, 64] bf16, sink [Hq] fp32, lse [Hq, rows] fp32; mask, sink
    and lse as in sinkattn_decode_fwd.  Entry b has rows cu_rows[b] ..
    cu_rows[b + 1] - 1 (int32 [len(slots) + 1], on the device; at most q_per_seq
    each), or without cu_rows q_per_seq rows each.  The new positions' keys and
    values are in the pages already.  Rows of idle slots and rows before a
    sequence's begin get o = 0 and lse = -inf; rows outside every entry's are
    left as they were.  A workspace (kv_decode_workspace) can be kept for calls
    that follow one another, of any shape; without one a zero-filled one is made
    per call.
    """
    dev = pages.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D tensor [rows, heads, head_dim]")
    rows, hq, d = q.shape
    if d != HEAD_DIM:
        raise ValueError(f"head_dim must be {HEAD_DIM} (q: {d})")
    if hq % pages.num_heads_kv != 0 or hq == 0:
        raise ValueError(f"query heads ({hq}) must be a multiple of key/value heads ({pages.num_heads_kv})")
    n = _vector("slots", slots, torch.int32, dev)
    sp = _tensor("slots", slots, torch.int32, (n,), dev)
    q_per_seq, window, prefix = int(q_per_seq), int(window), int(prefix)
    if cu_rows is None:
        rows, cp = n * q_per_seq, None
    else:
        cp = _tensor("cu_rows", cu_rows, torch.int32, (n + 1,), dev)
    shape = (rows, hq, HEAD_DIM)
    qp, kp = _tensor("q", q, torch.bfloat16, shape, dev), _tensor("sink", sink, torch.float32, (hq,), dev)
    o, op = _output("o", o, q, torch.bfloat16, shape, dev)
    if lse is None:
        lse = torch.empty((hq, rows), dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _tensor("lse", lse, torch.float32, (hq, rows), dev)
    if workspace is None:
        workspace = kv_decode_workspace(pages)
    wn = _vector("workspace", workspace, torch.uint8, dev)
    _call("sinkattn_kv_decode_fwd", dev, pages._ref, sp, cp, n, q_per_seq, rows, hq, window, prefix,
          _SCALE if scale is None else scale, qp, kp, op, lp, _tensor("workspace", workspace, torch.uint8, (wn,), dev), wn)
    return o, lse
