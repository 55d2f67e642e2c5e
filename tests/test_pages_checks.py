"""Rollout with drafted tokens on the CPU: refusals of the C ABI and of the binding, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.pages_ref as ref
from sink_aware_masked_gb300 import _lib, pages, rollout

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails validation first
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from sink_aware_masked_gb300 import build

    build.build()
    return _lib.load()


def pool(**kw):
    base = dict(k_pages=FAKE, v_pages=FAKE, block_table=FAKE, seqlens=FAKE, owner=FAKE, num_pages=8, page_size=64,
                num_heads_kv=2, num_slots=4, max_pages=4)
    base.update(kw)
    return _lib.KvPages(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=0), INVALID), (dict(num_slots=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_heads_kv=0), INVALID), (dict(num_heads_kv=257), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
    (dict(max_pages=(1 << 30) // 64 + 1), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED),
    (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(block_table=None), INVALID),
    (dict(seqlens=None), INVALID), (dict(owner=None), INVALID), (dict(k_pages=FAKE + 8), ALIGNMENT),
    (dict(v_pages=FAKE + 8), ALIGNMENT), (dict(block_table=FAKE + 4), ALIGNMENT), (dict(seqlens=FAKE + 4), ALIGNMENT),
    (dict(owner=FAKE + 4), ALIGNMENT),
])
def test_every_call_refuses_bad_pages(lib, kw, status):
    c, f = ctypes.byref(pool(**kw)), FAKE
    assert lib.sinkattn_kv_plan(c, f, f, f, 1, f, f, f, f, 1, None) == status
    assert lib.sinkattn_kv_write(c, f, 1, f, 128, f, 128, None) == status
    assert lib.sinkattn_kv_decode_fwd(c, f, None, 1, 1, 1, 4, -1, 0, 0.125, f, f, f, f, f, 1 << 30, None) == status
    assert lib.sinkattn_kv_plan(None, f, f, f, 1, f, f, f, f, 1, None) == INVALID


def test_plan_refuses(lib):
    c, f = ctypes.byref(pool()), FAKE

    def call(slots=f, drop=f, new=f, n=2, live=f, cu=f, slot_map=f, positions=f, total=2):
        return lib.sinkattn_kv_plan(c, slots, drop, new, n, live, cu, slot_map, positions, total, None)

    assert call(n=-1) == INVALID and call(n=4097) == UNSUPPORTED and call(total=-1) == INVALID
    for name in ("slots", "new", "live", "cu", "slot_map", "positions"):
        assert call(**{name: None}) == INVALID
    for name in ("slots", "drop", "new", "live", "cu", "slot_map", "positions"):
        assert call(**{name: f + 2}) == ALIGNMENT


def test_write_refuses(lib):
    c, f = ctypes.byref(pool()), FAKE

    def call(slot_map=f, rows=3, k=f, ks=128, v=f, vs=128):
        return lib.sinkattn_kv_write(c, slot_map, rows, k, ks, v, vs, None)

    assert call(rows=-1) == INVALID and call(ks=127) == INVALID and call(vs=64) == INVALID
    assert call(ks=132) == ALIGNMENT and call(vs=1001) == ALIGNMENT
    for name in ("slot_map", "k", "v"):
        assert call(**{name: None}) == INVALID
    assert call(slot_map=f + 2) == ALIGNMENT and call(k=f + 8) == ALIGNMENT and call(v=f + 8) == ALIGNMENT
    assert call(rows=0, k=None, v=None, slot_map=None) == OK


def test_decode_refuses(lib):
    c, f = ctypes.byref(pool()), FAKE
    ws = lib.sinkattn_kv_decode_workspace_size(2)

    def call(n=2, rows_each=1, rows=None, cu=None, hq=4, window=-1, prefix=0, scale=0.125, slots=f, q=f, sink=f, o=f,
             lse=f, w=f, size=ws):
        rows = n * rows_each if rows is None else rows
        return lib.sinkattn_kv_decode_fwd(c, slots, cu, n, rows_each, rows, hq, window, prefix, scale, q, sink, o, lse, w,
                                          size, None)

    assert call(rows_each=0) == INVALID and call(hq=3) == INVALID and call(hq=0) == INVALID and call(n=-1) == INVALID
    assert call(n=4097) == UNSUPPORTED and call(hq=512) == UNSUPPORTED and call(rows_each=65) == UNSUPPORTED
    assert call(window=-2) == INVALID and call(prefix=-1) == INVALID
    assert call(rows=3) == INVALID and call(rows=-1, cu=f) == INVALID and call(cu=f + 2) == ALIGNMENT
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == INVALID
    for name in ("q", "sink", "o", "lse", "w"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: f + 8}) == ALIGNMENT
    assert call(slots=None) == INVALID and call(slots=f + 2) == ALIGNMENT and call(size=ws - 1) == WORKSPACE
    assert call(n=0, slots=None) == OK and call(rows=0, cu=f, q=None, o=None) == OK
    size = lib.sinkattn_kv_decode_workspace_size
    assert size(0) == 0 and size(257) == 0
    # 256 partial rows of 64 accumulators and 4 statistics per SM, and a counter per entry and kv head
    assert size(3) - size(2) == 4096 * 4 and 0 < size(1) <= 152 * 256 * 68 * 4 + 4096 * 4


def test_verify_refuses(lib):
    f = FAKE
    ws = lib.sinkattn_verify_workspace_size(0, 5, 10)
    assert ws == 5 * (2 * 16 + 48 + 16 * 8 * 32)  # a slice of 16 bytes per row and draft row, what an entry stops with, its runs

    def call(x=f, xs=10, y=f, ys=10, dtype=0, rows=5, drafts=3, vocab=10, d=f, cu=f, n=2, u=f, t=f, tokens=f, logp=f, acc=f,
             rej=f, w=f, size=ws):
        return lib.sinkattn_verify_tokens(x, xs, y, ys, dtype, rows, drafts, vocab, d, cu, n, u, t, tokens, logp, acc, rej,
                                          w, size, None)

    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(drafts=-1), dict(drafts=6), dict(vocab=0), dict(xs=9),
               dict(ys=9), dict(n=-1)):
        assert call(**kw) == INVALID
    assert call(vocab=(1 << 18) + 1, xs=1 << 19, ys=1 << 19) == UNSUPPORTED and call(rows=(1 << 20) + 1) == UNSUPPORTED
    assert call(n=4097) == UNSUPPORTED
    for name in ("x", "d", "cu", "u", "t", "tokens", "logp", "acc", "rej", "w"):
        assert call(**{name: None}) == INVALID
    for name in ("x", "y", "d", "cu", "u", "t", "tokens", "logp", "acc", "rej"):
        assert call(**{name: f + 2}) == ALIGNMENT
    assert call(x=f + 1, dtype=1) == ALIGNMENT and call(w=f + 8) == ALIGNMENT and call(size=ws - 1) == WORKSPACE
    assert call(n=0, x=None, cu=None, t=None, acc=None, rej=None) == OK
    size = lib.sinkattn_verify_workspace_size
    assert size(3, 1, 1) == 0 and size(0, -1, 1) == 0 and size(0, 1, 0) == 0 and size(0, 1, (1 << 18) + 1) == 0


# ---------------------------------------------------------------- the binding
def _tensors(P=4, H=2, S=3, M=2, page=16):
    i32 = dict(dtype=torch.int32)
    return dict(k_pages=torch.zeros((P, page, H, 64), dtype=torch.bfloat16),
                v_pages=torch.zeros((P, page, H, 64), dtype=torch.bfloat16), block_table=torch.zeros((S, M), **i32),
                seqlens=torch.zeros(S, **i32), owner=torch.zeros(P, **i32))


@pytest.mark.parametrize("name,make,error,match", [
    ("k_pages", lambda t: t.half(), TypeError, "k_pages has dtype"),
    ("k_pages", lambda t: t[..., :32].contiguous(), ValueError, "k_pages has shape"),
    ("k_pages", lambda t: t.transpose(1, 2), ValueError, "v_pages has shape|contiguous"),
    ("v_pages", lambda t: t[:2], ValueError, "v_pages has shape"),
    ("block_table", lambda t: t.long(), TypeError, "block_table has dtype"),
    ("seqlens", lambda t: t[:2], ValueError, "seqlens has shape"),
    ("owner", lambda t: t[:2], ValueError, "owner has shape"),
    ("owner", lambda t: t, ValueError, "CUDA tensor"),
])
def test_pages_refuse(name, make, error, match):
    t = _tensors()
    t[name] = make(t[name])
    with pytest.raises(error, match=match):
        pages.KVPages(**t)


def test_empty_refuses_page_sizes():
    with pytest.raises(ValueError, match="page_size"):
        pages.KVPages.empty(4, 2, 2, 1, page_size=24)


def test_tensors_of_pages_cannot_be_replaced():
    p = object.__new__(pages.KVPages)
    p.owner = torch.zeros(3, dtype=torch.int32)
    first = p.owner
    p.owner += 1
    with pytest.raises(AttributeError, match="owner of a KVPages cannot be replaced"):
        p.owner = p.owner + 1
    assert p.owner is first


def _fake_pages():
    p = object.__new__(pages.KVPages)
    p.device, p.num_heads_kv = torch.device("cpu"), 2
    return p


def test_write_binding_refuses():
    p, at = _fake_pages(), torch.zeros(3, dtype=torch.int32)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for bad, error, match in ((k.float(), TypeError, "k has dtype"), (k[:2], ValueError, "k has shape"),
                              (k.transpose(1, 2).contiguous().transpose(1, 2), ValueError, "contiguous rows"),
                              (k[:1].expand(3, 2, 64), ValueError, "overlap"),
                              (torch.zeros((3, 2, 128), dtype=torch.bfloat16)[..., ::2], ValueError, "contiguous rows")):
        with pytest.raises(error, match=match):
            pages.kv_write(p, at, bad, k)
    with pytest.raises(TypeError, match="slot_map has dtype"):
        pages.kv_write(p, at.long(), k, k)


def test_plan_and_decode_bindings_refuse():
    p, two = _fake_pages(), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="new_tokens has dtype"):
        pages.kv_plan(p, two, two.long(), 4)
    with pytest.raises(ValueError, match="drop has shape"):
        pages.kv_plan(p, two, two, 4, drop=two[:1])
    with pytest.raises(ValueError, match="slot_map has shape"):
        pages.kv_plan(p, two, two, 4, slot_map=two)
    q, sink = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros(4)
    with pytest.raises(ValueError, match="cu_rows has shape"):
        pages.kv_decode_fwd(p, two, q, sink, q_per_seq=2, cu_rows=two)
    with pytest.raises(ValueError, match="q has shape"):
        pages.kv_decode_fwd(p, two, q, sink, q_per_seq=2)
    with pytest.raises(ValueError, match="multiple"):
        pages.kv_decode_fwd(p, two, q[:, :3], sink, q_per_seq=1)
    with pytest.raises(ValueError, match="sink has shape"):
        pages.kv_decode_fwd(p, two, q, sink[:2], q_per_seq=2, cu_rows=torch.zeros(3, dtype=torch.int32))


def test_verify_binding_refuses():
    x, u, cu = torch.zeros((3, 8)), torch.zeros(3), torch.tensor([0, 2, 3], dtype=torch.int32)
    d = torch.zeros(1, dtype=torch.int32)
    for bad, error, match in ((x[0], ValueError, "2-D"), (x.double(), TypeError, "logits has dtype"),
                              (torch.zeros((8, 3)).t(), ValueError, "rows"), (x[:1].expand(3, 8), ValueError, "overlap"),
                              (x, ValueError, "CUDA tensor")):
        with pytest.raises(error, match=match):
            rollout.verify_tokens(bad, d, u, cu)
    with pytest.raises(TypeError, match="draft_logits has dtype"):
        rollout.verify_tokens(x, d, u, cu, draft_logits=torch.zeros((1, 8)).half())
    with pytest.raises(ValueError, match="draft_logits has shape"):
        rollout.verify_tokens(x, d, u, cu, draft_logits=torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="u has shape"):
        rollout.verify_tokens(x, d, u[:2], cu)
    with pytest.raises(ValueError, match="temperature has shape"):
        rollout.verify_tokens(x, d, u, cu, temperature=u)
    with pytest.raises(ValueError, match="cu_rows"):
        rollout.verify_tokens(x, d, u, cu[:0])
    with pytest.raises(TypeError, match="drafts has dtype"):
        rollout.verify_tokens(x, d.long(), u, cu)


def test_decode_workspace_is_sized_on_the_pages_device(monkeypatch):
    current = ["cuda:0"]

    class Device:
        def __init__(self, device):
            self.device = str(device)

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *_):
            current.pop()

    class Library:
        @staticmethod
        def sinkattn_kv_decode_workspace_size(heads):
            return {"cuda:0": 100, "cuda:1": 300}[current[-1]] + heads

    made = {}
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(_lib, "load", lambda: Library)
    monkeypatch.setattr(torch, "zeros", lambda size, dtype, device: made.update(size=size, device=str(device)))
    p = object.__new__(pages.KVPages)
    p.device, p.num_heads_kv = torch.device("cuda:1"), 7
    pages.kv_decode_workspace(p)
    assert made == dict(size=307, device="cuda:1") and current == ["cuda:0"]


# ---------------------------------------------------------------- the oracle
def test_plan_by_hand():
    p = ref.Pages(4, 3, 3, 1, 16)
    live, cu, places, pos = p.plan([2, 0], [0, 0], [17, 16], 34)
    assert list(live) == [2, 0] and list(cu) == [0, 17, 33] and list(p.owner) == [2, 2, 0, -1]
    assert list(places[:17]) == list(range(17)) and list(places[17:]) == list(range(32, 48)) + [-1]
    assert list(pos[15:19]) == [15, 16, 0, 1]
    # slot 2 drops what its second page held and slot 0 takes that page; slot 1 needs one more than is left
    live, cu, places, pos = p.plan([2, 0, 1, 2], [1, 0, 0, 5], [0, 1, 17, 1], 30)
    assert list(live) == [2, 0, -1, -1] and list(cu) == [0, 0, 1, 18, 19] and list(p.owner) == [2, 0, 0, -1]
    assert list(p.lens) == [17, 0, 16] and list(places) == [16] + [-1] * 29 and list(pos) == [16] + [-1] * 29
    assert list(p.plan([0, 5, 1], [99, 0, 0], [-1, 2, 49], 2)[0]) == [-1, -1, -1]  # nothing of slot 0 is dropped either
    assert list(p.lens) == [17, 0, 16]


def test_verification_by_hand():
    x = np.log([[0.5, 0.25, 0.25], [0.2, 0.7, 0.1], [0.1, 0.1, 0.8]])
    y = np.log([[0.25, 0.5, 0.25], [0.6, 0.3, 0.1]])
    # draft 0: 0.25 u < 0.5 always; draft 1 (token 0): 0.6 u < 0.2 for u < 1/3
    tokens, logp, acc, w, _ = ref.verify(x, y, [0, 0], [0.9, 0.3, 0.15], 1.0)
    assert list(tokens) == [0, 0, 1] and acc == 2 and np.allclose(np.exp(logp), [0.5, 0.2, 0.1])
    tokens, logp, acc, w, _ = ref.verify(x, y, [0, 0], [0.9, 0.4, 0.99], 1.0)  # drawn from (0, 0.4, 0)
    assert list(tokens) == [0, 1, -1] and acc == 1 and np.allclose(w, [0, 0.4, 0]) and logp[2] == 0
    tokens, logp, acc, w, _ = ref.verify(x, None, [0, 1], [0.4, 0.8, 0.7], 1.0)  # without 1: 2/3 to 0, 1/3 to 2
    assert list(tokens) == [0, 2, -1] and acc == 1
    tokens, logp, acc, w, _ = ref.verify(x, y, [0, 1], [0.9, 0.9, 0.9], 0.0)
    assert list(tokens) == [0, 1, 2] and acc == 2
    tokens, logp, acc, w, _ = ref.verify(x, y, [7, 1], [0.0, 0.0, 0.0], 1.0)
    assert acc == 0 and tokens[0] == 0


def test_verified_tokens_follow_the_target():
    """Over a fine grid of random numbers the first token emitted is distributed as p, whatever q is."""
    x, y = np.log([[0.5, 0.3, 0.2], [1 / 3, 1 / 3, 1 / 3]]), np.log([[0.1, 0.3, 0.6]])
    count, N = np.zeros(3), 60
    grid = (np.arange(N) + 0.5) / N
    for d, qd in enumerate([0.1, 0.3, 0.6]):
        for u0 in grid:
            for u1 in grid:
                count[ref.verify(x, y, [d], [u0, u1], 1.0)[0][0]] += qd / N ** 2
    assert np.abs(count - [0.5, 0.3, 0.2]).max() < 2 / N
