"""Rollout-side operators on the CPU: refusals of the C ABI and of the binding, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.rollout_ref as ref
from sink_aware_masked_gb300 import _lib, rollout

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails validation first
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from sink_aware_masked_gb300 import build

    build.build()
    return _lib.load()


def cache(**kw):
    base = dict(pages=FAKE, page_table=FAKE, seqlens=FAKE, refcount=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=8,
                page_size=64, num_heads_kv=2, num_slots=4, max_pages=4)
    base.update(kw)
    return _lib.Kv4Cache(**base)


BAD_CACHES = [
    (dict(num_pages=0), INVALID), (dict(num_slots=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_heads_kv=0), INVALID), (dict(num_heads_kv=257), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
    (dict(max_pages=(1 << 30) // 64 + 1), UNSUPPORTED), (dict(pages=None), INVALID), (dict(k_scale=None), INVALID),
    (dict(refcount=FAKE + 4), ALIGNMENT), (dict(pages=FAKE + 8), ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, kw, status):
    c, good = ctypes.byref(cache(**kw)), ctypes.byref(cache())
    f = FAKE
    assert lib.sinkattn_kv4_reserve(c, f, f, 1, f, None) == status
    assert lib.sinkattn_kv4_fork(c, f, f, 1, f, None) == status
    assert lib.sinkattn_kv4_free(c, f, 1, None) == status
    assert lib.sinkattn_kv4_compact(c, good, f, f, 1 << 20, None) == status
    assert lib.sinkattn_kv4_compact(good, c, f, f, 1 << 20, None) == status
    assert lib.sinkattn_kv4_compact_workspace_size(c) == 0
    assert lib.sinkattn_kv4_append(c, f, 1, None, 4, f, f, None) == status
    assert lib.sinkattn_kv4_read(c, f, 1, None, 4, f, f, None) == status
    assert lib.sinkattn_kv4_decode_fwd(c, f, 1, 1, 4, -1, 0, 0.125, f, f, f, f, f, 1 << 30, None) == status
    assert lib.sinkattn_kv4_reserve(None, f, f, 1, f, None) == INVALID


@pytest.mark.parametrize("n,p,status", [(-1, FAKE, INVALID), (4097, FAKE, UNSUPPORTED), (1, None, INVALID),
                                        (1, FAKE + 2, ALIGNMENT), (0, None, OK)])
def test_lists_are_checked(lib, n, p, status):
    c, f = ctypes.byref(cache()), FAKE
    assert lib.sinkattn_kv4_free(c, p, n, None) == status
    for args in ((p, f, n, f), (f, p, n, f), (f, f, n, p)):
        assert lib.sinkattn_kv4_reserve(c, *args, None) == status
        assert lib.sinkattn_kv4_fork(c, *args, None) == status
    assert lib.sinkattn_kv4_append(c, p, n, None, 0, f, f, None) == status
    assert lib.sinkattn_kv4_decode_fwd(c, p, n, 1, 4, -1, 0, 0.125, f, f, f, f, f, 0 if n == 0 else 1 << 30,
                                       None) == status


def test_append_and_read_refuse(lib):
    c, f = ctypes.byref(cache()), FAKE
    for fn in (lib.sinkattn_kv4_append, lib.sinkattn_kv4_read):
        assert fn(c, f, 2, None, 3, f, f, None) == INVALID       # not the same number of rows each
        assert fn(c, f, 0, None, 3, f, f, None) == INVALID
        assert fn(c, f, 1, None, -1, f, f, None) == INVALID
        assert fn(c, f, 1, None, 3, None, f, None) == INVALID
        assert fn(c, f, 1, None, 3, f, f + 8, None) == ALIGNMENT
        assert fn(c, f, 1, f + 2, 3, f, f, None) == ALIGNMENT
        assert fn(c, f, 1, None, 0, None, None, None) == OK       # nothing to do


def test_decode_refuses(lib):
    c, f = ctypes.byref(cache()), FAKE
    ws = lib.sinkattn_kv4_decode_workspace_size(2, 4)

    def call(n=2, rows=1, hq=4, window=-1, prefix=0, scale=0.125, q=f, sink=f, o=f, lse=f, w=f, size=ws):
        return lib.sinkattn_kv4_decode_fwd(c, f, n, rows, hq, window, prefix, scale, q, sink, o, lse, w, size, None)

    assert call(rows=0) == INVALID and call(hq=3) == INVALID and call(hq=0) == INVALID
    assert call(hq=512) == UNSUPPORTED and call(rows=65) == UNSUPPORTED
    assert call(window=-2) == INVALID and call(prefix=-1) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == INVALID
    for name in ("q", "sink", "o", "lse", "w"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: f + 8}) == ALIGNMENT
    assert call(size=ws - 1) == WORKSPACE
    assert lib.sinkattn_kv4_decode_workspace_size(-1, 4) == 0 and lib.sinkattn_kv4_decode_workspace_size(1, 0) == 0
    assert lib.sinkattn_kv4_decode_workspace_size(1, 257) == 0


def test_compact_refuses(lib):
    other = dict(pages=2 * FAKE, page_table=2 * FAKE, seqlens=2 * FAKE, refcount=2 * FAKE)
    a, f = cache(), FAKE
    size = lib.sinkattn_kv4_compact_workspace_size(ctypes.byref(a))

    def call(b, count=f, ws=f, n=size):
        return lib.sinkattn_kv4_compact(ctypes.byref(a), ctypes.byref(b), count, ws, n, None)

    for name in other:  # shared memory
        assert call(cache(**{k: v for k, v in other.items() if k != name})) == INVALID
    for kw in (dict(page_size=32), dict(num_heads_kv=1), dict(num_slots=5), dict(max_pages=5)):
        assert call(cache(**other, **kw)) == INVALID
    good = cache(**other)
    assert call(good, count=None) == INVALID and call(good, count=f + 2) == ALIGNMENT
    assert call(good, ws=None) == INVALID and call(good, ws=f + 8) == ALIGNMENT and call(good, n=size - 1) == WORKSPACE


def test_sample_refuses(lib):
    f = FAKE

    def call(logits=f, dtype=0, rows=2, vocab=10, stride=10, ptrs=None):
        return lib.sinkattn_sample_tokens(logits, dtype, rows, vocab, stride, *(ptrs or [f] * 8), None)

    assert call(dtype=3) == INVALID and call(dtype=-1) == INVALID and call(rows=-1) == INVALID
    assert call(vocab=0) == INVALID and call(stride=9) == INVALID
    assert call(vocab=(1 << 18) + 1, stride=1 << 19) == UNSUPPORTED
    assert call(logits=None) == INVALID and call(logits=f + 2) == ALIGNMENT and call(logits=f + 1, dtype=1) == ALIGNMENT
    for i in range(8):
        assert call(ptrs=[f] * i + [None] + [f] * (7 - i)) == INVALID
        assert call(ptrs=[f] * i + [f + 2] + [f] * (7 - i)) == ALIGNMENT
    assert call(rows=0, ptrs=[None] * 8) == OK


# ---------------------------------------------------------------- the binding
def _cache_tensors(P=4, H=2, S=3, M=2, page=16):
    i32 = dict(dtype=torch.int32)
    return dict(pages=torch.zeros((P, H, page * 72), dtype=torch.uint8), page_table=torch.zeros((S, M), **i32),
                seqlens=torch.zeros(S, **i32), refcount=torch.zeros(P, **i32), k_scale=torch.ones(H),
                v_scale=torch.ones(H))


@pytest.mark.parametrize("name,make,error,match", [
    ("pages", lambda t: t.int(), TypeError, "pages has dtype"),
    ("pages", lambda t: t[:, :, :-1].contiguous(), ValueError, "multiple of 1152"),
    ("pages", lambda t: t.transpose(0, 1), ValueError, "contiguous|shape"),
    ("page_table", lambda t: t.long(), TypeError, "page_table has dtype"),
    ("seqlens", lambda t: t[:2], ValueError, "seqlens has shape"),
    ("refcount", lambda t: t[:2], ValueError, "refcount has shape"),
    ("k_scale", lambda t: t.double(), TypeError, "k_scale has dtype"),
    ("v_scale", lambda t: t[:1], ValueError, "v_scale has shape"),
    ("v_scale", lambda t: t, ValueError, "CUDA tensor"),
])
def test_cache_refuses(name, make, error, match):
    t = _cache_tensors()
    t[name] = make(t[name])
    with pytest.raises(error, match=match):
        rollout.KV4Cache(**t)


def test_empty_refuses_page_sizes():
    with pytest.raises(ValueError, match="page_size"):
        rollout.KV4Cache.empty(4, 2, 2, 1, page_size=24)


def test_sample_binding_refuses():
    x, u = torch.zeros((2, 8)), torch.zeros(2)
    for bad, error, match in ((x[0], ValueError, "2-D"), (x.double(), TypeError, "logits has dtype"),
                              (x.t(), ValueError, "rows"), (x[:1].expand(2, 8), ValueError, "overlap"),
                              (x, ValueError, "CUDA tensor")):
        with pytest.raises(error, match=match):
            rollout.sample_tokens(bad, torch.zeros(bad.shape[0]))
    with pytest.raises(ValueError, match="u has shape"):
        rollout.sample_tokens(x, u[:1])
    with pytest.raises(TypeError, match="top_k has dtype"):
        rollout.sample_tokens(x, u, top_k=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="temperature has shape"):
        rollout.sample_tokens(x, u, temperature=torch.zeros(3))


# ---------------------------------------------------------------- the oracle
def test_e4m3_table_is_torch_s():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref.E4M3, equal_nan=True)


def test_quantise_by_hand():
    x = np.zeros((1, 64))
    x[0, :8] = [6, 5, 3.5, 2.5, 1.25, 0.75, 0.25, -0.2]  # scale 1: half ways go to the even code
    x[0, 16] = 448 * 6 * 2                               # beyond the largest scale: saturates
    x[0, 32] = 2.0 ** -10 * 6                            # amax / 6 halfway to the smallest scale: 0
    x[0, 48] = np.inf
    codes, scales = ref.quantise(x, 1.0)
    y = ref.values(codes, scales, 1.0)
    assert list(y[0, :8]) == [6, 4, 4, 2, 1, 1, 0, 0]
    assert y[0, 16] == 448 * 6 and y[0, 32] == 0 and np.isnan(y[0, 48:]).all()


def test_cache_bytes_come_back_and_no_byte_is_shared():
    rng = np.random.RandomState(0)
    c = ref.Cache(3, 1, 2, 2, 32)
    c.reserve([0], [50])
    k, v = rng.randn(50, 2, 64), rng.randn(50, 2, 64)
    c.fill(0, k, v)
    kk, vv = c.sequence(0)
    for x, y in ((k, kk), (v, vv)):
        codes, scales = ref.quantise(x, 1.0)
        assert np.array_equal(ref.values(codes, scales, 1.0), y)


def test_sampling_by_hand():
    x = np.log([0.1, 0.4, 0.4, 0.1])
    assert ref.sample(x, 0.0, 0.0, 0, 1.0, 0.0)[0] == 1          # greedy: the lower of equal ones
    assert ref.sample(x, 0.6, 1.0, 2, 1.0, 0.0)[0] == 2          # top-k 2 keeps 1 and 2
    assert ref.sample(x, 0.999, 1.0, 0, 0.4 - 1e-9, 0.0)[0] == 1  # the first alone reaches p
    assert ref.sample(x, 0.999, 1.0, 0, 0.5, 0.0)[0] == 2
    token, logp, logq = ref.sample(x, 0.05, 1.0, 0, 1.0, 0.5)
    assert token == 1 and abs(logp - np.log(0.4)) < 1e-12 and abs(logq - np.log(0.5)) < 1e-12


def test_a_caches_tensors_cannot_be_replaced():
    """The library keeps their addresses; a write in place, also by an augmented assignment, is fine."""
    c = object.__new__(rollout.KV4Cache)
    c.seqlens, c.num_heads_kv = torch.zeros(3, dtype=torch.int32), 300
    first = c.seqlens
    c.seqlens += 2
    c.seqlens[1] = 5
    assert c.seqlens is first and first.tolist() == [2, 5, 2]
    with pytest.raises(AttributeError, match="seqlens of a KV4Cache cannot be replaced"):
        c.seqlens = c.seqlens + 1
    with pytest.raises(AttributeError, match="num_heads_kv"):
        c.num_heads_kv = 1
    assert c.seqlens is first and c.num_heads_kv == 300
    c.note = 1
    c.note = 2


@pytest.mark.parametrize("n,src,dst,done", [(1, 0, 64, 0), (1, 0, 64, 64), (8, 0, 64, 28), (8, 0, 64, 92), (8, 64, 0, 36),
                                            (4096, 0, 1 << 20, 4 * 4095)])
def test_fork_refuses_a_done_that_overlaps_its_lists(lib, n, src, dst, done):
    """Its second launch reads src and dst after the first one has written done."""
    c = ctypes.byref(cache())
    assert lib.sinkattn_kv4_fork(c, FAKE + src, FAKE + dst, n, FAKE + done, None) == INVALID
    assert lib.sinkattn_kv4_fork(c, FAKE, FAKE, 0, FAKE, None) == OK  # nothing is read or written


def test_decode_workspace_is_sized_on_the_caches_device(monkeypatch):
    """The size depends on the device's number of SMs: the cache's device is asked, whichever is current."""
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
        def sinkattn_kv4_decode_workspace_size(rows, heads):
            return {"cuda:0": 100, "cuda:1": 300}[current[-1]] + rows * heads

    made = {}
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(_lib, "load", lambda: Library)
    monkeypatch.setattr(torch, "zeros", lambda size, dtype, device: made.update(size=size, device=str(device)))
    c = object.__new__(rollout.KV4Cache)
    c.device = torch.device("cuda:1")
    rollout.kv4_decode_workspace(c, torch.empty(2, 8, 64))
    assert made == dict(size=316, device="cuda:1") and current == ["cuda:0"]


@pytest.mark.parametrize("kw", [dict(num_pages=2 ** 31 - 1, num_heads_kv=256, page_size=256), dict(num_pages=2 ** 31 - 1),
                                dict(num_pages=2 ** 28, num_heads_kv=2, page_size=256)])
def test_pools_of_any_size_are_taken(lib, kw):
    """Blocks are addressed in 64 bits; the header names no limit of a pool but its int32 count of pages."""
    c = ctypes.byref(cache(**kw))
    assert lib.sinkattn_kv4_free(c, None, 0, None) == OK and lib.sinkattn_kv4_reserve(c, None, None, 0, None, None) == OK
    assert lib.sinkattn_kv4_append(c, FAKE, 1, None, 0, None, None, None) == OK
    pages = kw["num_pages"]
    assert lib.sinkattn_kv4_compact_workspace_size(c) == 4 * (-(-pages // 1024) + 2 * pages)


def test_decode_workspace_holds_what_the_ctas_can_leave(lib):
    """At most 64 partial rows of 64 accumulators and two statistics per SM (two cut pairs a CTA), beside the counters."""
    size = lib.sinkattn_kv4_decode_workspace_size
    assert 0 < size(0, 1) <= 152 * 64 * 66 * 4 + 256
    assert size(100, 64) == size(0, 1) + 100 * 64 * 4
