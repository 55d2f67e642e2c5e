"""4-bit paged cache: CUDA path vs the float64 oracle (needs a GB300).

Tolerances of the decode outputs.  A score is a sum of 64 products, exact in
fp32 each, added in fp32: it is off by at most 64 * 2^-23 sum |q_d K_d| scale
=: ds (one step per addition, which covers truncating adders).  lse is then
off by ds plus the last roundings of a few units of 2^-23 relative to its
log2 value.  A probability is off by a factor e^(2 ds) and by half a step of
f16 (2^-11); exponentials and divisions add a few 2^-22.  So o, a weighted
mean of the values, is off by at most (2 ds + 2^-11 + 2^-20) max|v| before its
own rounding to bf16, half a step, 2^-8 |o|.
"""
import numpy as np
import pytest
import torch

import oracle
import oracle.rollout_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    from sink_aware_masked_gb300 import build

    build.build()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def handle(c):
    import sink_aware_masked_gb300 as sa

    return sa.KV4Cache(dev(c.pages), dev(c.table), dev(c.lens), dev(c.ref), dev(c.k_scale), dev(c.v_scale))


def bf16(a):
    return torch.from_numpy(a).to(torch.bfloat16)


def shuffled(rng, lens, page, heads, spare=3, factors=True):
    """A cache whose slots hold random tokens in pages in mixed order."""
    held = [-(-n // page) for n in lens]
    c = ref.Cache(sum(held) + spare, len(lens), max(max(held), 1) + 1, heads, page,
                  *((rng.uniform(0.5, 2, heads).astype(np.float32) for _ in range(2)) if factors else ()))
    order, at = rng.permutation(sum(held) + spare), 0
    for s, h in enumerate(held):
        c.table[s, :h] = order[at:at + h]
        c.ref[order[at:at + h]] = 1
        c.lens[s] = lens[s]
        at += h
    for s, n in enumerate(lens):
        if n:
            c.fill(s, rng.randn(n, heads, 64), rng.randn(n, heads, 64))
    return c


def check_decode(c, slots, n, hq, window, prefix, q, sink, o, lse, scale=0.125, keep=None):
    """Every row against the oracle over the slot's values; rows without a position are 0 and -inf."""
    q64, sink64 = q.double().cpu().numpy(), sink.double().cpu().numpy()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    group = hq // c.heads
    for b, s in enumerate(slots):
        L = int(c.lens[s]) if 0 <= s < len(c.lens) else 0
        there = min(n, L)
        rows = slice(b * n + n - there, (b + 1) * n)
        assert (o[b * n:b * n + n - there] == 0).all() and np.isneginf(lse[:, b * n:b * n + n - there]).all()
        if there == 0:
            continue
        k, v = c.sequence(s)
        want_o, want_l = oracle.decode_forward(q64[rows], k, v, sink64, [0, L], there, window, prefix, True, scale)
        ds = 64 * 2.0 ** -23 * scale * np.einsum("nhd,khd->nhk", np.abs(q64[rows]), np.abs(k).repeat(group, 1)).max(-1)
        vmax = np.abs(v).max((0, 2)).repeat(group)[None, :, None]
        err = np.abs(o[rows] - want_o)
        tol = (2 * ds[..., None] + 2.0 ** -11 + 2.0 ** -20) * vmax + 2.0 ** -8 * np.abs(want_o)
        assert (err <= tol).all(), (b, s, float((err / tol).max()))
        err = np.abs(lse[:, rows] - want_l)
        assert (err <= ds.T + 2.0 ** -21 * (np.abs(want_l) + 4)).all(), (b, s, float(err.max()))


# ---------------------------------------------------------------- append and read
@pytest.mark.parametrize("page,heads,lens,new", [
    (16, 1, [1], [1]), (64, 2, [40, 100], [40, 33]), (32, 3, [17, 16, 15, 200], [1, 16, 0, 199]),
    (128, 8, [130, 5], [130, 5]), (256, 1, [300, 256], [31, 256]), (64, 5, [64] * 9, [1] * 9),
])
def test_append_and_read_exactly(page, heads, lens, new):
    """Factors of powers of two: the quotients' borders are exact in fp32 too, so every value is the oracle's."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(page + heads)
    c = ref.Cache(2000 // page + 20, len(lens) + 1, 2 + max(lens) // page, heads, page,
                  *(2.0 ** rng.randint(-2, 3, heads).astype(np.float32) for _ in range(2)))
    slots = list(rng.permutation(len(lens) + 1)[:len(lens)])
    c.reserve(slots, lens)
    h = handle(c)
    T = sum(new)
    k, v = (bf16(rng.randn(T, heads, 64) * np.exp(rng.randn(T, heads, 64))) for _ in range(2))
    k[0, 0, :16] = 0  # a group of zeros
    cu = np.concatenate(([0], np.cumsum(new)))
    pad = torch.full((3, heads, 64), float("nan"), dtype=torch.bfloat16)  # rows behind the last: never read
    sa.kv4_append(h, i32(slots), torch.cat((k, pad)).to(DEV), torch.cat((v, pad)).to(DEV), cu_new=i32(cu))
    out = [torch.full((T + 3, heads, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    sa.kv4_read(h, i32(slots), T + 3, cu=i32(cu), k=out[0], v=out[1])
    for got, x, f in ((out[0], k, c.k_scale), (out[1], v, c.v_scale)):
        assert (got[T:] == 7).all()
        codes, scales = ref.quantise(x.double().numpy(), f[None, :, None].astype(np.float64))
        want = torch.from_numpy(ref.values(codes, scales, f[None, :, None].astype(np.float64))).to(torch.bfloat16)
        assert torch.equal(got[:T].cpu(), want)
    # the oracle reads the same bytes
    c.pages = h.pages.cpu().numpy()
    for b, s in enumerate(slots):
        ks, vs = c.sequence(s)
        mine = slice(cu[b], cu[b + 1])
        for x, got in ((ks, out[0]), (vs, out[1])):
            assert torch.equal(bf16(x[lens[b] - new[b]:]), got[mine].cpu())


def test_append_any_factor_and_its_error():
    """The scale s is off from a = max|y| / 6 by at most d = max(2^-4 a, 2^-10) (half a step of e4m3, of its
    subnormals below 2^-6).  A code is off by at most half of the widest step, 1 * s <= a + d, and the largest value,
    6 a, which saturates at 6 s, by 6 d; then bf16, half a step."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(5)
    f = rng.uniform(0.01, 30, 2).astype(np.float32)
    c = ref.Cache(20, 1, 20, 2, 64, f, f[::-1].copy())
    c.reserve([0], [700])
    h = handle(c)
    k, v = (bf16(rng.randn(700, 2, 64) * np.exp(2 * rng.randn(700, 1, 1))) for _ in range(2))
    sa.kv4_append(h, i32([0]), k.to(DEV), v.to(DEV))
    got = sa.kv4_read(h, i32([0]), 700)
    for y, x, factor in ((got[0], k, c.k_scale), (got[1], v, c.v_scale)):
        y, x = y.double().cpu().numpy(), x.double().numpy()
        amax = np.abs(x).reshape(700, 2, 4, 16).max(-1).repeat(16, -1)
        a = amax / 6
        d = np.maximum(2.0 ** -4 * a, 2.0 ** -10 * factor[None, :, None])
        bound = np.maximum(a + d, 6 * d) * (1 + 2.0 ** -20) + np.abs(y) * 2.0 ** -8  # 2^-20: the fp32 quotients
        assert (np.abs(y - x) <= bound).all()


def test_append_token_by_token_equals_append_at_once():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(6)
    k, v = (bf16(rng.randn(37, 2, 64)).to(DEV) for _ in range(2))
    caches = []
    for step in (37, 1):
        h = sa.KV4Cache.empty(4, 1, 4, 2, page_size=16)
        for i in range(0, 37, step):
            assert int(sa.kv4_reserve(h, i32([0]), i32([step]))[0]) == 1
            sa.kv4_append(h, i32([0]), k[i:i + step], v[i:i + step])
        caches.append(h)
    assert torch.equal(caches[0].pages, caches[1].pages) and torch.equal(caches[0].seqlens, caches[1].seqlens)


def test_append_what_is_not_finite_and_where_nothing_is():
    import sink_aware_masked_gb300 as sa

    c = ref.Cache(4, 3, 2, 1, 16)
    c.reserve([0, 1], [16, 20])
    c.table[1, 1] = 77  # a page that does not exist
    h = handle(c)
    before = h.pages.clone()
    k, v = torch.ones((30, 1, 64), dtype=torch.bfloat16), torch.ones((30, 1, 64), dtype=torch.bfloat16)
    k[3, 0, 17] = float("nan")
    v[4, 0, 60] = float("-inf")
    # slot 0: 10 rows; an idle entry: 5 rows; slot 1: 12 rows, of which 4 have no page; slot 2 is empty: 3 rows
    cu, slots = i32([0, 10, 15, 27, 30]), i32([0, -1, 1, 2])
    sa.kv4_append(h, slots, k.to(DEV), v.to(DEV), cu_new=cu)
    kk, vv = sa.kv4_read(h, slots, 30, cu=cu)
    kk, vv = kk.float().cpu(), vv.float().cpu()
    assert torch.isnan(kk[3, 0, 16:32]).all() and not torch.isnan(kk[3, 0, :16]).any()
    assert torch.isnan(vv[4, 0, 48:]).all() and not torch.isnan(vv[4, 0, :48]).any()
    one = 6 * 0.171875  # 16 ones: e4m3(1 / 6) = 11/64, and 1 / (11/64) = 5.8 is nearest to 6
    for x in (kk, vv):
        assert (x[10:15] == 0).all() and (x[27:] == 0).all()       # idle, empty
        assert (x[15:23] == one).all() and torch.isnan(x[23:27]).all()  # the page that is there, the one that is not
        assert (x[[0, 1, 2, 5, 9]] == one).all()
    free = [p for p in range(4) if c.ref[p] == 0]
    assert torch.equal(h.pages[free], before[free])


# ---------------------------------------------------------------- decode
DECODE = [
    # lens, hq, hkv, rows, window, prefix, page
    ([1], 8, 1, 1, -1, 0, 16),
    ([37, 1, 16, 17, 300], 16, 2, 1, -1, 0, 64),
    ([129, 15], 8, 8, 1, -1, 0, 32),                  # one row per kv head
    ([400, 33, 7], 10, 2, 1, 20, 3, 16),              # group of 5
    ([200, 64, 65], 16, 2, 2, 64, 5, 128),            # 16 rows
    ([150, 3], 12, 4, 3, 0, 0, 64),                   # window 0: each row sees itself alone
    ([90, 31], 24, 1, 1, -1, 0, 64),                  # 24 rows
    ([260, 40, 2], 16, 2, 4, 30, 100, 16),            # 32 rows; a sequence shorter than the rows
    ([170, 20], 40, 1, 3, -1, 0, 32),                 # 120 rows: four row groups
    ([70], 64, 1, 2, 9, 2, 256),                      # 128 rows
    ([1500], 8, 1, 1, -1, 0, 64),                     # cut between CTAs
    ([700, 0, 900], 21, 3, 2, 130, 4, 64),            # an empty slot
]


@pytest.mark.parametrize("lens,hq,hkv,n,window,prefix,page", DECODE)
def test_decode_parity(lens, hq, hkv, n, window, prefix, page):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(len(lens) * 100 + hq + n)
    c = shuffled(rng, lens, page, hkv)
    h = handle(c)
    slots = [int(s) for s in rng.permutation(len(lens))] + [-1, len(lens)]  # two idle entries
    q = bf16(rng.randn(len(slots) * n, hq, 64) * 1.5).to(DEV)
    sink = dev(rng.uniform(-2, 2, hq), torch.float32)
    kw = dict(q_per_seq=n, window=window, prefix=prefix)
    ws = sa.kv4_decode_workspace(h, q)
    o, lse = sa.kv4_decode_fwd(h, i32(slots), q, sink, workspace=ws, **kw)
    check_decode(c, slots, n, hq, window, prefix, q, sink, o, lse)
    again = sa.kv4_decode_fwd(h, i32(slots), q, sink, workspace=ws, **kw)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)  # same bits, same workspace


def test_decode_ranges_of_q_and_sink():
    """Rows far beyond f16's range, sinks that take everything and nothing."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(8)
    c = shuffled(rng, [50], 16, 1, factors=False)
    h = handle(c)
    q = bf16(rng.randn(1, 8, 64))
    q[0, 0] *= 2.0 ** 90
    q[0, 1] *= 2.0 ** -90
    q[0, 2] = 0
    q[0, 3, 5] = 2.0 ** 40
    sink = torch.tensor([0, 0, 0, 0, float("inf"), float("-inf"), 1e30, -1e30])
    o, lse = sa.kv4_decode_fwd(h, i32([0]), q.to(DEV), sink.to(DEV), q_per_seq=1)
    k, v = c.sequence(0)
    s = 0.125 * np.einsum("hd,kd->hk", q[0].double().numpy(), k[:, 0])
    m = s.max(-1)
    want_l = m + np.log(np.exp(s - m[:, None]).sum(-1))
    p = np.exp(s - want_l[:, None])
    with np.errstate(over="ignore"):
        want = (p @ v[:, 0]) / (1 + np.exp(sink.double().numpy() - want_l))[:, None]
    o, lse = o[0].double().cpu().numpy(), lse[:, 0].double().cpu().numpy()
    for r in (1, 2, 4, 5, 6, 7):
        assert np.allclose(o[r], want[r], rtol=2.0 ** -7, atol=2.0 ** -9 * np.abs(v).max())
        assert abs(lse[r] - want_l[r]) <= 1e-5 * max(1, abs(want_l[r]))
    for r in (0, 3):  # one key takes all
        assert np.allclose(o[r], v[s[r].argmax(), 0], rtol=2.0 ** -8, atol=0)
        assert abs(lse[r] / want_l[r] - 1) < 1e-5
    assert (o[4] == 0).all()


@pytest.mark.parametrize("factor", [1.0, 2.0 ** -8, 2.0 ** -40, 2.0 ** -120])
@pytest.mark.parametrize("n,hq", [(1, 8), (2, 8), (4, 16)])
def test_decode_rows_of_zeros_and_tiny_queries(n, hq, factor):
    """Such a row's scores are 0, or nothing beside 1: it is the mean of what it sees, and no masked key is in it."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(13)
    c = shuffled(rng, [37, 5, 200], 16, 2, factors=False)
    c.k_scale = np.full(2, factor, dtype=np.float32)
    x = rng.randn(3 * n, hq, 64)
    x[:, 0] = 0
    x[:, 1] *= 2.0 ** -126
    x[:, 2] *= 2.0 ** -133  # bf16 subnormals
    x[:, hq - 1] = 0
    q, sink = bf16(x).to(DEV), dev(rng.randn(hq), torch.float32)
    for window, prefix in ((-1, 0), (20, 3)):
        o, lse = sa.kv4_decode_fwd(handle(c), i32([0, 1, 2]), q, sink, q_per_seq=n, window=window, prefix=prefix)
        check_decode(c, [0, 1, 2], n, hq, window, prefix, q, sink, o, lse)


@pytest.mark.parametrize("n,hq", [(1, 8), (3, 8), (4, 16)])
def test_decode_not_finite_only_where_it_is_seen(n, hq):
    """A NaN value, key or query, and a missing page, reach exactly the rows (and dims) that see them."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(9)
    L, window, prefix = 100, 10, 3
    c = shuffled(rng, [L], 16, 1, factors=False)
    q = bf16(rng.randn(n, hq, 64)).to(DEV)
    sink = torch.zeros(hq, device=DEV)
    kw = dict(q_per_seq=n, window=window, prefix=prefix)
    base, _ = sa.kv4_decode_fwd(handle(c), i32([0]), q, sink, **kw)
    assert torch.isfinite(base.float()).all()
    for key in (1, 2, 3, 50, L - n - window, L - 1 - window, L - 1 - window + 1, L - n, L - 1):
        sees = [key <= L - n + i and (L - n + i - key <= window or key < prefix) for i in range(n)]
        for what in ("k", "v", "page"):
            pages, table = c.pages.copy(), c.table.copy()
            page, at, r = c._block(0, key)
            t, i = (r % 8) // 2, r % 2 + 2 * (r // 8)
            if what == "k":
                c.pages[page, 0, at + 1024 + 2 * (4 * (r % 8) + 1) + r // 8] = 0x7F
            elif what == "v":
                c.pages[page, 0, at + 1088 + 4 * (4 * 2 + t) + i] = 0xFF
            else:
                c.table[0, key // 16] = -5
            o, lse = sa.kv4_decode_fwd(handle(c), i32([0]), q, sink, **kw)
            o = o.float().cpu()
            for row in range(n):
                if what == "page":
                    hit = any(k2 // 16 == key // 16 and k2 <= L - n + row and
                              (L - n + row - k2 <= window or k2 < prefix) for k2 in range(L))
                    assert torch.isnan(o[row]).all() if hit else torch.equal(o[row], base[row].float().cpu())
                elif not sees[row]:
                    assert torch.equal(o[row], base[row].float().cpu()), (key, what, row)
                elif what == "k":
                    assert torch.isnan(o[row]).all() and torch.isnan(lse[:, row]).all()
                else:
                    assert torch.isnan(o[row, :, 32:48]).all()
                    rest = torch.cat((o[row, :, :32], o[row, :, 48:]), -1)
                    assert torch.isfinite(rest).all() and torch.isfinite(lse[:, row]).all()
            c.pages, c.table = pages, table
    bad = q.clone()
    bad[0, 1, 7] = float("nan")
    o, lse = sa.kv4_decode_fwd(handle(c), i32([0]), bad, sink, **kw)
    assert torch.isnan(o[0, 1].float()).all() and torch.isnan(lse[1, 0])
    mask = torch.ones((n, hq), dtype=torch.bool, device=DEV)
    mask[0, 1] = False
    assert torch.equal(o[mask], base[mask])


def test_decode_what_lies_behind_the_last_token_is_not_read_into_the_result():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(10)
    c = shuffled(rng, [21], 64, 2, factors=False)
    q, sink = bf16(rng.randn(1, 16, 64)).to(DEV), torch.zeros(16, device=DEV)
    want = sa.kv4_decode_fwd(handle(c), i32([0]), q, sink, q_per_seq=1)
    keep = c.sequence(0)
    c.pages[:] = 0xFF  # codes of -6 under NaN scales everywhere else
    c.fill(0, *keep)
    got = sa.kv4_decode_fwd(handle(c), i32([0]), q, sink, q_per_seq=1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_one_workspace_for_calls_of_many_shapes():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(11)
    c = shuffled(rng, [900, 50, 333, 1200], 64, 2)
    h = handle(c)
    big = sa.kv4_decode_workspace(h, torch.empty((16, 16, 64)))
    for n, slots in ((4, [0, 1, 2, 3]), (1, [3]), (2, [2, 0]), (4, [1, 3, 0, 2]), (1, [0, 1, 2, 3])):
        q = bf16(rng.randn(n * len(slots), 16, 64)).to(DEV)
        sink = dev(rng.randn(16), torch.float32)
        o, lse = sa.kv4_decode_fwd(h, i32(slots), q, sink, q_per_seq=n, window=400, prefix=9, workspace=big)
        check_decode(c, slots, n, 16, 400, 9, q, sink, o, lse)
    part = big.numel() - 16 * 16 * 4
    assert (big[part:] == 0).all()


def test_decode_many_sequences():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(12)
    c = shuffled(rng, [int(x) for x in rng.randint(0, 40, 23)], 16, 1)
    h = handle(c)
    slots = [int(s) for s in rng.randint(-1, 24, 4096)]  # the largest call; slots read more than once
    q, sink = bf16(rng.randn(4096, 2, 64)).to(DEV), torch.zeros(2, device=DEV)
    o, lse = sa.kv4_decode_fwd(h, i32(slots), q, sink, q_per_seq=1)
    check_decode(c, slots[:300], 1, 2, -1, 0, q[:300], sink, o[:300], lse[:, :300])
    check_decode(c, slots[-50:], 1, 2, -1, 0, q[-50:], sink, o[-50:], lse[:, -50:])


@pytest.mark.parametrize("n,window,prefix", [(1, -1, 0), (2, -1, 0), (4, 30000, 5)])
def test_decode_long_against_the_bf16_kernel(n, window, prefix):
    """Shares of many blocks, pairs cut at many places.  The values are exact in bf16 here (factors 1), so the bf16
    decode works on the same numbers; its P is rounded to bf16 (2^-8 of the values) where this one's is in f16."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(13)
    lens, hkv, hq = [40011, 31, 52000, 38005, 700, 44444], 8, 64
    c = sa.KV4Cache.empty(sum(-(-x // 64) for x in lens), len(lens), 1000, hkv, page_size=64)
    slots = i32(list(range(len(lens))))
    assert sa.kv4_reserve(c, slots, i32(lens)).tolist() == [1] * len(lens)
    cu = [0] + [int(x) for x in np.cumsum(lens)]
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((cu[-1], hkv, 64), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    sa.kv4_append(c, slots, k, v, cu_new=i32(cu))
    k, v = sa.kv4_read(c, slots, cu[-1], cu=i32(cu))
    q = bf16(rng.randn(len(lens) * n, hq, 64) * 2).to(DEV)
    sink = dev(rng.randn(hq), torch.float32)
    o, lse = sa.kv4_decode_fwd(c, slots, q, sink, q_per_seq=n, window=window, prefix=prefix)
    o2, lse2 = sa.sinkattn_decode_fwd(q, k, v, sink, q_per_seq=n, cu_seqlens=i32(cu), cu_seqlens_host=cu, window=window,
                                      prefix=prefix)
    assert (o.float() - o2.float()).abs().max() <= 3 * 2.0 ** -8 * v.float().abs().max()
    # the mean over the rows is far below the largest error: a block lost or taken twice would show
    assert (o.float() - o2.float()).abs().mean() <= 2.0 ** -8 * o2.float().abs().mean()
    assert (lse - lse2).abs().max() <= 1e-4


# ---------------------------------------------------------------- pages
def same_state(h, c):
    assert np.array_equal(h.seqlens.cpu().numpy(), c.lens)
    assert np.array_equal(h.refcount.cpu().numpy(), c.ref)
    table = h.page_table.cpu().numpy()
    for s, n in enumerate(c.lens):
        held = c._pages_of(n)
        assert np.array_equal(table[s, :held], c.table[s, :held]), s


@pytest.mark.parametrize("seed", range(6))
def test_pages_any_order_of_calls(seed):
    """Random reserve, fork and free, among them slots named twice, out of range, full and empty, and too few pages."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(seed)
    page = int(rng.choice([16, 32, 64]))
    c = ref.Cache(int(rng.choice([5, 40, 300])), 40, 6, 2, page)
    c.pages = rng.randint(0, 256, c.pages.shape).astype(np.uint8)
    h = handle(c)
    for _ in range(40):
        n = int(rng.choice([1, 3, 30]))
        op = rng.choice(["reserve", "reserve", "fork", "free"])
        slots = rng.randint(-2, 42, n).astype(np.int32)
        if op == "reserve":
            new = rng.choice([-1, 0, 1, 5, 16, page, 3 * page, 7 * page], n).astype(np.int32)
            assert np.array_equal(sa.kv4_reserve(h, dev(slots), dev(new)).cpu().numpy(), c.reserve(slots, new))
        elif op == "fork":
            src = rng.randint(-1, 41, n).astype(np.int32)
            assert np.array_equal(sa.kv4_fork(h, dev(src), dev(slots)).cpu().numpy(), c.fork(src, slots))
        else:
            sa.kv4_free(h, dev(slots))
            c.free(slots)
        same_state(h, c)
        assert np.array_equal(h.pages.cpu().numpy(), c.pages)


def test_fork_of_a_slot_whose_open_page_is_missing():
    """Its tokens read as NaN from the copy as from the source, never as what a page held before."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(3)
    c = shuffled(rng, [40, 0, 0, 21], 16, 2)
    c.pages[c.ref == 0] = 0x11
    h = handle(c)
    lost = int(h.page_table[0, 2])
    h.page_table[0, 2] = c.pages.shape[0] + 5
    assert sa.kv4_fork(h, i32([0, 3]), i32([1, 2])).tolist() == [1, 1]
    assert h.seqlens.tolist() == [40, 40, 21, 21]
    assert int(h.page_table[1, 2]) == -1
    want = c.ref.copy()
    want[c.table[0, :2]] += 1
    want[c.table[3, 0]] += 1
    want[int(h.page_table[2, 1])] += 1  # the second entry's page; the first one's is free again
    assert c.ref[int(h.page_table[2, 1])] == 0 and h.refcount.tolist() == want.tolist() and c.ref[lost] == 1
    for x, y in zip(sa.kv4_read(h, i32([0, 1]), 80), sa.kv4_read(handle(c), i32([0]), 40)):
        for got in (x[:40], x[40:]):
            assert torch.equal(got[:32], y[:32]) and torch.isnan(got[32:].float()).all()


@pytest.mark.parametrize("n,pages", [(4096, 70000), (1025, 1500), (2048, 17)])
def test_pages_many_requests(n, pages):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(n)
    c = ref.Cache(pages, 5000, 40, 1, 16)
    c.ref[rng.rand(pages) < 0.7] = 1  # held by somebody else
    h = handle(c)
    slots = rng.randint(0, 5000, n).astype(np.int32)
    new = rng.randint(0, 200, n).astype(np.int32)
    assert np.array_equal(sa.kv4_reserve(h, dev(slots), dev(new)).cpu().numpy(), c.reserve(slots, new))
    same_state(h, c)
    src, dst = rng.choice(slots, n).astype(np.int32), rng.randint(0, 5000, n).astype(np.int32)
    assert np.array_equal(sa.kv4_fork(h, dev(src), dev(dst)).cpu().numpy(), c.fork(src, dst))
    same_state(h, c)
    assert np.array_equal(h.pages.cpu().numpy(), c.pages)
    sa.kv4_free(h, dev(dst))
    c.free(dst)
    same_state(h, c)


@pytest.mark.parametrize("page,heads,pool", [(16, 1, 30), (64, 3, 5000), (32, 8, 4097), (16, 1, 40001)])
def test_compact(page, heads, pool):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(page)
    c = ref.Cache(pool, 9, 7, heads, page)
    c.ref[rng.rand(pool) < 0.5] = 1  # so that the live pages lie apart
    held = c.ref.copy()
    c.reserve([0, 1, 2, 5], [3, 2 * page, page + 1, 1])
    c.fork([1, 2, 2], [3, 4, 8])
    c.ref -= held
    c.pages = rng.randint(0, 256, c.pages.shape).astype(np.uint8)
    h = handle(c)
    live = int((c.ref > 0).sum())
    for room in (live, live + 5):
        to = sa.KV4Cache.empty(room, 9, 7, heads, page_size=page)
        to.refcount.fill_(9)
        assert int(sa.kv4_compact(h, to)[0]) == live
        order = np.nonzero(c.ref)[0]
        assert np.array_equal(to.pages[:live].cpu().numpy(), c.pages[order])
        assert np.array_equal(to.refcount.cpu().numpy(), np.concatenate((c.ref[order], np.zeros(room - live))))
        assert np.array_equal(to.seqlens.cpu().numpy(), c.lens)
        place = {p: i for i, p in enumerate(order)}
        for s in range(9):
            n = c._pages_of(c.lens[s])
            assert to.page_table[s].tolist() == [place[p] for p in c.table[s, :n]] + [-1] * (7 - n)
    same_state(h, c)
    small = sa.KV4Cache.empty(max(live - 1, 1), 9, 7, heads, page_size=page)
    assert int(sa.kv4_compact(h, small)[0]) == live  # does not fit: nothing happens
    assert (small.refcount == 0).all() and (small.page_table == -1).all() and (small.pages == 0).all()


# ---------------------------------------------------------------- streams, graphs, the run of all
def test_step_captured_and_replayed_while_sequences_grow():
    """reserve, append and decode in one graph, replayed; each replay equals eager calls on a cache of its own."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(20)
    slots = i32([2, 0, -1])
    caches = [sa.KV4Cache.empty(12, 3, 5, 2, page_size=16) for _ in range(2)]
    one, sink = i32([1, 1, 1]), dev(rng.randn(16), torch.float32)
    k, v = (torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, o = torch.zeros((3, 16, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((3, 16, 64), dtype=torch.bfloat16, device=DEV)
    lse, done = torch.zeros((16, 3), device=DEV), i32([0, 0, 0])
    ws = sa.kv4_decode_workspace(caches[0], q)

    def step(c, o, lse, done):
        sa.kv4_reserve(c, slots, one, done=done)
        sa.kv4_append(c, slots, k, v)
        return sa.kv4_decode_fwd(c, slots, q, sink, q_per_seq=1, window=20, prefix=2, o=o, lse=lse, workspace=ws)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = sa.KV4Cache.empty(12, 3, 5, 2, page_size=16)
        step(warm, o, lse, done)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(caches[0], o, lse, done)
    for turn in range(40):
        for t in (k, v, q):
            t.copy_(bf16(rng.randn(*t.shape)))
        graph.replay()
        got = o.clone(), lse.clone(), done.clone()
        eager = [torch.empty_like(x) for x in (o, lse, done)]
        step(caches[1], *eager)
        for a, b in zip(got, eager):
            assert torch.equal(a, b), turn
    for a in ("pages", "page_table", "seqlens", "refcount"):
        assert torch.equal(getattr(caches[0], a), getattr(caches[1], a))
    assert caches[0].seqlens.tolist() == [40, 0, 40]


def test_two_streams_at_once():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(21)
    c = shuffled(rng, [1000, 700], 64, 2)
    h = handle(c)
    q, sink = bf16(rng.randn(2, 16, 64)).to(DEV), torch.zeros(16, device=DEV)
    want = sa.kv4_decode_fwd(h, i32([0, 1]), q, sink, q_per_seq=1)
    slots = i32([0, 1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [sa.kv4_decode_workspace(h, q) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, w in zip(streams, spaces):
            with torch.cuda.stream(s):
                outs.append(sa.kv4_decode_fwd(h, slots, q, sink, q_per_seq=1, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in outs)


def test_a_group_of_rollouts():
    """A prompt is prefilled, forked, grown and sampled; attention over the pages equals the bf16 attention over what
    they hold, and the samples' log-probabilities serve the GRPO loss."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(22)
    G, P, hq, hkv, V = 4, 75, 16, 2, 1000
    c = sa.KV4Cache.empty(64, G + 1, 12, hkv, page_size=16)
    prompt, rollouts = i32([0]), i32(list(range(1, G + 1)))
    assert sa.kv4_reserve(c, prompt, i32([P])).tolist() == [1]
    sa.kv4_append(c, prompt, *(bf16(rng.randn(P, hkv, 64)).to(DEV) for _ in range(2)))
    assert sa.kv4_fork(c, i32([0] * G), rollouts).tolist() == [1] * G
    assert int((c.refcount == G + 1).sum()) == P // 16
    sink = dev(rng.randn(hq), torch.float32)
    tokens, logps = [], []
    for turn in range(30):
        assert sa.kv4_reserve(c, rollouts, i32([1] * G)).tolist() == [1] * G
        sa.kv4_append(c, rollouts, *(bf16(rng.randn(G, hkv, 64)).to(DEV) for _ in range(2)))
        q = bf16(rng.randn(G, hq, 64)).to(DEV)
        o, lse = sa.kv4_decode_fwd(c, rollouts, q, sink, q_per_seq=1, window=50, prefix=4)
        L = P + turn + 1
        cu = i32([i * L for i in range(G + 1)])
        k, v = sa.kv4_read(c, rollouts, G * L, cu=cu)  # factors 1: bf16 holds the values exactly
        o2, lse2 = sa.sinkattn_decode_fwd(q, k, v, sink, q_per_seq=1, num_seqs=G, window=50, prefix=4)
        assert (o.float() - o2.float()).abs().max() <= 3 * 2.0 ** -8 * v.float().abs().max()  # P in bf16 there
        assert (lse - lse2).abs().max() <= 1e-4
        logits = dev(rng.randn(G, V) * 3, torch.float32)
        t, logp, _ = sa.sample_tokens(logits, dev(rng.rand(G), torch.float32), top_p=torch.full((G,), 0.9, device=DEV))
        full = torch.log_softmax(logits.double(), -1).gather(1, t.long()[:, None]).reshape(-1)
        assert (logp - full).abs().max() < 1e-5
        tokens.append(t)
        logps.append(logp)
    first = sa.kv4_read(c, i32([0, 1]), 2 * P + 30, cu=i32([0, P, 2 * P + 30]))
    for x in first:
        assert torch.equal(x[:P], x[P:2 * P])  # the prompt's own tokens, shared and copied
    old = torch.stack(logps, 1).reshape(-1).contiguous()
    stats, dlogp, adv = sa.grpo_loss(old, old, torch.ones(G * 30, dtype=torch.uint8, device=DEV),
                                     dev(rng.rand(G), torch.float32), i32([30 * i for i in range(G + 1)]),
                                     [30 * i for i in range(G + 1)], group_size=G)
    assert torch.isfinite(dlogp).all() and abs(float(stats[0])) < 1e-5
    sa.kv4_free(c, rollouts)
    assert int((c.refcount > 0).sum()) == -(-P // 16) and int(c.refcount.max()) == 1


def test_nothing_is_written_outside_the_outputs():
    """Sentinels around every output, the workspace, and the pool's pages that are not the call's."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(30)

    def guarded(shape, dtype, zero=False):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((4096 + n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        t = buf[4096:4096 + n].view(dtype).view(shape)
        if zero:
            t.zero_()
        return t, buf

    kept = []

    def out(shape, dtype, zero=False):
        t, buf = guarded(shape, dtype, zero)
        kept.append((buf, t.numel() * t.element_size()))
        return t

    lens, hkv = [1000, 17, 333, 64], 2
    c = shuffled(rng, lens, 16, hkv)
    pages, table = out(c.pages.shape, torch.uint8), out(c.table.shape, torch.int32)
    seqlens, refcount = out(c.lens.shape, torch.int32), out(c.ref.shape, torch.int32)
    for t, a in ((pages, c.pages), (table, c.table), (seqlens, c.lens), (refcount, c.ref)):
        t.copy_(dev(a))
    h = sa.KV4Cache(pages, table, seqlens, refcount, dev(c.k_scale), dev(c.v_scale))
    slots = i32([0, 1, 2, 3])
    for n in (1, 3, 8):
        q = bf16(rng.randn(4 * n, 16, 64)).to(DEV)
        ws = out(tuple(sa.kv4_decode_workspace(h, q).shape), torch.uint8, zero=True)
        o, lse = out(q.shape, torch.bfloat16), out((16, 4 * n), torch.float32)
        sa.kv4_decode_fwd(h, slots, q, torch.zeros(16, device=DEV), q_per_seq=n, o=o, lse=lse, workspace=ws)
    cu = i32([0, 5, 22, 122, 123])
    k, v = out((123, hkv, 64), torch.bfloat16), out((123, hkv, 64), torch.bfloat16)
    sa.kv4_read(h, slots, 123, cu=cu, k=k, v=v)
    before = h.pages.clone()
    sa.kv4_append(h, slots, k, v, cu_new=cu)
    mine = torch.zeros(h.pages.shape[0], dtype=torch.bool)
    for s, n in enumerate([5, 17, 100, 1]):
        for pos in range(lens[s] - n, lens[s]):
            mine[c.table[s, pos // 16]] = True
    assert torch.equal(h.pages[~mine.to(DEV)], before[~mine.to(DEV)])
    done = out((4,), torch.int32)
    sa.kv4_reserve(h, slots, i32([0, 40, 3, 1]), done=done)
    sa.kv4_free(h, i32([1]))
    sa.kv4_fork(h, i32([2, 0, 0, 9]), i32([1, 1, 3, 0]), done=done)
    to = sa.KV4Cache(out(c.pages.shape, torch.uint8), out(c.table.shape, torch.int32), out(c.lens.shape, torch.int32),
                     out(c.ref.shape, torch.int32), h.k_scale, h.v_scale)
    size = 2 * c.pages.shape[0] * 4 + 4096
    sa.kv4_compact(h, to, count=out((1,), torch.int32), workspace=out((size,), torch.uint8))
    for B, V in ((3, 50001), (2, 5)):
        x, one = torch.randn((B, V), device=DEV), torch.ones(B, device=DEV)
        for p in (0.9, 1.0):
            sa.sample_tokens(x, one * 0.5, top_p=one * p, tokens=out((B,), torch.int32), logp=out((B,), torch.float32),
                             logq=out((B,), torch.float32))
    torch.cuda.synchronize()
    assert sa.sinkattn_get_device_status() == 0
    for buf, n in kept:
        assert (buf[:4096] == 0xA5).all() and (buf[4096 + n:] == 0xA5).all()


@pytest.mark.parametrize("n,lens", [(1, [1]), (1, [900, 2]), (2, [900, 40]), (4, [5000, 7])])
def test_decode_sinks_that_leave_almost_nothing(n, lens):
    """sigmoid(l - sink) down to 2^-133 still multiplies: o = e^(l - sink) softmax(s) V is in bf16's normal range under
    the factor.  The exponential's argument is off by a few 2^-24 of itself (up to 92), so the relative error is under
    2^-15 beside the roundings of both results to bf16."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(31)
    hq = 8
    c = shuffled(rng, lens, 16, 1, factors=False)
    c.v_scale = np.array([2.0 ** 30], dtype=np.float32)
    q = bf16(rng.randn(len(lens) * n, hq, 64)).to(DEV)
    base = torch.full((hq,), -1e30, device=DEV)
    slots = i32(list(range(len(lens))))
    h = handle(c)
    plain, lse = sa.kv4_decode_fwd(h, slots, q, base, q_per_seq=n)
    for above in (20.0, 60.0, 80.0, 86.0):
        sink = torch.full((hq,), float(lse.max()) + above, device=DEV)
        o, lse2 = sa.kv4_decode_fwd(h, slots, q, sink, q_per_seq=n)
        assert torch.equal(lse2, lse)
        w = torch.exp(lse.double() - sink.double()[:, None])
        want = plain.double() * (w / (1 + w)).t()[:, :, None]
        assert ((o.double() - want).abs() <= (2 * 2.0 ** -8 + 2.0 ** -15) * want.abs() + 2.0 ** -126).all(), above


@pytest.mark.parametrize("n", [1, 2, 4])
def test_decode_small_factors_over_many_keys(n):
    """The mean of many equal values under a value factor of 2^-100 is that value: factor / (sum of probabilities)
    may leave fp32's range on the way, the result does not."""
    import sink_aware_masked_gb300 as sa

    L = 1 << 20
    c = sa.KV4Cache.empty(L // 256, 1, L // 256, 1, page_size=256, v_scale=torch.full((1,), 2.0 ** -100, device=DEV))
    sa.kv4_reserve(c, i32([0]), i32([L]))
    x = torch.zeros((L, 1, 64), dtype=torch.bfloat16, device=DEV)
    sa.kv4_append(c, i32([0]), x, torch.full_like(x, 1.5 * 2.0 ** -100))
    q = torch.zeros((100 * n, 8, 64), dtype=torch.bfloat16, device=DEV)
    o, lse = sa.kv4_decode_fwd(c, i32([0] * 100), q, torch.full((8,), -1e30, device=DEV), q_per_seq=n)
    assert ((o.double() / (1.5 * 2.0 ** -100) - 1).abs() <= 2.0 ** -8 + 2.0 ** -11).all()
    assert (lse - np.log(L)).abs().max() < 1e-4


@pytest.mark.parametrize("entries,n,far,score", [(500, 1, 262144, 17.53125), (500, 2, 262144, 17.53125),
                                                 (250, 4, 262144, 17.53125), (1, 1, 262144, 17.53125),
                                                 (3, 1, 700, 17.53125), (3, 2, 700, 5.25), (3, 4, 700, 5.25), (3, 1, 700, 5.625)])
def test_decode_one_strong_key_over_many_weak_ones(entries, n, far, score):
    """One key takes nearly all and its value is 0, as with the first token of trained models: what is left is the
    many others' share.  The largest probability stands in f16 as 2^7 at least, so one that is weaker is off by half
    a step, 2^-11 of itself or 2^-25 where f16 is subnormal, 2^-32 of the largest: o is off by
    (2 ds + 2^-11 + 2^-20) sum p |v| + far 2^-32 max|v| and its own rounding (ds as above).  l is a running sum in
    fp32, one addition per block and lane: an addition is off by 2^-24 of the sum at most, and here, where all weak
    keys are alike, always to the same side, so that lse is off by that much for every block of a warp: a pair's
    blocks are shared by 4 warps at least, those of a short one (700 keys) by none."""
    import sink_aware_masked_gb300 as sa

    hq, a, at = 8, 1.5, 40 if far < 1000 else 5
    q1 = score / 8 / a  # 64 dims, scale 1/8
    assert float(torch.tensor(q1).to(torch.bfloat16)) == q1
    c = sa.KV4Cache.empty(-(-far // 64), 1, -(-far // 64), 1, page_size=64)
    assert sa.kv4_reserve(c, i32([0]), i32([far])).tolist() == [1]
    k, v = torch.zeros((far, 1, 64), dtype=torch.bfloat16, device=DEV), torch.full((far, 1, 64), a, dtype=torch.bfloat16, device=DEV)
    k[at], v[at] = a, 0  # 6 * 2^-2: exact in the cache
    sa.kv4_append(c, i32([0]), k, v)
    q = torch.full((entries * n, hq, 64), q1, dtype=torch.bfloat16, device=DEV)
    sink = torch.full((hq,), -1e30, device=DEV)
    o, lse = sa.kv4_decode_fwd(c, i32([0] * entries), q, sink, q_per_seq=n)
    weak = (far - n + np.arange(n)).astype(np.float64)  # weak keys that row i sees
    total = np.exp(score) + weak
    p = np.tile(weak / total, entries)[:, None, None]
    want, want_l = p * a, np.tile(np.log(total), entries)[None]
    ds = 64 * 2.0 ** -23 * score
    tol = (2 * ds + 2.0 ** -11 + 2.0 ** -20) * p * a + far * 2.0 ** -32 * a + 2.0 ** -8 * want
    err = np.abs(o.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())
    err = np.abs(lse.double().cpu().numpy() - want_l)
    additions = far / 16 / (4 if far > 1000 else 1)
    assert (err <= ds + 2.0 ** -21 * (np.abs(want_l) + 4) + additions * 2.0 ** -24).all(), float(err.max())
