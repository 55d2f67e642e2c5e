"""Pages of bf16 keys and values: CUDA path vs the float64 oracle (needs a GB300).

Tolerances of the decode outputs.  A score is a sum of 64 products, exact in
fp32 each, added in fp32: it is off by at most 64 * 2^-23 sum |q_d K_d| scale
=: ds (one step per addition, which covers truncating adders).  lse is then
off by ds plus the last roundings of a few units of 2^-23 relative to its log2
value.  A probability is off by a factor e^(2 ds) and, in the product with the
values and in what that is divided by alike, by half a step of bf16 (2^-8);
exponentials and divisions add a few 2^-22.  So o, a weighted mean of the
values, is off by at most (2 ds + 2 * 2^-8 + 2^-20) times the mean |v| under
the same weights, and by its own rounding, 2^-8 |o|; what is below 2^-126, the
least normal number, may come out as 0 (a sink 100 above lse leaves e^-100,
2^-144, of the mean).
"""
import numpy as np
import pytest
import torch

import oracle
import oracle.pages_ref as ref
from oracle.sinkattn_ref import visible

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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf16(rng, *shape):
    return torch.from_numpy(rng.randn(*shape)).to(torch.bfloat16)


def handle(c):
    import sink_aware_masked_gb300 as sa

    return sa.KVPages(dev(c.k, torch.bfloat16), dev(c.v, torch.bfloat16), dev(c.table), dev(c.lens), dev(c.owner))


def same_tables(c, h):
    assert np.array_equal(h.seqlens.cpu().numpy(), c.lens)
    assert np.array_equal(h.owner.cpu().numpy(), c.owner)
    for s, n in enumerate(c.lens):
        held = c.pages_of(n)
        assert np.array_equal(h.block_table[s, :held].cpu().numpy(), c.table[s, :held]), s


def shuffled(rng, lens, page, heads, spare=3):
    """Slots that hold random tokens in pages in mixed order; what is not held is NaN."""
    held = [-(-n // page) for n in lens]
    c = ref.Pages(sum(held) + spare, len(lens), max(max(held), 1) + 1, heads, page)
    c.k[:] = c.v[:] = np.nan
    order, at = rng.permutation(sum(held) + spare), 0
    for s, n in enumerate(lens):
        c.table[s, :held[s]] = order[at:at + held[s]]
        c.owner[order[at:at + held[s]]] = s
        c.lens[s] = n
        at += held[s]
        k, v = bf16(rng, n, heads, 64).double().numpy(), bf16(rng, n, heads, 64).double().numpy()
        c.write([c.place(s, i) for i in range(n)], k, v)
    return c


def check_decode(c, slots, counts, hq, window, prefix, q, sink, o, lse, scale=0.125):
    """Every row against the oracle over the slot's values; rows without a position are 0 and -inf."""
    q64, sink64 = q.double().cpu().numpy(), sink.double().cpu().numpy()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    group, at = hq // c.heads, 0
    for b, (s, n) in enumerate(zip(slots, counts)):
        L = int(c.lens[s]) if 0 <= s < len(c.lens) else 0
        there = min(n, L)
        first, rows = slice(at, at + n - there), slice(at + n - there, at + n)
        at += n
        assert (o[first] == 0).all() and np.isneginf(lse[:, first]).all()
        if there == 0:
            continue
        k, v = c.sequence(s)
        unseen = ~visible(np.arange(L - there, L), np.arange(L), window, prefix, True).any(0)
        k[unseen] = v[unseen] = 0.0  # the oracle multiplies them by 0
        args = [0, L], there, window, prefix, True, scale
        want_o, want_l = oracle.decode_forward(q64[rows], k, v, sink64, *args)
        mean = oracle.decode_forward(q64[rows], k, np.abs(v), sink64, *args)[0]
        ds = 64 * 2.0 ** -23 * scale * np.einsum("nhd,khd->nhk", np.abs(q64[rows]), np.abs(k).repeat(group, 1)).max(-1)
        err = np.abs(o[rows] - want_o)
        tol = (2 * ds[..., None] + 2.0 ** -7 + 2.0 ** -20) * mean + 2.0 ** -8 * np.abs(want_o) + 2.0 ** -126
        assert (err <= tol).all(), (b, s, float((err / tol).max()))
        err = np.abs(lse[:, rows] - want_l)
        assert (err <= ds.T + 2.0 ** -21 * (np.abs(want_l) + 4)).all(), (b, s, float(err.max()))


# ---------------------------------------------------------------- plan
@pytest.mark.parametrize("page,slots,max_pages,pages", [(16, 7, 9, 40), (64, 40, 5, 90), (256, 3, 2, 5), (32, 300, 4, 700)])
def test_plans_follow_the_definition(page, slots, max_pages, pages):
    """Random requests one after another, pools that run out, repeated, idle and invalid entries among them."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(page)
    c = ref.Pages(pages, slots, max_pages, 1, page)
    h = handle(c)
    for turn in range(12):
        n = int(rng.randint(1, slots + 3))
        s = rng.randint(-1, slots + 1, n) if turn % 3 == 2 else rng.permutation(slots)[:n]
        n = len(s)
        new = rng.randint(0, page * 3, n) if turn % 2 else rng.randint(0, 4, n)
        drop = np.where(rng.rand(n) < 0.2, 2 ** 31 - 1, rng.randint(-3, page * 2, n))
        if turn % 4 == 3:
            new[rng.randint(n)] = -5
        total = int(np.maximum(new, 0).sum()) + int(rng.randint(0, 5))
        want = c.plan([int(x) for x in s], drop, [int(x) for x in new], total)
        got = sa.kv_plan(h, i32(s), i32(new), total, drop=i32(drop))
        for name, a, b in zip(("live", "cu", "slot_map", "positions"), got, want):
            assert np.array_equal(a.cpu().numpy(), b), (turn, name)
        same_tables(c, h)


@pytest.mark.parametrize("total", [4096, 4097, 30011])
def test_long_plans(total):
    """Rows beyond what one CTA places; most of them new prompts, one request that finds no room."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(1)
    new = rng.multinomial(total - 7, np.ones(50) / 50)
    c = ref.Pages(-(-total // 16) + 60, 51, -(-total // 16), 1, 16)
    h = handle(c)
    for slots, count in ((list(range(50)), new), ([50] + list(range(49, -1, -1)), np.concatenate(([total], new)))):
        count = [int(x) for x in count]
        rows = sum(count) + 7
        drop = [2 ** 31 - 1] * len(slots)
        want = c.plan(slots, drop, count, rows)
        got = sa.kv_plan(h, i32(slots), i32(count), rows, drop=i32(drop))
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)
        same_tables(c, h)


def test_plan_without_requests_and_in_place():
    import sink_aware_masked_gb300 as sa

    h = sa.KVPages.empty(4, 2, 2, 1, page_size=16)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    live, cu, places, pos = sa.kv_plan(h, none, none, 3)
    assert cu.tolist() == [0] and places.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3
    slots = i32([1, 9, 0])
    live, cu, places, pos = sa.kv_plan(h, slots, i32([1, 1, 1]), 3, live=slots)
    assert live is slots and slots.tolist() == [1, -1, 0] and places.tolist() == [0, -1, 16] and pos.tolist() == [0, -1, 0]
    sa.kv_plan(h, i32([1]), i32([0]), 0)
    assert h.seqlens.tolist() == [1, 1]


def test_pages_of_others_are_left_alone():
    """A table entry whose page belongs to another slot, or lies outside the pool, is cleared and nothing is freed."""
    import sink_aware_masked_gb300 as sa

    c = ref.Pages(6, 2, 4, 1, 16)
    c.plan([0, 1], [0, 0], [48, 32], 80)
    c.table[0, 1], c.table[0, 2] = c.table[1, 0], 99
    h = handle(c)
    want = c.plan([0], [2 ** 31 - 1], [16], 16)
    got = sa.kv_plan(h, i32([0]), i32([16]), 16, drop=i32([2 ** 31 - 1]))
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    same_tables(c, h)
    assert h.owner.tolist()[3:5] == [1, 1]


# ---------------------------------------------------------------- write
@pytest.mark.parametrize("heads", [1, 2, 3, 5, 8, 16])
@pytest.mark.parametrize("T", [1, 3, 64, 1001])
def test_write(heads, T):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(T + heads)
    h = sa.KVPages.empty(-(-T // 16) + 2, 1, 80, heads, page_size=16)
    h.k_pages.fill_(7.0)
    h.v_pages.fill_(9.0)
    places = rng.permutation(h.num_pages * 16)[:T]
    skipped = rng.rand(T) < 0.2
    at = np.where(skipped, rng.choice([-1, h.num_pages * 16, 2 ** 31 - 1], T), places)
    rows = bf16(rng, T, 4 * heads + 1, 64).to(DEV)  # k and v are views of wider rows
    k, v = rows[:, heads:2 * heads], rows[:, 3 * heads:4 * heads]
    want_k, want_v = h.k_pages.clone(), h.v_pages.clone()
    for want, x in ((want_k, k), (want_v, v)):
        want.view(-1, heads, 64)[torch.from_numpy(places[~skipped]).to(DEV)] = x[torch.from_numpy(~skipped).to(DEV)]
    sa.kv_write(h, i32(at), k, v)
    assert torch.equal(h.k_pages, want_k) and torch.equal(h.v_pages, want_v)


# ---------------------------------------------------------------- decode
CASES = [
    # page, kv heads, group, lengths, rows per sequence, window, prefix
    (16, 1, 8, [1], [1], -1, 0),
    (16, 2, 8, [37, 16, 17, 0, 33], [1, 1, 1, 1, 1], -1, 0),
    (64, 2, 4, [5, 64, 65, 300, 129], [3, 1, 4, 2, 4], -1, 0),
    (32, 8, 8, [700, 31, 32], [1, 1, 1], 50, 3),
    (128, 1, 16, [1000, 3], [2, 5], -1, 0),
    (256, 3, 7, [513, 1, 256, 90], [1, 8, 3, 1], 100, 4),
    (16, 1, 32, [400, 18], [4, 4], 0, 0),
    (64, 2, 5, [2000], [1], 128, 40),
    (16, 1, 1, [3000, 5, 77], [1, 1, 1], -1, 0),
    (64, 1, 64, [333], [2], 7, 130),
    (32, 2, 8, [9, 70], [8, 16], 5, 2),
    (16, 1, 128, [300, 40], [1, 1], -1, 0),
    (64, 1, 100, [131], [1], 64, 1),
]


@pytest.mark.parametrize("page,heads,group,lens,counts,window,prefix", CASES)
def test_decode(page, heads, group, lens, counts, window, prefix):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(page + sum(lens))
    c = shuffled(rng, lens, page, heads)
    h, hq = handle(c), heads * group
    slots = list(rng.permutation(len(lens)))
    counts = [counts[s] for s in slots]
    R = sum(counts)
    q, sink = bf16(rng, R, hq, 64).to(DEV), dev(rng.randn(hq), torch.float32)
    cu = i32(np.concatenate(([0], np.cumsum(counts))))
    ws = sa.kv_decode_workspace(h)
    o, lse = sa.kv_decode_fwd(h, i32(slots), q, sink, q_per_seq=max(counts), cu_rows=cu, window=window, prefix=prefix,
                              workspace=ws)
    check_decode(c, slots, counts, hq, window, prefix, q, sink, o, lse)
    for _ in range(3):  # the workspace serves the next call, and the result is the same
        o2, lse2 = sa.kv_decode_fwd(h, i32(slots), q, sink, q_per_seq=max(counts), cu_rows=cu, window=window,
                                    prefix=prefix, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if len(set(counts)) == 1:
        o2, lse2 = sa.kv_decode_fwd(h, i32(slots), q, sink, q_per_seq=counts[0], window=window, prefix=prefix)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("batch,length,page,heads,group,n", [(5, 9000, 64, 2, 8, 1), (1, 40000, 16, 1, 8, 1),
                                                             (2, 12001, 128, 2, 8, 2), (3, 7000, 64, 2, 8, 4),
                                                             (2, 9001, 64, 2, 8, 7), (1, 20001, 32, 1, 64, 2),
                                                             (2, 9001, 64, 2, 8, 5), (3, 8000, 16, 1, 6, 8),
                                                             (300, 40, 16, 2, 4, 1), (400, 70, 16, 2, 8, 2)])
def test_decode_cut_between_ctas(batch, length, page, heads, group, n):
    """Long sequences, whose pairs are cut and merged, and many short ones, which warps take alone."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(length)
    lens = [length - 6 * (b % 7) for b in range(batch)]
    c = shuffled(rng, lens, page, heads)
    h, hq = handle(c), heads * group
    q, sink = (bf16(rng, batch * n, hq, 64) * 2).to(DEV), dev(rng.randn(hq), torch.float32)
    slots = list(range(batch))
    o, lse = sa.kv_decode_fwd(h, i32(slots), q, sink, q_per_seq=n)
    check_decode(c, slots, [n] * batch, hq, -1, 0, q, sink, o, lse)


@pytest.mark.parametrize("n,group", [(1, 5), (2, 8), (4, 8), (5, 8), (7, 8), (8, 16), (3, 40), (1, 50)])
@pytest.mark.parametrize("window,prefix,hi", [(40, 3, 500), (0, 0, 90), (-1, 0, 150)])
def test_many_short_pairs(n, group, window, prefix, hi):
    """Warps that take whole pairs, alone: every count of rows, some entries without any, some longer than their slots."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(n + group)
    lens = [int(x) for x in rng.randint(0, hi, 90)]
    c = shuffled(rng, lens, 16, 2)
    h, hq = handle(c), 2 * group
    counts = [int(x) for x in rng.randint(0, n + 1, 90)]
    counts[7] = n
    R = sum(counts)
    q, sink = bf16(rng, R, hq, 64).to(DEV), dev(rng.randn(hq), torch.float32)
    cu = i32(np.concatenate(([0], np.cumsum(counts))))
    slots = [int(x) for x in rng.permutation(90)]
    slots[3] = -1
    o, lse = sa.kv_decode_fwd(h, i32(slots), q, sink, q_per_seq=n, cu_rows=cu, window=window, prefix=prefix)
    check_decode(c, slots, counts, hq, window, prefix, q, sink, o, lse)


@pytest.mark.parametrize("longest", [3, 5000])
def test_as_many_entries_as_a_call_takes(longest):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(longest)
    lens = [1 + b % 3 for b in range(4096)]
    lens[1234] = longest
    c = shuffled(rng, lens, 16, 1)
    q, sink = bf16(rng, 4096, 4, 64).to(DEV), dev(rng.randn(4), torch.float32)
    o, lse = sa.kv_decode_fwd(handle(c), i32(range(4096)), q, sink, q_per_seq=1)
    check_decode(c, list(range(4096)), [1] * 4096, 4, -1, 0, q, sink, o, lse)


def test_pools_beyond_32_bits():
    """Pages whose bytes, and whose values, lie beyond 2^32: written, attended to, and no other place touched."""
    import sink_aware_masked_gb300 as sa

    page, heads, pages = 64, 8, 135000  # 8.6 M tokens: 8.8 GB of keys, 4.4 G values
    rng = np.random.RandomState(12)
    pool = [torch.empty((pages, page, heads, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    at = [pages - 1, 5, pages - 3, 70000]
    for t in pool:
        t[[0, 4, 6, 69999, 70001, pages - 2]] = 3.0
    table = i32([at])
    h = sa.KVPages(*pool, table, i32([4 * page - 7]), torch.full((pages,), -1, dtype=torch.int32, device=DEV))
    T = 4 * page - 7
    places = np.array([at[i // page] * page + i % page for i in range(T)])
    k, v = bf16(rng, T, heads, 64), bf16(rng, T, heads, 64)
    sa.kv_write(h, i32(places), k.to(DEV), v.to(DEV))
    q, sink = bf16(rng, 2, 16, 64).to(DEV), dev(rng.randn(16), torch.float32)
    o, lse = sa.kv_decode_fwd(h, i32([0]), q, sink, q_per_seq=2)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, want_l = oracle.decode_forward(f64(q), f64(k), f64(v), f64(sink), [0, T], 2)
    assert np.abs(f64(o) - want).max() < 2.0 ** -5 and np.abs(f64(lse) - want_l).max() < 2.0 ** -14
    for t in pool:
        assert (t[[0, 4, 6, 69999, 70001, pages - 2]] == 3.0).all()


def test_rows_outside_the_entries_are_left_alone():
    """Padding before, behind and in place of entries; idle slots; a row count of zero."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(3)
    c = shuffled(rng, [50, 20, 30], 16, 2)
    h = handle(c)
    q, sink = bf16(rng, 12, 8, 64).to(DEV), dev(rng.randn(8), torch.float32)
    o, lse = torch.full_like(q, 5.0), torch.full((8, 12), 5.0, device=DEV)
    sa.kv_decode_fwd(h, i32([2, -1, 0, 1, 7]), q, sink, q_per_seq=3, cu_rows=i32([2, 5, 6, 6, 8, 9]), o=o, lse=lse)
    check_decode(c, [2, -1, 1, 7], [3, 1, 2, 1], 8, -1, 0, q[2:9], sink, o[2:9], lse[:, 2:9])
    rest = [0, 1, 9, 10, 11]
    assert (o[rest] == 5).all() and (lse[:, rest] == 5).all()


def test_rows_beyond_q_per_seq_are_left_alone():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(4)
    c = shuffled(rng, [50, 20], 16, 2)
    q, sink = bf16(rng, 7, 6, 64).to(DEV), dev(rng.randn(6), torch.float32)
    h, cu = handle(c), i32([0, 3, 7])
    want, want_l = sa.kv_decode_fwd(h, i32([0, 1]), q, sink, q_per_seq=4, cu_rows=cu)
    check_decode(c, [0, 1], [3, 4], 6, -1, 0, q, sink, want, want_l)
    for most in (1, 2, 3):
        o, lse = torch.full_like(q, 5.0), torch.full((6, 7), 5.0, device=DEV)
        sa.kv_decode_fwd(h, i32([0, 1]), q, sink, q_per_seq=most, cu_rows=cu, o=o, lse=lse)
        there = torch.tensor([i < most for i in (0, 1, 2, 0, 1, 2, 3)], device=DEV)
        assert torch.equal(lse[:, there], want_l[:, there]) and (lse[:, ~there] == 5).all()
        assert torch.equal(o[there], want[there]) and (o[~there] == 5).all()


@pytest.mark.parametrize("heads,group,n", [(40, 1, 1), (200, 1, 2), (160, 1, 1), (3, 16, 6)])
def test_many_kv_heads(heads, group, n):
    """More kv heads than there are shares, or than CTAs."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(heads)
    lens = [333, 65, 0, 1200]
    c = shuffled(rng, lens, 32, heads)
    q, sink = bf16(rng, 4 * n, heads * group, 64).to(DEV), dev(rng.randn(heads * group), torch.float32)
    o, lse = sa.kv_decode_fwd(handle(c), i32([3, 1, 2, 0]), q, sink, q_per_seq=n)
    check_decode(c, [3, 1, 2, 0], [n] * 4, heads * group, -1, 0, q, sink, o, lse)


@pytest.mark.parametrize("n,group", [(1, 8), (2, 8), (4, 8), (6, 8), (8, 8), (3, 32)])
@pytest.mark.parametrize("window,prefix", [(-1, 0), (9, 2)])
def test_what_is_not_seen_does_not_matter(n, group, window, prefix):
    """NaN and infinities behind the length, below the window and after a row's own position."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(n)
    lens = [75, 130, 64]
    c = shuffled(rng, lens, 32, 2)
    hq = 2 * group
    q, sink = bf16(rng, 3 * n, hq, 64).to(DEV), dev(rng.randn(hq), torch.float32)
    h = handle(c)
    o, lse = sa.kv_decode_fwd(h, i32([0, 1, 2]), q, sink, q_per_seq=n, window=window, prefix=prefix)
    check_decode(c, [0, 1, 2], [n] * 3, hq, window, prefix, q, sink, o, lse)
    for bad in (np.nan, np.inf, -np.inf):
        for s, L in enumerate(lens):
            at = [L - 1]  # seen by the last row alone
            if window >= 0:
                at += [i for i in range(prefix, L - n - window) if i % 3]
            for i in at:
                page, row = divmod(c.place(s, i), 32)
                c.k[page, row] = bad
                c.v[page, row] = bad
        h = handle(c)
        o2, lse2 = sa.kv_decode_fwd(h, i32([0, 1, 2]), q, sink, q_per_seq=n, window=window, prefix=prefix)
        last = torch.arange(3 * n, device=DEV) % n == n - 1
        assert torch.equal(o[~last], o2[~last]) and torch.equal(lse[:, ~last], lse2[:, ~last])
        assert not torch.isfinite(o2[last]).any()


def test_values_that_are_infinite_reach_the_rows_that_see_them():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(5)
    c = shuffled(rng, [40], 16, 1)
    for i, bad in ((38, np.inf), (20, -np.inf)):
        page, row = divmod(c.place(0, i), 16)
        c.v[page, row, 0, 5] = bad
    q, sink = bf16(rng, 2, 8, 64).to(DEV), torch.zeros(8, device=DEV)
    o, _ = sa.kv_decode_fwd(handle(c), i32([0]), q, sink, q_per_seq=2, window=10)
    assert torch.isposinf(o[..., 5]).all()                      # 38 is seen by both rows, 20 by neither
    assert torch.isfinite(o[..., :5]).all() and torch.isfinite(o[..., 6:]).all()


def test_pages_that_are_missing_read_as_nan():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(6)
    c = shuffled(rng, [100, 100, 100], 16, 2)
    c.table[0, 1], c.table[1, 6], c.table[2, 0] = -1, 10 ** 6, -7
    q, sink = bf16(rng, 3, 8, 64).to(DEV), torch.zeros(8, device=DEV)
    h = handle(c)
    o, lse = sa.kv_decode_fwd(h, i32([0, 1, 2]), q, sink, q_per_seq=1)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    o, lse = sa.kv_decode_fwd(h, i32([0, 1, 2]), q, sink, q_per_seq=1, window=30)  # sees tokens 69 and on
    assert torch.isnan(o[1]).all() and torch.isnan(lse[:, 1]).all()
    check_decode(c, [0], [1], 8, 30, 0, q[:1], sink, o[:1], lse[:, :1])
    check_decode(c, [2], [1], 8, 30, 0, q[2:], sink, o[2:], lse[:, 2:])


def test_pages_may_be_shared_and_extreme_sinks():
    """Two slots with the same first pages; sinks far above and below every score."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(7)
    c = shuffled(rng, [96, 80], 32, 1)
    c.table[1, :2] = c.table[0, :2]
    sink = dev([-1e4, -50.0, 0.0, 5.0, 60.0, 100.0, 1e4, 3.0], torch.float32)
    q = bf16(rng, 2, 8, 64).to(DEV)
    o, lse = sa.kv_decode_fwd(handle(c), i32([0, 1]), q, sink, q_per_seq=1)
    check_decode(c, [0, 1], [1, 1], 8, -1, 0, q, sink, o, lse)


@pytest.mark.parametrize("scale", [1e-40, 1e-20, 0.01, 3.0])
def test_scales(scale):
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(8)
    c = shuffled(rng, [150, 31], 64, 1)
    q, sink = bf16(rng, 4, 8, 64).to(DEV), dev(rng.randn(8), torch.float32)
    o, lse = sa.kv_decode_fwd(handle(c), i32([0, 1]), q, sink, q_per_seq=2, scale=scale)
    check_decode(c, [0, 1], [2, 2], 8, -1, 0, q, sink, o, lse, scale=float(np.float32(scale)))


def test_one_strong_key_over_many_weak_ones():
    """The weak keys' share of the output is not lost, and the strong key alone gives its value."""
    import sink_aware_masked_gb300 as sa

    c = ref.Pages(2200, 1, 2200, 1, 16)
    L = 32768
    c.plan([0], [0], [L], 0)
    k, v = np.zeros((L, 1, 64)), np.ones((L, 1, 64)) * 64.0
    k[1000, 0, 0], v[1000] = 12.0, 0.0
    c.write([c.place(0, i) for i in range(L)], k, v)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 8.0  # a score of 12 against 0: e^12 = 162755 against 32767 ones
    sink = torch.full((1,), -1e4, device=DEV)
    o, lse = sa.kv_decode_fwd(handle(c), i32([0]), q, sink, q_per_seq=1)
    check_decode(c, [0], [1], 1, -1, 0, q, sink, o, lse)


# ---------------------------------------------------------------- together
def test_a_rollout_with_drafts_in_a_graph():
    """Plan, write, decode and verify captured once and replayed: every step's tables, outputs and tokens."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(9)
    B, most, Hkv, hq, V = 4, 3, 2, 8, 300
    c = ref.Pages(60, B, 12, Hkv, 16)
    h = handle(c)
    slots, T = i32([2, 0, 3, 1]), B * most
    new, drop = i32([37, 5, 16, 1]), i32([0] * B)
    total = 59 + T
    live, cu, places, pos = sa.kv_plan(h, slots, new, total)
    want = c.plan([2, 0, 3, 1], [0] * B, [37, 5, 16, 1], total)
    k, v = bf16(rng, total, Hkv, 64), bf16(rng, total, Hkv, 64)
    sa.kv_write(h, places, k.to(DEV), v.to(DEV))
    c.write(want[2], k.double().numpy(), v.double().numpy())

    k, v = (torch.empty((T, Hkv, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, sink = torch.empty((T, hq, 64), dtype=torch.bfloat16, device=DEV), dev(rng.randn(hq), torch.float32)
    x, y = torch.empty((T, V), device=DEV), torch.empty((T - B, V), device=DEV)
    drafts, u = i32([0] * (T - B)), torch.empty(T, device=DEV)
    temp = dev([1.0, 0.7, 0.0, 1.3], torch.float32)
    ws, vs = sa.kv_decode_workspace(h), sa.verify_workspace(x)

    def step():
        live, cu, places, pos = sa.kv_plan(h, slots, new, T, drop=drop)
        sa.kv_write(h, places, k, v)
        o, lse = sa.kv_decode_fwd(h, live, q, sink, q_per_seq=most, cu_rows=cu, workspace=ws)
        out = sa.verify_tokens(x, drafts, u, cu, draft_logits=y, temperature=temp, workspace=vs)
        drop.copy_(out[3])
        return (live, cu, places, pos), (o, lse), out

    counts, rejected = [3, 1, 2, 3], [0] * B
    new.copy_(i32(counts))
    state = [t.clone() for t in (h.block_table, h.seqlens, h.owner)]
    step()  # first calls outside the capture
    for t, s in zip((h.block_table, h.seqlens, h.owner), state):
        t.copy_(s)
    drop.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        planned, attended, verified = step()
    for turn in range(12):
        counts = [int(z) for z in rng.randint(1, most + 1, B)]
        new.copy_(i32(counts))
        R, D = sum(counts), sum(counts) - B
        for t in (k, v, q):
            t.copy_(bf16(rng, *t.shape))
        x.copy_(torch.from_numpy(rng.randn(T, V) * 2))
        y.copy_(x[:T - B] + torch.from_numpy(rng.randn(T - B, V)).to(DEV))
        rows = [r for b in range(B) for r in range(sum(counts[:b]), sum(counts[:b + 1]) - 1)]
        y[:D] = (x[rows].cpu() + torch.from_numpy(rng.randn(D, V) * 0.3).float()).to(DEV)
        pick = [int(rng.choice(V, p=torch.softmax(z.double(), -1).numpy())) for z in y[:D].cpu()]
        drafts.copy_(i32(pick + [0] * (T - B - D)))
        u.copy_(torch.from_numpy(rng.rand(T)))
        want = c.plan([2, 0, 3, 1], rejected, counts, T)
        graph.replay()
        for a, b in zip(planned, want):
            assert np.array_equal(a.cpu().numpy(), b), turn
        same_tables(c, h)
        c.write(want[2], k.double().cpu().numpy(), v.double().cpu().numpy())
        check_decode(c, [2, 0, 3, 1], counts, hq, -1, 0, q[:R], sink, attended[0][:R], attended[1][:, :R])
        at, rejected = 0, []
        for b, n in enumerate(counts):
            rows = slice(at, at + n)
            f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
            tokens, logp, acc, _, _ = ref.verify(f64(x[rows]), f64(y[at - b:at - b + n - 1]), pick[at - b:at - b + n - 1],
                                                 f64(u[rows]), float(temp[b]))
            assert verified[0][rows].tolist() == list(tokens) and int(verified[2][b]) == acc, (turn, b)
            assert np.abs(f64(verified[1][rows]) - logp).max() <= 2.0 ** -18
            rejected.append(n - 1 - acc)
            at += n
        assert verified[3].tolist() == rejected


def test_another_stream():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(10)
    c = shuffled(rng, [90, 200], 64, 2)
    h = handle(c)
    q, sink = bf16(rng, 2, 8, 64).to(DEV), dev(rng.randn(8), torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o, lse = sa.kv_decode_fwd(h, i32([1, 0]), q, sink, q_per_seq=1)
    side.synchronize()
    check_decode(c, [1, 0], [1, 1], 8, -1, 0, q, sink, o, lse)


def test_layers_share_one_table():
    """One plan for two layers whose pages are their own."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(11)
    one = sa.KVPages.empty(8, 2, 4, 2, page_size=32)
    two = sa.KVPages(torch.zeros_like(one.k_pages), torch.zeros_like(one.v_pages), one.block_table, one.seqlens, one.owner)
    live, cu, places, pos = sa.kv_plan(one, i32([1, 0]), i32([45, 3]), 48)
    q, sink = bf16(rng, 2, 4, 64).to(DEV), dev(rng.randn(4), torch.float32)
    for layer in (one, two):
        k, v = bf16(rng, 48, 2, 64), bf16(rng, 48, 2, 64)
        sa.kv_write(layer, places, k.to(DEV), v.to(DEV))
        o, lse = sa.kv_decode_fwd(layer, live, q, sink, q_per_seq=1)
        want, want_l = oracle.decode_forward(q.double().cpu().numpy(), k.double().numpy(), v.double().numpy(),
                                             sink.double().cpu().numpy(), [0, 45, 48], 1)
        assert np.abs(o.double().cpu().numpy() - want).max() < 2.0 ** -5
        assert np.abs(lse.double().cpu().numpy() - want_l).max() < 2.0 ** -14
