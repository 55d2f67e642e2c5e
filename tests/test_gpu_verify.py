"""Verification of drafted tokens: CUDA path vs the float64 oracle (needs a GB300).

A draft's test compares u q(d) with p(d), each off by a few 2^-22 of itself (the
sums' exponentials, their fp32 additions), so it may fall either way where the
two agree to 2^-18; the cases' seeds have none that does.  The drawn token is
decided where u times the whole lies among the cumulated masses, which are off
by well under TOL = 2^-24 of the target's whole (two-part exponents leave the
hardware exponential's 2^-22 of masses below 2^-13 each, and larger ones are
exact to 2^-40); the weights max(p - q, 0) are a part of it, so the bound
relative to their own whole is TOL over their sum.  The token given must own a
stretch that lies within the bound of u's place, and where no border is that
near it is the oracle's.  log p is off by the maximum's sums, a few 2^-22, and
by its own rounding, 2^-23 of its value: 2^-18 covers both.
"""
import numpy as np
import pytest
import torch

import oracle.pages_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TOL = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from sink_aware_masked_gb300 import build

    build.build()


def run(x, drafts, u, counts, y=None, temp=None, first=0):
    import sink_aware_masked_gb300 as sa

    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    f32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device=DEV)  # noqa: E731
    cu = np.concatenate(([0], np.cumsum(counts))) + first
    out = sa.verify_tokens(x, i32(drafts), f32(u), i32(cu), draft_logits=y, temperature=None if temp is None else f32(temp))
    return [a.cpu().numpy() for a in out]


def check(x, drafts, u, counts, y=None, temp=None, first=0):
    """Every entry against the oracle; returns how many tokens were drawn from what p leaves over q."""
    tokens, logp, accepted, rejected = run(x, drafts, u, counts, y, temp, first)
    u = np.asarray(u, dtype=np.float32).astype(np.float64)
    at, d, rest = first, 0, 0
    for b, n in enumerate(counts):
        if n == 0:
            assert accepted[b] == rejected[b] == 0
            continue
        rows, mine = slice(at, at + n), slice(d, d + n - 1)
        at, d = at + n, d + n - 1
        T = 1.0 if temp is None else float(np.float32(temp[b]))
        x64 = x[rows].double().cpu().numpy()
        want, want_logp, acc, weights, border = ref.verify(
            x64, None if y is None else y[mine].double().cpu().numpy(), drafts[mine], u[rows], T)
        assert border > 0 or acc == n - 1 or T == 0
        assert accepted[b] == acc and rejected[b] == n - 1 - acc, (b, acc, accepted[b])
        got = tokens[rows]
        if weights is None:
            assert np.array_equal(got, want)
        else:
            assert np.array_equal(np.delete(got, acc), np.delete(want, acc))
            rest += acc < n - 1
            cum = np.cumsum(weights)
            place, tol = min(max(u[rows][-1], 0.0), 1 - 2.0 ** -24) * cum[-1], TOL  # in units of the target's whole
            t = int(got[acc])
            assert weights[t] > 0 or tol > cum[-1], (b, t, "has no weight")
            assert (cum[t - 1] if t else 0.0) - tol <= place <= cum[t] + tol, (b, t)
            if np.abs(cum - place).min() > tol:
                assert t == want[acc], b
            p = ref.softmax(x64[acc], T)
            want_logp[acc] = p[1][t]
        with np.errstate(invalid="ignore"):
            near = np.abs(logp[rows] - want_logp) <= 2.0 ** -18 + 2.0 ** -23 * np.abs(want_logp)
        assert (near | (logp[rows] == want_logp) | (np.isnan(logp[rows]) & np.isnan(want_logp))).all(), b
    return rest


def case(rng, counts, V, dtype, proposal=True, spread=3.0, apart=1.0, pad=0, front=0):
    """Rows of any alignment with junk behind them; drafts from q, or from p."""
    R, D = sum(counts), sum(counts) - sum(n > 0 for n in counts)
    x = torch.from_numpy(rng.randn(front + R, V + pad) * spread).to(dtype).to(DEV)
    rows = np.concatenate([np.arange(a, a + n - 1) for a, n in zip(np.cumsum([0] + list(counts)), counts) if n > 1] or
                          [np.zeros(0)]).astype(int) + front
    y = (x[rows, :].float() + torch.from_numpy(rng.randn(D, V + pad) * apart).float().to(DEV)).to(dtype)
    z = (y if proposal else x[rows])[:, :V].double()
    drafts = torch.multinomial(torch.softmax(z, -1).cpu(), 1, generator=torch.Generator().manual_seed(1))[:, 0].numpy() \
        if D else np.zeros(0, dtype=np.int64)
    x[:, V:], y[:, V:] = 1e4, 1e4
    return x[:, :V], drafts, y[:, :V] if proposal else None, rng.rand(front + R)


SIZES = [([1], 1), ([2, 1, 3], 2), ([4, 4], 7), ([1, 5, 2, 9], 33), ([3, 3], 500), ([2], 4096), ([3, 2], 4099), ([2, 4], 8193),
         ([2], 32768), ([3], 50257), ([2, 2], 201088), ([2], 262144)]


@pytest.mark.parametrize("proposal", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,vocab", SIZES)
def test_parity(counts, vocab, dtype, proposal):
    rng = np.random.RandomState(vocab % 1000 + len(counts))
    for pad, temp in ((5, 1.0), (0, 0.6), (3, 1.7)):
        x, drafts, y, u = case(rng, counts, vocab, dtype, proposal, pad=pad)
        check(x, drafts, u, counts, y, [temp] * len(counts))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_entries(dtype):
    """Entries of 0 to 6 rows, every temperature in turn, flat and steep rows; draws from what p leaves over q among them."""
    rng = np.random.RandomState(2)
    counts = [int(c) for c in rng.randint(0, 7, 200)]
    temp = [[1.0, 0.0, 0.3, 2.0][i % 4] for i in range(200)]
    rest = 0
    for spread, apart in ((0.0, 0.5), (1.0, 0.3), (6.0, 2.0)):
        x, drafts, y, u = case(rng, counts, 1000, dtype, spread=spread, apart=apart)
        rest += check(x, drafts, u, counts, y, temp)
    assert rest > 50


def test_ties_and_greedy_entries():
    """Few values: the largest is the first of many, drafts that are another of them do not stand."""
    rng = np.random.RandomState(3)
    x = torch.from_numpy(rng.randint(0, 3, (12, 20011)) * 0.5).float().to(DEV)
    x[0], x[1] = 1.25, 0.0
    x[1, ::2] = -0.0  # one value
    best = x.argmax(-1).cpu().numpy()
    first = np.array([int(np.flatnonzero(r == r.max())[0]) for r in x.cpu().numpy()])
    drafts = first[[0, 1, 2, 4, 5, 6, 8, 9, 10]].copy()
    drafts[4] = int(np.flatnonzero(x[5].cpu().numpy() == 1.0)[1])
    tokens, logp, acc, rej = run(x, drafts, rng.rand(12), [4, 4, 4], temp=[0.0] * 3)
    assert acc.tolist() == [3, 1, 3] and rej.tolist() == [0, 2, 0]
    assert tokens.tolist() == list(first[:6]) + [-1, -1] + list(first[8:]), best
    check(x, drafts, rng.rand(12), [4, 4, 4], x[[0, 1, 2, 4, 5, 6, 8, 9, 10]].contiguous(), [1.0, 0.0, 1e30])


def test_equal_rows_always_stand():
    """p = q: a draft stands whatever u is, but for the sums' rounding (the rows lie at different alignments)."""
    rng = np.random.RandomState(4)
    x, drafts, y, u = case(rng, [8] * 6, 5003, torch.bfloat16, apart=0.0)
    u[:] = 1 - 2.0 ** -17
    assert run(x, drafts, u, [8] * 6, y)[2].tolist() == [7] * 6


def test_masked_rows_and_what_is_not_valid():
    inf, nan = float("inf"), float("nan")
    rng = np.random.RandomState(5)
    counts = [3] * 12
    x, drafts, y, u = case(rng, counts, 3000, torch.float32, apart=0.0)
    u[:] = 0.25
    temp = [1.0] * 12
    x[3 * 0] = -inf                       # nothing allowed in a row with a draft: nothing stands, nothing is drawn
    x[3 * 1 + 2] = -inf                   # nor in the last row
    x[3 * 2 + 1, 17] = nan
    x[3 * 3 + 2, 2999] = inf
    y[2 * 4 + 1, 5] = nan
    y[2 * 5 + 1] = -inf
    temp[6], temp[7] = nan, -1.0
    drafts[2 * 8], drafts[2 * 9 + 1] = 3000, -1
    x[3 * 10 + 1, :2990] = -inf           # ten allowed
    x[3 * 10 + 1, 2990:] = 0.0
    drafts[2 * 10 + 1] = 7
    u[3 * 11 + 2] = nan
    tokens, logp, acc, rej = run(x, drafts, u, counts, y, temp)
    assert acc.tolist() == [0, 2, 1, 2, 1, 1, 0, 0, 0, 1, 1, 2]
    assert rej.tolist() == [2 - a for a in acc]
    ends = [tokens[3 * b + a] for b, a in enumerate(acc)]
    assert ends[:8] == [-1] * 8 and min(ends[8:]) >= 0 and 2990 <= ends[10] < 3000
    last = [logp[3 * b + a] for b, a in enumerate(acc)]
    assert np.isneginf(last[:2]).all() and np.isnan(last[2:8]).all() and np.isfinite(last[8:]).all()
    assert abs(last[10] + np.log(10)) < 1e-6
    for b, a in enumerate(acc):
        assert (tokens[3 * b + a + 1:3 * b + 3] == -1).all() and (logp[3 * b + a + 1:3 * b + 3] == 0).all()
        assert np.array_equal(tokens[3 * b:3 * b + a], drafts[2 * b:2 * b + a])
    check(x[24:33], drafts[16:22], u[24:33], counts[8:11], y[16:22], temp[8:11])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("level", [0.0, 3e4])
def test_masks_of_the_lowest_finite_value(dtype, level):
    """Masked by the type's lowest value instead of -inf, in one row or both, drafts among the masked tokens."""
    rng = np.random.RandomState(10)
    counts = [3] * 8
    low = torch.finfo(dtype).min
    x, drafts, y, u = case(rng, counts, 3001, dtype)
    x, y = (x.float() + level).to(dtype), (y.float() + level).to(dtype)
    x[:9, 40:], y[4:10, 60:] = low, low
    drafts[[0, 1, 8, 9]] = [2000, 39, 2500, 3000]  # masked in p; allowed in it; masked in q alone: they stand
    tokens, logp, acc, rej = run(x, drafts, u, counts, y)
    assert acc[0] == 0 and tokens[0] < 40 and acc[4] == 2
    check(x, drafts, u, counts, y)
    check(x, drafts, u, counts)


def test_extreme_temperatures():
    rng = np.random.RandomState(11)
    temp = [2e-38, 1e-30, 1e-6, 1e4, 1e30, 1e36]  # (1e-38 is subnormal, and counts as 0)
    counts = [3] * 6
    for V in (900, 20000):
        x, drafts, y, u = case(rng, counts, V, torch.float32)
        x[:, 5], y[:, 5] = torch.finfo(torch.float32).min, -float("inf")
        check(x, drafts, u, counts, y, temp)
        check(x, drafts, u, counts, None, temp)


def test_random_numbers_at_their_ends():
    rng = np.random.RandomState(6)
    x, drafts, y, u = case(rng, [2] * 6, 4001, torch.float32)
    drafts[:] = 4000
    y[:, 4000] = 50.0  # q is 1 there, p is not: nothing stands but with u = 0
    u[:] = [0.9, 0.0, 0.9, -3.0, 0.9, 1.0, 0.9, np.float32(0.99999994), 0.0, 0.5, 0.9, 2.0]
    tokens, logp, acc, rej = run(x, drafts, u, [2] * 6, y)
    assert acc.tolist() == [0, 0, 0, 0, 1, 0]
    assert tokens[0] == tokens[2] == 0 and tokens[4] == tokens[6] == tokens[10]
    check(x, drafts, u, [2] * 6, y)


def test_rows_outside_the_entries_are_left_alone():
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(7)
    x, drafts, y, u = case(rng, [2, 0, 3], 700, torch.float32, front=2)
    assert check(x, drafts, u, [2, 0, 3], y, first=2) >= 0
    x = torch.cat((x, torch.full((3, 700), float("nan"), device=DEV)))
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    tokens, logp = torch.full((10,), 77, dtype=torch.int32, device=DEV), torch.full((10,), 77.0, device=DEV)
    out = sa.verify_tokens(x, i32(drafts), torch.rand(10, device=DEV), i32([2, 4, 4, 7]), draft_logits=y, tokens=tokens,
                           logp=logp)
    assert out[0] is tokens and out[1] is logp
    rest = [0, 1, 7, 8, 9]
    assert (tokens[rest] == 77).all() and (logp[rest] == 77).all() and (tokens[2:7] < 700).all()


def test_no_rows_and_no_entries():
    import sink_aware_masked_gb300 as sa

    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    x, u = torch.zeros((0, 9), device=DEV), torch.zeros(0, device=DEV)
    tokens, logp, acc, rej = sa.verify_tokens(x, i32([]), u, i32([0, 0, 0]))
    assert tokens.numel() == 0 and acc.tolist() == [0, 0] and rej.tolist() == [0, 0]
    sa.verify_tokens(torch.zeros((2, 9), device=DEV), i32([]), torch.zeros(2, device=DEV), i32([0]))


@pytest.mark.parametrize("proposal", [True, False])
def test_tokens_follow_the_target(proposal):
    """100 k entries: what is emitted first is distributed as p (5 sigma of each count)."""
    rng = np.random.RandomState(8)
    V, N = 7, 4000
    row = torch.from_numpy(rng.randn(1, V) * 1.5).float().to(DEV)
    q = torch.from_numpy(rng.randn(1, V) * 1.5).float().to(DEV)
    count = np.zeros(V)
    for _ in range(25):
        x, y = row.expand(2 * N, V).contiguous(), q.expand(N, V).contiguous()
        drafts = rng.choice(V, N, p=torch.softmax(q[0].double(), 0).cpu().numpy() if proposal else None)
        tokens = run(x, drafts, rng.rand(2 * N), [2] * N, y if proposal else None)[0]
        count += np.bincount(tokens[::2], minlength=V)
    p = torch.softmax(row[0].double(), 0).cpu().numpy()
    n = 25 * N
    assert (np.abs(count - n * p) <= 5 * np.sqrt(n * p * (1 - p))).all(), (count / n, p)


def test_results_repeat():
    rng = np.random.RandomState(9)
    x, drafts, y, u = case(rng, [4] * 40, 33001, torch.bfloat16)
    first = run(x, drafts, u, [4] * 40, y)
    for _ in range(3):
        assert all(np.array_equal(a, b) for a, b in zip(first, run(x, drafts, u, [4] * 40, y)))
