"""Token sampling: CUDA path vs the float64 oracle (needs a GB300).

A token is decided where u times the kept mass lies among the cumulated
masses.  The kernel's exponentials are off by a few 2^-22 each (the exponent
is rounded to 2^-24 of its value, up to about 20 where mass still counts, and
the hardware exponential adds 2^-22), so a cumulated mass is off by well under
TOL = 2^-18 of the whole: the token given must own a stretch of the cumulated
mass that lies within TOL of u's place, and where no border is that near it is
the oracle's.  The logarithms are held to the same bound (plus their own
rounding, 2^-23 of their value).  A cut of top-p or min-p nearer than rounding
to a border may fall on either side of one token; the cases' seeds have none
that shows.
"""
import numpy as np
import pytest
import torch

import oracle.rollout_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TOL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from sink_aware_masked_gb300 import build

    build.build()


def run(x, u, t, k, p, m):
    import sink_aware_masked_gb300 as sa

    f = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device=DEV)  # noqa: E731
    out = sa.sample_tokens(x, f(u), temperature=f(t), top_k=torch.tensor(np.asarray(k), dtype=torch.int32, device=DEV),
                           top_p=f(p), min_p=f(m))
    return [a.cpu().numpy() for a in out]


def check(x, u, t, k, p, m):
    """Every row against the oracle."""
    got = run(x, u, t, k, p, m)
    xs = x.double().cpu().numpy()
    r32 = lambda a: np.asarray(a, dtype=np.float32).astype(np.float64)  # noqa: E731
    u, t, p, m = r32(u), r32(t), r32(p), r32(m)
    for r in range(x.shape[0]):
        row = xs[r], u[r], t[r], int(k[r]), p[r], m[r]
        token = int(got[0][r])
        bad = ref.sample_invalid(*row)
        if bad is not None:
            assert token == -1 and all(np.array_equal(a[r], np.float32(bad), equal_nan=True) for a in got[1:])
            continue
        z, total, kept, cum, at = ref.kept_tokens(*row)
        i = int(np.searchsorted(kept, token))
        assert i < len(kept) and kept[i] == token, (r, token, "is not kept")
        lo, hi = (cum[i - 1] if i else 0.0) / cum[-1], cum[i] / cum[-1]
        assert lo - TOL <= at / cum[-1] <= hi + TOL, (r, token, lo, at / cum[-1], hi)
        if len(kept) == 1 or np.abs(cum[:-1] - at).min() > TOL * cum[-1]:
            assert token == ref.sample(*row)[0], r
        for a, b in ((got[1][r], z[token] - np.log(total)), (got[2][r], z[token] - np.log(cum[-1]))):
            assert abs(a - b) <= TOL + 2.0 ** -23 * abs(b), (r, a, b)


SIZES = [(1, 1), (3, 2), (2, 7), (5, 33), (4, 500), (2, 4096), (3, 4099), (2, 8193), (2, 32768), (2, 50257), (1, 201088),
         (1, 262144)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_parity(rows, vocab, dtype):
    rng = np.random.RandomState(vocab % 1000 + rows)
    combos = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.1), (0.9, 300, 0.8, 0.01),
              (0.0, 0, 1.0, 0.0), (1.0, 1, 0.5, 0.0), (1.0, 5000, 0.999, 0.0), (1.0, 0, 0.05, 0.0), (2.0, 7, 0.0, 0.0)]
    # a row stride that leaves rows at any alignment, and junk behind the row's end
    pad = 5
    x = torch.from_numpy(rng.randn(rows * len(combos), vocab + pad) * 3).to(dtype).to(DEV)
    x[:, vocab:] = 1e4
    t, k, p, m = (np.array([c[i] for c in combos] * rows) for i in range(4))
    check(x[:, :vocab], rng.rand(rows * len(combos)), t, k, p, m)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(dtype):
    """Rows of few values: the cuts of top-k and top-p lie among equal logits, thousands of them."""
    rng = np.random.RandomState(3)
    V = 20011
    x = torch.from_numpy(rng.randint(0, 3, (12, V)) * 0.5).to(dtype).to(DEV)
    x[0] = 1.25   # all equal
    x[1] = 0.0
    x[1, ::2] = -0.0  # one value
    k = [700, 12345, 0, 5, 20010, 0, 0, 9000, 1, 0, 3000, 0]
    p = [1.0, 1.0, 0.123, 1.0, 1.0, 0.9, 0.5, 0.3, 1.0, 0.7, 0.99, 0.0]
    check(x, rng.rand(12), np.ones(12), k, p, np.zeros(12))


def test_masked_rows_and_what_is_not_valid():
    x = torch.randn((14, 3000), device=DEV)
    x[0] = float("-inf")                    # nothing allowed
    x[1] = float("-inf")
    x[1, 2777] = -50.0                      # one allowed
    x[2, 5] = float("nan")
    x[3, 2999] = float("inf")
    x[4] = float("nan")
    x[5, :2990] = float("-inf")             # ten allowed, top-k of 100
    x[6, 1:] = torch.finfo(torch.float32).min
    x[13, 3] = -float("nan")
    t = [1.0] * 14
    t[7], t[8], t[9] = -1.0, float("inf"), float("nan")
    p = [1.0] * 14
    p[10] = float("nan")
    m = [0.0] * 14
    m[11] = float("nan")
    u = [0.5] * 14
    u[12] = float("nan")
    tok, logp, logq = run(x, u, t, [100] * 14, p, m)
    assert tok[0] == -1 and np.isneginf(logp[0]) and np.isneginf(logq[0])
    assert tok[1] == 2777 and abs(logp[1]) < 1e-6 and abs(logq[1]) < 1e-6
    assert tok[5] >= 2990 and tok[6] == 0 and logp[6] == 0
    for r in (2, 3, 4, 7, 8, 9, 10, 11, 12, 13):
        assert tok[r] == -1 and np.isnan(logp[r]) and np.isnan(logq[r]), r
    check(x, u, t, [100] * 14, p, m)


def test_ends_of_u_and_of_the_parameters():
    x = torch.tensor([[0.0, 1.0, 2.0, -1.0, float("-inf")]], device=DEV).repeat(8, 1)
    tok, logp, logq = run(x, [0, 1 - 2.0 ** -24, -3, 7, 0.5, 0.5, 0.5, 0.5], [1, 1, 1, 1, 1e-30, 1e30, 1, 1],
                          [0, 0, 0, 0, 0, 0, -5, 10 ** 9], [1] * 7 + [2], [0, 0, 0, 0, 0, 0, 1.0, 9.0])
    assert tok.tolist() == [0, 3, 0, 3, 2, 2, 2, 2]
    assert abs(logp[5] - np.log(0.25)) < 1e-6 and logp[4] == 0 and logq[6] == 0 and logq[7] == 0


def test_the_largest_temperatures():
    """1e36 still is one, with masked logits of -inf and of fp32's lowest value; what lies beyond is refused."""
    rng = np.random.RandomState(6)
    x = torch.from_numpy(rng.randn(10, 40009)).float().to(DEV)
    x[:, 5::3] = float("-inf")
    x[:, 6::3] = torch.finfo(torch.float32).min
    t = [1e36] * 6 + [1e37, 1.3e38, 3.4e38, 1e36]
    k, p, m = [0, 100, 0, 0, 9000, 30, 0, 0, 0, 0], [1, 1, 0.9, 1, 0.5, 0.4, 1, 1, 0.9, 0.01], [0, 0, 0, 0.1] + [0] * 6
    tok, logp, _ = run(x, [0.5] * 10, t, k, p, m)
    assert (tok[[6, 7, 8]] == -1).all() and np.isnan(logp[[6, 7, 8]]).all() and (tok[[0, 1, 2, 3, 4, 5, 9]] >= 0).all()
    check(x, rng.rand(10), t, k, p, m)


def test_rows_stand_alone_and_repeat_bit_by_bit():
    rng = np.random.RandomState(5)
    x = torch.from_numpy(rng.randn(300, 10007) * 3).float().to(DEV)
    u, t, k, p, m = rng.rand(300), rng.uniform(0, 2, 300), rng.randint(0, 400, 300), rng.uniform(0.2, 1.2, 300), np.zeros(300)
    a = run(x, u, t, k, p, m)
    b = run(x, u, t, k, p, m)
    assert all(np.array_equal(i, j) for i, j in zip(a, b))
    for r in (0, 17, 299):
        one = run(x[r:r + 1], u[r:r + 1], t[r:r + 1], k[r:r + 1], p[r:r + 1], m[r:r + 1])
        assert all(i[0] == j[r] for i, j in zip(one, a))
    check(x[:40], u[:40], t[:40], k[:40], p[:40], m[:40])


def test_frequencies():
    """Many u over one row: each token's share is its probability (the u are a grid, so within two grid steps)."""
    probs = np.array([0.5, 0.25, 0.125, 0.125])
    n = 4096
    x = torch.from_numpy(np.log(probs)).float().to(DEV)[None].repeat(n, 1)
    tok, _, _ = run(x, (np.arange(n) + 0.5) / n, np.ones(n), np.zeros(n), np.ones(n), np.zeros(n))
    assert np.abs(np.bincount(tok, minlength=4) / n - probs).max() <= 2 / n


def test_captured_and_replayed():
    import sink_aware_masked_gb300 as sa

    x, u = torch.zeros((4, 5000), device=DEV), torch.zeros(4, device=DEV)
    kw = dict(temperature=torch.full((4,), 0.8, device=DEV), top_k=torch.full((4,), 40, dtype=torch.int32, device=DEV),
              top_p=torch.full((4,), 0.9, device=DEV), min_p=torch.zeros(4, device=DEV))
    outs = [torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)]
    names = dict(zip(("tokens", "logp", "logq"), outs))
    sa.sample_tokens(x, u, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sample_tokens(x, u, **kw, **names)
    for seed in range(5):
        torch.manual_seed(seed)
        x.copy_(torch.randn(4, 5000) * 2)
        u.copy_(torch.rand(4))
        graph.replay()
        want = sa.sample_tokens(x, u, **kw)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("k,p,m", [(200, 0.95, 0.0), (3000, 1.0, 0.0), (9000, 0.9, 0.01), (0, 0.95, 0.02), (0, 0.4, 0.0),
                                   (0, 1.0, 1e-6), (40, 1.0, 0.3), (2048, 0.999, 0.0)])
def test_rows_by_cta_and_by_cluster(rows, k, p, m):
    """Batches on both sides of the rules for the cluster's size, lists on both sides of what is sorted at once."""
    rng = np.random.RandomState(rows + k)
    x = torch.from_numpy(-1.3 * np.log(1 + rng.rand(rows, 30011) * 30011) + rng.randn(rows, 30011)).float().to(DEV)
    x[::3, 700:] = float("-inf")  # all that is allowed lies in one place
    check(x, rng.rand(rows), np.full(rows, 0.9), [k] * rows, [p] * rows, [m] * rows)


@pytest.mark.parametrize("t", [0.01, 1.0, 20.0])
def test_cuts_far_below_the_largest_logit(t):
    """One logit far above the rest: the first histogram's range ends before the cut, whose step then holds all below."""
    rng = np.random.RandomState(9)
    x = torch.from_numpy(rng.randn(4, 40003)).float().to(DEV)
    x[:, 77] = 45.0 * max(t, 1.0)
    check(x, [0.1, 0.9, 0.5, 1 - 2.0 ** -24], [t] * 4, [3000, 20000, 39000, 5000], [1.0, 1.0, 0.999, 1.0], [0.0] * 4)


def sentinel_outputs(rows):
    return dict(tokens=torch.full((rows,), -77, dtype=torch.int32, device=DEV),
                logp=torch.full((rows,), 7e7, device=DEV), logq=torch.full((rows,), 7e7, device=DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab,peak,height,gap", [
    (16384, 12000, 28.5, 16384), (201088, 150000, 30.0, 16384), (201088, 3, 28.5, 201088), (201088, 201080, 28.5, 201088),
    (40009, 20000, 30.0, 40009)])
@pytest.mark.parametrize("k,m", [(0, 0.0), (-9, 0.0), (0, 1e-30)])
def test_masses_that_count_together_alone(vocab, peak, height, gap, k, m, dtype):
    """Logits more than 27.7 below the largest have masses under 2^-40 of its mass, yet thousands of them together
    have more: where u lies among them the row still gets a token, the first one for u = 0.  `gap` logits from the
    first on are 0 (the others are masked), one is `height`; k < 0: all but -k of the allowed ones are kept."""
    import sink_aware_masked_gb300 as sa

    u = [0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, -3.0, 7.0]
    n = len(u)
    x = torch.full((n, vocab), float("-inf"), dtype=dtype, device=DEV)
    x[:, :gap] = 0
    x[:, peak] = height
    full = lambda v, t=torch.float32: torch.full((n,), v, dtype=t, device=DEV)  # noqa: E731
    top_k = gap + k if k < 0 else 0
    out = sentinel_outputs(n)
    sa.sample_tokens(x, torch.tensor(u, device=DEV), temperature=full(1.0), top_k=full(top_k, torch.int32),
                     top_p=full(1.0), min_p=full(m), **out)
    tokens = out["tokens"].tolist()
    # every output is written; a logarithm is off by TOL at most (see above), so one of a probability is below TOL
    assert all(0 <= t < vocab for t in tokens) and (out["logp"] <= TOL).all() and (out["logq"] <= TOL).all(), tokens
    # a warp's masses together reach 2^-40 from the first logits on, so that u = 0 finds the very first
    assert tokens[0] == tokens[4] == (0 if peak != 3 else tokens[0]) and tokens[2] == peak
    check(x, u, [1.0] * n, [top_k] * n, [1.0] * n, [m] * n)


@pytest.mark.parametrize("vocab", [16384, 40009, 262144])
@pytest.mark.parametrize("t", [1.0, 0.001, 300.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_around_the_end_of_the_fused_exponents(sign, t, vocab):
    """Where |x| log2(e) / T passes 2^20 the exponent is computed another way: a thread whose maximum crosses the
    border, up or down, keeps the whole of what it has summed before.  The logits are spaced as fp32 has them there
    (2^-24 of their value, 0.06 T), all within 4 T of the border; nothing below is cut but where k says so."""
    rng = np.random.RandomState(11)
    t32, m = float(np.float32(t)), np.linspace(-4.0, 4.0, vocab)
    edge = sign * 2.0 ** 20 / np.log2(np.e) * t32
    rows = [m, m[::-1], rng.permutation(m)]
    for at in (0.1, 0.3, 0.6, 0.9):  # two levels, one on either side
        rows += [np.where(np.arange(vocab) < at * vocab, lo, -lo) for lo in (-1.0, -0.1)]
    x = torch.from_numpy(edge + np.stack(rows) * t32).float().to(DEV)
    r = len(x)
    for k, floor in ((0, 0.0), (vocab - 7, 0.0), (0, 1e-9), (100, 0.0)):
        check(x, rng.rand(r), [t] * r, [k] * r, [1.0] * r, [floor] * r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [100, 5000, 40009])
def test_min_p_of_one_keeps_the_largest_alone(vocab, dtype):
    """Also where a smaller logit's e is 1 to fp32's, or to 64 bits', last place: a large temperature, a neighbouring
    fp32 value.  So what min-p keeps of the oracle's other choices is told by the logits, not by their e."""
    rng = np.random.RandomState(vocab)
    x = torch.from_numpy(rng.randn(14, vocab)).to(dtype).to(DEV)
    if dtype == torch.float32:
        x[7:] = 1.0 + 2.0 ** -23 * torch.from_numpy(rng.randint(0, 3, (7, vocab))).float().to(DEV)
    else:
        x[7:] = torch.from_numpy(rng.randint(0, 3, (7, vocab))).to(dtype).to(DEV)
    k = [0, 50, 4000, 0, 30, 4500, 0] * 2
    p = [1.0, 1.0, 1.0, 0.9, 0.9, 0.99999, 0.0] * 2
    for t in (1e10, 1e36, 40.0):
        for m in (1.0, 3.0):
            u = rng.rand(14).astype(np.float32)
            token, logp, logq = run(x, u, [t] * 14, k, p, [m] * 14)
            for r, row in enumerate(x.double().cpu().numpy()):
                kept = ref.kept_tokens(row, 0.0, float(np.float32(t)), k[r], float(np.float32(p[r])), 0.0)[2]
                kept = kept[row[kept] == row.max()]
                n = len(kept)
                assert token[r] == kept[int(float(u[r]) * n)], (t, m, r, token[r], n)
                assert abs(logq[r] + np.log(n)) <= TOL + 2.0 ** -23 * np.log(n)
                total = np.exp((row - row.max()) / float(np.float32(t))).sum()
                assert abs(logp[r] + np.log(total)) <= TOL + 2.0 ** -23 * np.log(total)


@pytest.mark.parametrize("vocab", [16384, 16385, 32768, 32769])
@pytest.mark.parametrize("k,p,m", [(200, 0.95, 0.0), (3000, 1.0, 0.0), (9000, 0.9, 0.01), (0, 0.95, 0.02), (0, 0.4, 0.0),
                                   (0, 1.0, 1e-6), (40, 1.0, 0.3), (2048, 0.999, 0.0), (0, 1.0, 0.0), (1, 1.0, 0.0)])
def test_clusters_of_every_size(k, p, m, vocab):
    """Vocabularies on both sides of the borders between one, two and four CTAs a row, at any alignment of the rows;
    lists on both sides of what is sorted at once."""
    rng = np.random.RandomState(vocab + k)
    x = -1.3 * np.log(1 + rng.rand(6, vocab + 3) * vocab) + rng.randn(6, vocab + 3)
    x[::3, 700:] = float("-inf")  # all that is allowed lies in one place
    for dtype in (torch.float32, torch.float16):
        check(torch.from_numpy(x).to(dtype).to(DEV)[:, :vocab], rng.rand(6), [0.9] * 6, [k] * 6, [p] * 6, [m] * 6)
