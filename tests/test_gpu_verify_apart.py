"""Verification of drafts whose model and target disagree: CUDA path vs the float64 oracle (needs a GB300).

A token that one row makes likely can have any logit in the other row: a mask
of whatever finite value, or one far below the other row's favourite at a low
temperature.  Every entry here ends at a refused draft, so that its last token
is drawn from max(p - q, 0); tolerances are those of the verification's other
tests (a place drawn is compared to 2^-24 of the target's whole).
"""
import numpy as np
import pytest
import torch

import oracle.pages_ref as ref
from tests.test_gpu_verify import DEV, built, check, run  # noqa: F401

pytestmark = pytest.mark.gpu
TEMPERATURES = [0.05, 0.1, 0.2, 0.3, 0.6, 0.7, 0.8, 0.9, 1.0, 1.2]


def softmax(x, temps):
    return torch.softmax(x.double().cpu() / torch.tensor(np.float32(temps), dtype=torch.float64)[:, None], -1)


def refused(x, y, temps, rng):
    """One draft an entry (rows 2 b and 2 b + 1 of x, row b of y), the one that q likes best beyond p: none stands."""
    p, q = softmax(x[::2], temps), softmax(y, temps)
    drafts = (q - p).argmax(-1)
    at = torch.arange(len(temps))
    assert (q[at, drafts] > 1.01 * p[at, drafts]).all()  # u is 0.999 or more
    u = np.stack((0.999 + 0.0009 * rng.rand(len(temps)), rng.rand(len(temps))), -1).reshape(-1)
    assert check(x, drafts.numpy(), u, [2] * len(temps), y, temps) == len(temps)


@pytest.mark.parametrize("vocab", [4, 37, 4099, 50257])
@pytest.mark.parametrize("dtype,mask", [(t, m) for t in (torch.float32, torch.bfloat16, torch.float16)
                                        for m in (-100.0, -200.0, -1e4, -65504.0, -1e9)
                                        if t is not torch.float16 or m >= -65504.0])
@pytest.mark.parametrize("side", ["target", "draft", "both"])
def test_finite_masks_of_one_row(side, dtype, mask, vocab):
    """The other row's favourite is masked, and a third of the tokens with it; "both": each row masks its own."""
    rng = np.random.RandomState(vocab + int(-mask) % 97)
    temps = [t for t in TEMPERATURES for _ in range(4 if vocab < 1000 else 1)]
    B = len(temps)
    x, y = (torch.from_numpy(rng.randn(n, vocab) * 2).to(dtype).to(DEV) for n in (2 * B, B))
    for b in range(B):
        best = int((x[2 * b] if side == "draft" else y[b]).argmax())
        masked = torch.from_numpy(rng.rand(vocab) < 0.3).to(DEV)
        masked[best] = True
        masked[(best + 1) % vocab] = False
        if side == "both":
            x[2 * b, (best + 1) % vocab] = 9.0
            y[b, best], y[b, (best + 1) % vocab] = 9.0, mask
        if side == "draft":
            x[2 * b, best] = 9.0
            y[b, masked] = mask
        else:
            x[2 * b, masked] = mask
    refused(x, y, temps, rng)


def test_masks_drawn_over_a_grid():
    """Small rows, a grid of the random numbers: a token masked in the target is never drawn, one masked in the draft is."""
    rows = [((-1e9, 2, 1, 0), (3, 0.5, 1, 1.5)), ((-1e4, 2, 1, 0), (3, 0.5, 1, 1.5)), ((-100, 2, 1, 0), (3, 0.5, 1, 1.5)),
            ((3, 2, 1, 0), (-1e9, 2, 1, 0)), ((3, 2, 1, 0), (-1e4, 2, 1, 0)), ((3, 2, 1, 0), (-100, 2, 1, 0))]
    for x, y in rows:
        for T in TEMPERATURES:
            N = 64
            xs, ys = (torch.tensor([r], device=DEV).expand(n, 4).float().contiguous() for r, n in ((x, 2 * N), (y, N)))
            drafts = np.full(N, 0 if x[0] < 0 else 1)  # q likes it more than p does
            u = np.stack((np.full(N, 0.9999), (np.arange(N) + 0.37) / N), -1).reshape(-1)
            assert check(xs, drafts, u, [2] * N, ys, [T] * N) == N


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [0.05, 0.1, 0.7, 1.0])
@pytest.mark.parametrize("vocab", [5, 3001])
def test_favourites_that_the_other_row_has_far_below(vocab, T, dtype):
    """Each row's favourite lies 0.1 to 800 log2 units below the other's: in the target, in the draft row, in both."""
    rng = np.random.RandomState(vocab)
    gaps = np.linspace(0.1, 800, 240) * T * np.log(2)
    B = len(gaps)
    x, y = (torch.from_numpy(rng.randn(n, vocab) * 0.5).to(dtype).to(DEV) for n in (2 * B, B))
    for b, gap in enumerate(gaps):
        side = b % 3
        x[2 * b, 2], y[b, 2] = 3.0, 3.0  # a token that both like
        x[2 * b, 0], y[b, 1] = 4.0, 4.0
        x[2 * b, 1] = 3.0 - gap if side != 1 else 2.5
        y[b, 0] = 3.0 - gap if side != 0 else 2.5
    refused(x, y, [T] * B, rng)


def test_rows_that_have_nothing_in_common():
    """Half of the vocabulary masked in one row, the other half in the other, by values of every size."""
    rng = np.random.RandomState(1)
    temps = TEMPERATURES * 6
    B, V = len(temps), 2500
    x, y = (torch.from_numpy(rng.randn(n, V)).float().to(DEV) for n in (2 * B, B))
    for b in range(B):
        low = -float(10.0 ** (1.5 + 8 * rng.rand()))
        x[2 * b, :V // 2], y[b, V // 2:] = low, low * 1.5
    refused(x, y, temps, rng)


@pytest.mark.parametrize("entries", [3, 30, 900])
@pytest.mark.parametrize("proposal", [True, False])
def test_offsets_outside_the_rows(entries, proposal):
    """Offsets that begin below 0 and end behind the rows, also with more entries than rows: the rows that are there count,
    and nothing is written around the workspace."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(entries)
    R, V = 12, 300
    x = torch.from_numpy(rng.randn(R, V)).float().to(DEV)
    drafts = torch.from_numpy(rng.randint(0, V, R)).int().to(DEV)
    y = torch.from_numpy(rng.randn(R, V)).float().to(DEV) if proposal else None
    u = torch.from_numpy(rng.rand(R)).float().to(DEV)
    # rows -3 .. 1 (of which 0 and 1 are there, behind three drafts of rows that are not), empty entries, 2 .. 6, 7 .. 19
    cu = [-3] + [2] * (entries - 2) + [7, 20]
    want = sa.verify_tokens(x, drafts[3:], u, torch.tensor([0, 2, 7, 12], dtype=torch.int32, device=DEV),
                            draft_logits=None if y is None else y[3:])
    size = sa.verify_workspace(x).numel()
    room = torch.full((size + (2 << 16),), 91, dtype=torch.uint8, device=DEV)
    got = sa.verify_tokens(x, drafts, u, torch.tensor(cu, dtype=torch.int32, device=DEV), draft_logits=y,
                           workspace=room[1 << 16:-(1 << 16)])
    assert (room[:1 << 16] == 91).all() and (room[-(1 << 16):] == 91).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(got[2:], want[2:]):
        assert a[[0, -2, -1]].tolist() == b.tolist() and (a[1:-2] == 0).all()


@pytest.mark.parametrize("T", [0.05, 1.0, 2.5])
@pytest.mark.parametrize("proposal", [True, False])
def test_probabilities_and_random_numbers_near_zero(proposal, T):
    """p(d) and q(d) from 1 to 2^-1150 of their largest, u from 0 and 2^-126 on: a draft stands if log u + log q < log p.
    Random numbers lie 2^-19 of themselves and more from the border (either side may be given up to 2^-20); what lies
    below 2^-1074 of the largest counts as 0."""
    rng = np.random.RandomState(int(T * 20) + proposal)
    B, V = 4000, 4
    T = float(np.float32(T))
    x, y = torch.zeros((2 * B, V)), torch.zeros((B, V))
    for t in (x[::2], y):
        t[:, 1:3] = -torch.from_numpy(rng.rand(B, 2)).float() * T
        t[:, 3] = -torch.from_numpy(1150 * rng.rand(B) ** rng.randint(1, 4, B) * np.log(2) * T).float()

    def log2_of(t):  # (log2 of token 3's share, whether it counts as more than 0); no power below 2^-1022 is taken
        z = t.double().numpy() / T / np.log(2)
        z -= z.max(-1, keepdims=True)
        return z[:, 3] - np.log2((2.0 ** np.maximum(z, -1000)).sum(-1)), z[:, 3] > -1074

    (lp, p_is), (lq, q_is) = log2_of(x[::2]), log2_of(y) if proposal else (np.zeros(B), np.ones(B, dtype=bool))
    away = rng.choice([-1, 1], B) * 2.0 ** rng.uniform(-19, 2, B)  # from the border, relative to it
    border = lp - lq + np.log2(np.maximum(1 + away, 2.0 ** -30))
    lu = np.where((border < 0) & (border >= -126) & (rng.rand(B) < 0.8), border, rng.uniform(-126, 0, B))
    u = np.float32(np.where(rng.rand(B) < 0.2, 0.0, 2.0 ** np.maximum(lu, -126.0)))
    with np.errstate(divide="ignore"):
        lu = np.log2(u.astype(np.float64))
    far = np.abs(2.0 ** np.clip(lu + lq - lp, -30, 30) - 1) > 2.0 ** -19.5  # (rounding u may have brought one nearer)
    far &= (u < 0.9999999) & (np.abs(x[::2, 3].double().numpy() / T / np.log(2) + 1074) > 0.01)
    far &= np.abs(y[:, 3].double().numpy() / T / np.log(2) + 1074) > 0.01
    stands = p_is & (~q_is | (lu + lq < lp))
    assert far.sum() > 0.95 * B and 0.2 * B < stands.sum() < 0.8 * B
    assert (stands & (u == 0) & (lp < -126)).sum() > 20 and (~stands & (u == 0)).sum() > 5
    all_u = np.stack((u, rng.rand(B).astype(np.float32)), -1).reshape(-1)
    accepted = run(x.to(DEV), np.full(B, 3), all_u, [2] * B, y.to(DEV) if proposal else None, [T] * B)[2]
    assert np.array_equal(accepted[far], stands[far].astype(np.int32)), np.flatnonzero(far & (accepted != stands))[:9]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [3, 300, 20011])
def test_rows_that_agree_but_for_one_token(vocab, dtype):
    """q gives one token 2^-13 to 2^-33 more than p does, and that is the draft: what is left, as much, is shared among all
    others, whose p and q agree to that.  Equal tokens have equal exponentials in both rows, so what is left of each is
    off by its units of 2^-40 (up to 3 a token: its mass in p, its mass in q, its own rounding)."""
    rng = np.random.RandomState(vocab)
    B = 200 if vocab < 1000 else 40
    x = torch.from_numpy(rng.randn(2 * B, vocab) * 1.5).to(dtype)
    x[::2, 1], x[::2, 0] = 4.0, -30.0
    less = torch.softmax(x[::2].double(), -1)[:, 1]
    # p of token 0 from 2^-12 to 2^-32, less than half of what q gives it
    x[::2, 0] = (4.0 - np.log(2) * torch.linspace(12, 32, B) - less.log()).to(dtype)
    y = x[::2].clone()
    y[:, 0] = (y[:, 0].float() + 0.75).to(dtype)
    u = np.stack((0.99 + 0.009 * rng.rand(B), rng.rand(B)), -1).reshape(-1).astype(np.float32)
    tokens, logp, accepted, rejected = run(x.to(DEV), np.zeros(B, dtype=int), u, [2] * B, y.to(DEV))
    assert (accepted == 0).all() and (rejected == 1).all() and (tokens[1::2] == -1).all()
    tol, small = 2.0 ** -40 * (3 * vocab + 64), 0
    for b in range(B):
        _, _, acc, w, _ = ref.verify(x[2 * b:2 * b + 2].double().numpy(), y[b:b + 1].double().numpy(), [0],
                                     u[2 * b:2 * b + 2].astype(np.float64), 1.0)
        cum, t = np.cumsum(w), int(tokens[2 * b])
        place = float(u[2 * b + 1]) * cum[-1]
        small += cum[-1] < 2.0 ** -23
        assert acc == 0 and t > 0 and cum[t - 1] - tol <= place <= cum[t] + tol, (b, t, cum[-1], place - cum[t])
    assert small > B // 5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [0.05, 0.3, 1.0])
def test_rows_that_nearly_agree(T, dtype):
    """q beside p by 10^-9 to 10^-4 of itself or not at all, u next to 1, the draft that q likes best beyond p: where it
    falls, the token is drawn from the little that p leaves, or from p where that is nothing, to 2^-24 of the whole."""
    rng = np.random.RandomState(3)
    B, T, refusals = 600, float(np.float32(T)), 0
    at = torch.arange(B, device=DEV)
    for turn in range(80):
        V = int(2 ** rng.uniform(1, 11))
        x = (torch.from_numpy(rng.randn(2 * B, V)).to(DEV) * [0.3, 1, 3, 8][turn % 4]).to(dtype)
        y = (x[::2].float() + torch.from_numpy(rng.randn(B, V)).float().to(DEV) * 10 ** rng.uniform(-9, -4)).to(dtype)
        p, q = (torch.softmax(t.double() / T, -1) for t in (x[::2], y))
        drafts = (q - p).argmax(-1)
        u = np.stack((np.full(B, 1 - 2.0 ** -24), rng.rand(B)), -1).reshape(-1).astype(np.float32)
        tokens, _, accepted, _ = (torch.from_numpy(t).to(DEV) for t in run(x, drafts.tolist(), u, [2] * B, y, [T] * B))
        w, t = (p - q).clamp(min=0), tokens[::2].long()
        # Equal rows leave nothing.  Rows that differ leave something, be it less than 2^-24 of the whole, where every
        # border of w lies within that of every place and any token may be given.
        cum = torch.where((x[::2] == y).all(-1, keepdim=True), p, w).cumsum(-1)
        place = torch.from_numpy(u[1::2]).double().to(DEV) * cum[:, -1]
        before = torch.where(t > 0, cum[at, (t - 1).clamp(min=0)], torch.zeros_like(place))
        good = (t >= 0) & (before - 2.0 ** -24 <= place) & (place <= cum[at, t.clamp(min=0)] + 2.0 ** -24)
        assert good[accepted == 0].all(), (turn, V, int((~good & (accepted == 0)).sum()))
        refusals += int((accepted == 0).sum())
    assert refusals > 5000
