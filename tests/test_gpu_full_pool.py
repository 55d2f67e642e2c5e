"""Rollout with drafted tokens whose pool runs out: entries that were not served lose nothing (needs a GB300)."""
import numpy as np
import pytest
import torch

import oracle.pages_ref as ref
from tests.test_gpu_pages import DEV, bf16, check_decode, dev, handle, i32, same_tables
from tests.test_gpu_verify import built, case  # noqa: F401

pytestmark = pytest.mark.gpu
ALL = 2 ** 31 - 1


def test_a_captured_rollout_whose_pool_runs_out_and_recovers():
    """Captured once and replayed: slots grow until some find no page, then one is freed and they go on."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(1)
    B, most, Hkv, hq, V = 5, 4, 1, 4, 60
    c = ref.Pages(9, B, 6, Hkv, 16)
    h = handle(c)
    order, T = [2, 0, 4, 3, 1], B * most
    slots, new, drop = i32(order), i32([0] * B), i32([0] * B)
    k, v = (torch.empty((T, Hkv, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, sink = torch.zeros((T, hq, 64), dtype=torch.bfloat16, device=DEV), dev(rng.randn(hq), torch.float32)
    x, y = torch.zeros((T, V), device=DEV), torch.zeros((T - B, V), device=DEV)
    drafts, u = i32([0] * (T - B)), torch.zeros(T, device=DEV)
    ws, vs = sa.kv_decode_workspace(h), sa.verify_workspace(x)

    def step():
        live, cu, places, pos = sa.kv_plan(h, slots, new, T, drop=drop)
        sa.kv_write(h, places, k, v)
        o, lse = sa.kv_decode_fwd(h, live, q, sink, q_per_seq=most, cu_rows=cu, workspace=ws)
        out = sa.verify_tokens(x, drafts, u, cu, draft_logits=y, live=live, workspace=vs)
        drop.copy_(out[3])
        return (live, cu, places, pos), (o, lse), out

    step()  # first calls outside the capture: no new tokens
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        planned, attended, verified = step()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    rejected, unserved, recovered, waited = [0] * B, 0, 0, set()
    for turn in range(60):
        if len(waited) >= 2 and turn % 4 == 0:  # the longest sequence has ended: its slot begins anew
            b = int(np.argmax(c.lens[order]))
            rejected[b] = ALL
            drop[b] = ALL
        assert drop.tolist() == rejected
        counts = [int(z) for z in rng.randint(1, most + 1, B)]
        R, D = sum(counts), sum(counts) - B
        new.copy_(i32(counts))
        for t in (k, v, q):
            t.copy_(bf16(rng, *t.shape))
        x.copy_(torch.from_numpy(rng.randn(T, V) * 2))
        rows = [r for b in range(B) for r in range(sum(counts[:b]), sum(counts[:b + 1]) - 1)]
        y[:D] = x[rows] + torch.from_numpy(rng.randn(D, V)).float().to(DEV)
        pick = [int(rng.choice(V, p=torch.softmax(z.double(), -1).numpy())) for z in y[:D].cpu()]
        drafts.copy_(i32(pick + [0] * (T - B - D)))
        u.copy_(torch.from_numpy(rng.rand(T)))
        want = c.plan(order, rejected, counts, T)
        for b in range(B):
            if want[0][b] < 0:  # logits of nothing
                x[sum(counts[:b]):sum(counts[:b + 1])] = float("nan")
        graph.replay()
        for a, b in zip(planned, want):
            assert np.array_equal(a.cpu().numpy(), b), turn
        same_tables(c, h)
        c.write(want[2], f64(k), f64(v))
        check_decode(c, [int(s) for s in want[0]], counts, hq, -1, 0, q[:R], sink, attended[0][:R], attended[1][:, :R])
        at, rejected = 0, []
        for b, n in enumerate(counts):
            mine, d = slice(at, at + n), slice(at - b, at - b + n - 1)
            at += n
            if want[0][b] < 0:
                unserved += 1
                waited.add(b)
                assert verified[0][mine].tolist() == [-1] * n and (verified[1][mine] == 0).all()
                assert int(verified[2][b]) == 0
                rejected.append(0)
                continue
            recovered += b in waited
            waited.discard(b)
            tokens, logp, acc, _, _ = ref.verify(f64(x[mine]), f64(y[d]), pick[d], f64(u[mine]), 1.0)
            assert verified[0][mine].tolist() == list(tokens) and int(verified[2][b]) == acc, (turn, b)
            assert np.abs(f64(verified[1][mine]) - logp).max() <= 2.0 ** -18
            rejected.append(n - 1 - acc)
        assert verified[3].tolist() == rejected
    assert unserved > 20 and recovered > 5


@pytest.mark.parametrize("proposal", [True, False])
@pytest.mark.parametrize("B,rows_to", [(3, 5), (70, 5), (700, 5), (900, 1)])
def test_entries_that_were_not_served(B, rows_to, proposal):
    """Calls of every make-up (drafts tested apart or not, more entries than rows): the others as if alone, -1 and 0 there."""
    import sink_aware_masked_gb300 as sa

    rng = np.random.RandomState(B)
    counts = [int(n) for n in rng.randint(0, rows_to + 1, B)]
    counts[0] = rows_to
    x, drafts, y, u = case(rng, counts, 501, torch.float32, proposal)
    live = rng.randint(-3, 4, B)
    live[0], live[1] = -1, 7
    temp = torch.from_numpy(rng.choice([0.0, 0.7, 1.0], B)).float().to(DEV)
    cu = np.concatenate(([0], np.cumsum(counts)))
    u = torch.from_numpy(u).float().to(DEV)
    want = [t.clone() for t in sa.verify_tokens(x, i32(drafts), u, i32(cu), draft_logits=y, temperature=temp)]
    for b in range(B):
        if live[b] < 0:
            rows = slice(int(cu[b]), int(cu[b + 1]))
            want[0][rows], want[1][rows], want[2][b], want[3][b] = -1, 0.0, 0, 0
            x[rows] = float("nan")
    got = sa.verify_tokens(x, i32(drafts), u, i32(cu), draft_logits=y, temperature=temp, live=i32(live))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = sa.verify_tokens(x, i32(drafts), u, i32(cu), draft_logits=y, temperature=temp, live=i32([-1] * B))
    assert (got[0] == -1).all() and all((t == 0).all() for t in got[1:])
