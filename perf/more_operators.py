"""Rollout operators over bf16 pages and drafted tokens, as they are measured: cases, inputs, plain forms, 64-bit values.

A rollout that drafts several tokens a step keeps its keys and values in pages
of bf16, the type the trainer's attention works in.  One step plans where the
new tokens of every sequence go, writes their keys and values there, attends
to the pages for all of them at once and verifies the drafts against the
target's logits; the rejected ones are dropped by the next step's plan.  Four
kinds of case:

  plan     block tables and slot maps from the requests' lengths: what a slot drops, what it gets, where each row goes
  write    new keys and values into the pages, by the slot map
  decode   the new rows of each sequence against its pages (sink, window, prefix), one or several rows each
  verify   drafted tokens against the target's probabilities, from given random numbers

The pages.  ``k_pages`` and ``v_pages`` are bf16 [num_pages, page_size,
kv_heads, 64]; place p of the pool is row p % page_size of page p //
page_size.  Slot s holds ``seqlens[s]`` tokens in the pages
``block_table[s][0 .. ceil(seqlens[s] / page_size) - 1]`` (the other entries
are -1 here); ``owner[p]`` is the slot that holds page p, -1 where it is free.

Rows of several sequences stand one after another: those of sequence b are
cu[b] .. cu[b + 1] - 1.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 64
DEV = "cuda"
ALL = (1 << 31) - 1  # dropped from a slot: everything


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence grows by a token (latency counts)
        {"name": "plan_1_step", "op": "plan", "slots": 1, "len_lo": 37, "len_hi": 37, "new": 1, "renew": 0, "page": 64},
        # a step of 256 sequences with up to 4 drafts each, after the last step's rejections
        {"name": "plan_256_drafted", "op": "plan", "slots": 256, "len_lo": 60, "len_hi": 8192, "new": 5, "renew": 0,
         "page": 16},
        # 512 sequences of which every eighth has ended and makes room for a new prompt
        {"name": "plan_512_refilled", "op": "plan", "slots": 512, "len_lo": 101, "len_hi": 16001, "new": 1, "renew": 8,
         "page": 64},
        # one new token of 64 sequences
        {"name": "write_64_tokens", "op": "write", "tokens": 64, "kv_heads": 8, "q_heads": 64, "fused": True, "page": 16},
        # prompts and tool answers being filled in, out of the fused projection's rows
        {"name": "write_70001_tokens", "op": "write", "tokens": 70001, "kv_heads": 8, "q_heads": 16, "fused": True,
         "page": 64},
        # the smallest step: one sequence that has just begun (latency counts)
        {"name": "decode_1x37", "op": "decode", "batch": 1, "len_lo": 37, "len_hi": 37, "heads": 64, "kv_heads": 8,
         "rows_lo": 1, "rows_hi": 1, "window": -1, "prefix": 0, "page": 16},
        # an ordinary step of 32 sequences without drafts
        {"name": "decode_32x8192", "op": "decode", "batch": 32, "len_lo": 8192, "len_hi": 8192, "heads": 64,
         "kv_heads": 8, "rows_lo": 1, "rows_hi": 1, "window": -1, "prefix": 0, "page": 64},
        # long sequences with 1 to 5 rows each, drafted tokens among them
        {"name": "decode_8x32768_drafted", "op": "decode", "batch": 8, "len_lo": 30011, "len_hi": 32768, "heads": 64,
         "kv_heads": 8, "rows_lo": 1, "rows_hi": 5, "window": -1, "prefix": 0, "page": 64},
        # trajectories of very different lengths under window and prefix, odd head counts, small pages
        {"name": "decode_200_ragged_w128", "op": "decode", "batch": 200, "len_lo": 3, "len_hi": 20001, "heads": 40,
         "kv_heads": 8, "rows_lo": 1, "rows_hi": 2, "window": 128, "prefix": 4, "page": 16},
        # one sequence's three drafts, float32 logits over an odd vocabulary (latency counts)
        {"name": "verify_1x3_50257", "op": "verify", "batch": 1, "drafts_lo": 3, "drafts_hi": 3, "vocab": 50257,
         "dtype": "float32", "temperature": 0.8, "proposal": True, "mixed": False},
        # a large batch with up to 4 drafts of a smaller model each, some rows greedy, some under a grammar
        {"name": "verify_128x4_201088", "op": "verify", "batch": 128, "drafts_lo": 0, "drafts_hi": 4, "vocab": 201088,
         "dtype": "bfloat16", "temperature": 1.0, "proposal": True, "mixed": True},
        # drafts looked up in the text so far: no probabilities come with them
        {"name": "verify_48x7_lookup", "op": "verify", "batch": 48, "drafts_lo": 1, "drafts_hi": 7, "vocab": 100003,
         "dtype": "float16", "temperature": 0.9, "proposal": False, "mixed": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "plan", "write", "decode", "decode", "decode", "verify", "verify"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        hi = _log_int(rng, 1, 16000)
        slots = max(1, min(_log_int(rng, 1, 1024), (1 << 22) // hi))
        return {"op": op, "slots": slots, "len_lo": _log_int(rng, 1, hi), "len_hi": hi,
                "new": rng.choice([1, 1, 2, 5, 9]), "renew": rng.choice([0, 0, 1, 3, 8]), "page": page}
    if op == "write":
        kv = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "tokens": _log_int(rng, 1, 70001), "kv_heads": kv, "q_heads": kv * rng.choice([1, 2, 5, 8]),
                "fused": rng.choice([True, False]), "page": page}
    if op == "decode":
        kv, group = rng.choice([(1, 8), (2, 8), (4, 4), (8, 8), (8, 1), (8, 5), (3, 7), (1, 16)])
        hi = _log_int(rng, 2, 100000)
        batch = max(1, min(_log_int(rng, 1, 256), (1 << 18) // hi))
        rows = rng.choice([1, 1, 1, 2, 4, 6, 8])
        return {"op": op, "batch": batch, "len_lo": _log_int(rng, 1, hi), "len_hi": hi, "heads": kv * group,
                "kv_heads": kv, "rows_lo": rng.choice([1, rows]), "rows_hi": rows,
                "window": rng.choice([-1, -1, 0, 128, 1000]), "prefix": rng.choice([0, 4, 100]), "page": page}
    vocab, drafts = _log_int(rng, 100, 201088), rng.choice([0, 1, 2, 4, 7])
    proposal = rng.choice([True, True, False])
    return {"op": op, "batch": max(1, min(_log_int(rng, 1, 256), 384 * 201088 // (vocab * (2 * drafts + 1)))),
            "drafts_lo": rng.choice([0, drafts]), "drafts_hi": drafts, "vocab": vocab,
            "dtype": rng.choice(["float32", "bfloat16", "float16"]), "temperature": round(rng.uniform(0.3, 1.5), 3),
            "proposal": proposal, "mixed": rng.choice([True, False])}


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread over their logarithm, in a fixed mixed order."""
    x = np.exp(np.linspace(math.log(lo), math.log(hi), n)).round().astype(np.int64)
    x[-1] = hi
    return np.random.RandomState(1).permutation(x)


def _counts(n, lo, hi):
    """n counts from lo to hi in turn, in a fixed mixed order."""
    return np.random.RandomState(2).permutation(lo + np.arange(n)[::-1] % (hi - lo + 1))


def _plan_numbers(case):
    """Per slot: tokens held, dropped and new.  A slot ends as long as it was, so that a pass can follow a pass."""
    n = case["slots"]
    lens = _spread(n, case["len_lo"], case["len_hi"])
    new = np.minimum(_counts(n, 1, case["new"]), lens)
    drop = new.copy()
    if case["renew"]:
        ended = np.arange(n) % case["renew"] == case["renew"] - 1
        new, drop = np.where(ended, lens, new), np.where(ended, ALL, drop)
    return lens, drop, new


def _visible_keys(length, rows, window, prefix):
    """Keys that at least one of the last `rows` positions sees."""
    first = max(0, length - rows)
    lo = 0 if window < 0 else max(0, first - window)
    return length - lo + min(prefix, lo)


def work(case):
    op = case["op"]
    if op == "plan":
        lens, drop, new = _plan_numbers(case)
        left = np.maximum(lens - drop, 0)
        moved = int((-(-lens // case["page"]) - -(-left // case["page"])).sum())  # pages that go, and as many that come
        # lists in and out, lengths; an entry and an owner of each page that goes or comes; the rows' places and positions
        return {"bytes": 4 * (7 * len(lens) + 5 * moved + 2 * int(new.sum())), "flops": 0}
    if op == "write":
        return {"bytes": case["tokens"] * (case["kv_heads"] * 4 * 128 + 4), "flops": 0}
    if op == "decode":
        lens, rows = _decode_numbers(case)
        keys = [_visible_keys(int(x), int(n), case["window"], case["prefix"]) for x, n in zip(lens, rows)]
        return {"bytes": sum(keys) * case["kv_heads"] * 256 + int(rows.sum()) * case["heads"] * (2 * 128 + 4)
                + case["heads"] * 4,
                "flops": 4 * 64 * case["heads"] * sum(k * int(n) for k, n in zip(keys, rows))}
    drafts = _counts(case["batch"], case["drafts_lo"], case["drafts_hi"])
    rows = int(drafts.sum()) * (2 if case["proposal"] else 1) + case["batch"]
    size = 4 if case["dtype"] == "float32" else 2
    return {"bytes": rows * case["vocab"] * size + int(drafts.sum() + case["batch"]) * 20, "flops": rows * case["vocab"] * 5}


def _decode_numbers(case):
    lens = _spread(case["batch"], case["len_lo"], case["len_hi"])
    return lens, _counts(case["batch"], case["rows_lo"], case["rows_hi"])


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 31))


def _i32(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).to(DEV)


def _offsets(counts):
    return _i32(np.concatenate(([0], np.cumsum(counts))))


def _kv(shape, g):
    """Keys with a few strong channels, values without, as trained models have them."""
    H = shape[-2]
    gain = 0.5 + 2.5 * torch.rand((H, HEAD_DIM), generator=g, device=DEV) ** 6
    shift = torch.randn((H, HEAD_DIM), generator=g, device=DEV) * 0.5
    k = torch.randn(shape, generator=g, device=DEV).mul_(gain).add_(shift).to(torch.bfloat16)
    return k, torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _tables(lens, page, g, pool):
    """Block table, lengths and owners of slots that hold `lens` tokens in pages that lie in mixed order."""
    held = [-(-int(x) // page) for x in lens]
    order = torch.randperm(pool, generator=g, device=DEV)[:sum(held)].to(torch.int32).cpu().numpy()
    table = np.full((len(lens), max(max(held), 1)), -1, dtype=np.int32)
    owner = np.full(pool, -1, dtype=np.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        owner[order[at:at + h]] = i
        at += h
    return {"block_table": _i32(table), "seqlens": _i32(lens), "owner": _i32(owner), "page": page}


def prepare(case, seed):
    return {"plan": _prepare_plan, "write": _prepare_write, "decode": _prepare_decode,
            "verify": _prepare_verify}[case["op"]](case, _gen(seed))


def _pools(num_pages, page, kv_heads, g=None):
    shape = (num_pages, page, kv_heads, HEAD_DIM)
    if g is not None:
        return _kv(shape, g)
    return torch.zeros(shape, dtype=torch.bfloat16, device=DEV), torch.zeros(shape, dtype=torch.bfloat16, device=DEV)


def _prepare_plan(case, g):
    lens, drop, new = _plan_numbers(case)
    held = -(-lens // case["page"])
    # behind the slots of the call one that waits, with pages of its own; some more pages are free
    waits = max(40, int(held.max()))
    state = _tables(np.append(lens, waits * case["page"]), case["page"], g, int(held.sum()) * 5 // 4 + waits + 24)
    # a plan does not touch keys or values: one head stands for all
    state["k_pages"], state["v_pages"] = _pools(state["owner"].numel(), case["page"], 1)
    order = np.random.RandomState(3).permutation(len(lens))
    state.update(case, slots=_i32(order), drop=_i32(drop[order]), new=_i32(new[order]), total=int(new.sum()))
    _plain_plan(state)  # the loop has run before: pages taken from here on are the lowest free ones
    return state


def _prepare_write(case, g):
    T, H, page = case["tokens"], case["kv_heads"], case["page"]
    num_pages = -(-T // page) + 3
    state = {"block_table": torch.full((1, num_pages), -1, dtype=torch.int32, device=DEV), "page": page,
             "seqlens": torch.zeros(1, dtype=torch.int32, device=DEV),
             "owner": torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)}
    state["k_pages"], state["v_pages"] = _pools(num_pages, page, H)
    # runs of tokens in pages of mixed order; one row in 50 has no place (its request found no room)
    place = torch.randperm(num_pages, generator=g, device=DEV)[:, None] * page + torch.arange(page, device=DEV)
    place = place.reshape(-1)[:T].to(torch.int32)
    place[torch.rand(T, generator=g, device=DEV) < 0.02] = -1
    k, v = _kv((T, H, HEAD_DIM), g)
    if case["fused"]:
        rows = torch.empty((T, case["q_heads"] + 2 * H, HEAD_DIM), dtype=torch.bfloat16, device=DEV)
        rows[:, :case["q_heads"]] = 1.0
        rows[:, case["q_heads"]:-H], rows[:, -H:] = k, v
        k, v = rows[:, case["q_heads"]:-H], rows[:, -H:]
    state.update(case, slot_map=place, k=k, v=v)
    return state


def _prepare_decode(case, g):
    lens, rows = _decode_numbers(case)
    held = int((-(-lens // case["page"])).sum())
    state = _tables(lens, case["page"], g, held + 5)
    state["k_pages"], state["v_pages"] = _pools(held + 5, case["page"], case["kv_heads"], g)
    R = int(rows.sum())
    state.update(case, slots=torch.arange(case["batch"], device=DEV, dtype=torch.int32), cu=_offsets(rows),
                 ragged=case["rows_lo"] != case["rows_hi"],
                 q=(1.5 * torch.randn((R, case["heads"], HEAD_DIM), generator=g, device=DEV)).to(torch.bfloat16),
                 sink=torch.randn(case["heads"], generator=g, device=DEV))
    return state


def _prepare_verify(case, g):
    B, V = case["batch"], case["vocab"]
    drafts = _counts(B, case["drafts_lo"], case["drafts_hi"])
    R, D = int(drafts.sum()) + B, int(drafts.sum())
    # a few likely tokens and a long tail, as language models give them
    rank = torch.rand((R, V), generator=g, device=DEV).clamp_(min=1e-7).mul_(V).add_(1.0)
    x = rank.log_().mul_(-1.2).add_(12.0).add_(torch.randn((R, V), generator=g, device=DEV), alpha=0.8)
    T = torch.full((B,), case["temperature"], device=DEV)
    seq = torch.from_numpy(np.repeat(np.arange(B), drafts + 1)).to(DEV)
    last = torch.from_numpy(np.cumsum(drafts + 1) - 1).to(DEV)
    tested = torch.ones(R, dtype=torch.bool, device=DEV)
    tested[last] = False  # the rows that a draft follows
    if case["mixed"]:
        i = torch.arange(B, device=DEV)
        T[i % 7 == 1] = 0.0
        T[i % 7 == 2] = 0.6
        x[(seq % 6 == 5).nonzero().reshape(-1), V // 50 + 1:] = -math.inf  # a grammar that allows the first tokens alone
    dtype = getattr(torch, case["dtype"])
    y = None
    if case["proposal"]:
        y = x[tested]
        y = y.add_(torch.randn((D, V), generator=g, device=DEV), alpha=0.5).to(dtype)
    x = x.to(dtype)
    # drafts: drawn from the smaller model's probabilities, or, looked up, mostly what the target finds likely too
    z = (y if case["proposal"] else x[tested]).float()
    t = T[seq[tested]][:, None]
    noise = torch.rand((D, V), generator=g, device=DEV).clamp_(min=1e-12).log_().neg_().log_().neg_()
    z = torch.where(t > 0, z / torch.where(t > 0, t, torch.ones_like(t)) + noise, z)
    draft = z.argmax(-1) if D else torch.zeros(0, dtype=torch.int64, device=DEV)
    if not case["proposal"]:
        stray = torch.rand(D, generator=g, device=DEV) < 0.3
        draft = torch.where(stray, torch.randint(0, V, (D,), generator=g, device=DEV), draft)
    return dict(case, logits=x, draft_logits=y, drafts=draft.to(torch.int32), cu=_offsets(drafts + 1), temp=T,
                u=torch.rand(R, generator=g, device=DEV))


# ---------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _own_pages(sa, state):
    """The framework's handle of the pages, kept as a user's program keeps it."""
    if "handle" not in state:
        state["handle"] = sa.KVPages(*(state[x] for x in ("k_pages", "v_pages", "block_table", "seqlens", "owner")))
    return state["handle"]


def _run_own(state):
    import sink_aware_masked_gb300 as sa

    op = state["op"]
    if op == "verify":
        if "workspace" not in state:
            state["workspace"] = sa.verify_workspace(state["logits"])
        return sa.verify_tokens(state["logits"], state["drafts"], state["u"], state["cu"],
                                draft_logits=state["draft_logits"], temperature=state["temp"],
                                workspace=state["workspace"])
    pages = _own_pages(sa, state)
    if op == "plan":
        live, cu, slot_map, positions = sa.kv_plan(pages, state["slots"], state["new"], state["total"],
                                                   drop=state["drop"])
        return live, cu, slot_map, positions, state["block_table"], state["seqlens"], state["owner"]
    if op == "write":
        sa.kv_write(pages, state["slot_map"], state["k"], state["v"])
        return state["k_pages"], state["v_pages"]
    if "workspace" not in state:
        state["workspace"] = sa.kv_decode_workspace(pages)
    return sa.kv_decode_fwd(pages, state["slots"], state["q"], state["sink"], q_per_seq=state["rows_hi"],
                            cu_rows=state["cu"] if state["ragged"] else None, window=state["window"],
                            prefix=state["prefix"], workspace=state["workspace"])


def _run_plain(state):
    return {"plan": _plain_plan, "write": _plain_write, "decode": _plain_decode, "verify": _plain_verify}[state["op"]](
        state)


def _plain_plan(state):
    table, lens, owner, page = state["block_table"], state["seqlens"], state["owner"], state["page"]
    s, new = state["slots"].long(), state["new"].long()
    size = lens[s].long()
    left = (size - state["drop"].long()).clamp(min=0)
    held, kept, want = -(-size // page), -(-left // page), -(-(left + new) // page)
    column = torch.arange(table.shape[1], device=DEV)[None, :]
    # what is dropped gives its pages back, before anything is handed out
    row = table[s].long()
    gone = (column >= kept[:, None]) & (column < held[:, None])
    owner[row[gone]] = -1
    row = torch.where(gone, torch.full_like(row, -1), row)
    # the lowest free pages to the requests in order, until one does not fit
    free = (owner < 0).nonzero().reshape(-1)
    need = want - kept
    upto = torch.cumsum(need, 0)
    ok = (upto <= free.numel()) | (need == 0)
    take = (column >= kept[:, None]) & (column < want[:, None]) & ok[:, None]
    got = free[((upto - need)[:, None] + column - kept[:, None])[take]]
    row[take] = got
    owner[got] = s[:, None].expand_as(take)[take].to(torch.int32)
    table[s] = row.to(torch.int32)
    lens[s] = torch.where(ok, left + new, left).to(torch.int32)
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)))
    at = torch.arange(state["total"], device=DEV)
    b = torch.searchsorted(cu[1:], at, right=True)
    pos = left[b] + at - cu[b]
    place = row[b, pos // page] * page + pos % page
    place, pos = (torch.where(ok[b], x, torch.full_like(x, -1)) for x in (place, pos))
    return (torch.where(ok, s, torch.full_like(s, -1)).to(torch.int32), cu.to(torch.int32), place.to(torch.int32),
            pos.to(torch.int32), table, lens, owner)


def _plain_write(state):
    at = state["slot_map"].long()
    there = at >= 0
    for pages, x in ((state["k_pages"], state["k"]), (state["v_pages"], state["v"])):
        pages.view(-1, *pages.shape[2:])[at[there]] = x[there]
    return state["k_pages"], state["v_pages"]


def _plain_decode(state):
    page, Hq, H, n = state["page"], state["heads"], state["kv_heads"], state["rows_hi"]
    slots, cu = state["slots"].long(), state["cu"].long()
    B = slots.numel()
    table, lens, count = state["block_table"].long()[slots], state["seqlens"].long()[slots], cu[1:] - cu[:-1]
    k, v = (state[x][table.clamp(min=0)].reshape(B, -1, H, 64).permute(0, 2, 1, 3).float()
            for x in ("k_pages", "v_pages"))  # [B, H, L, 64]
    # every sequence's rows side by side, the missing ones anything
    i = torch.arange(n, device=DEV)
    there = i < count[:, None]
    row = torch.where(there, cu[:-1, None] + i, torch.zeros_like(i))
    q = state["q"].float()[row].view(B, n, H, Hq // H, 64).permute(0, 2, 3, 1, 4).reshape(B, H, -1, 64)
    pos_k, pos_q = torch.arange(k.shape[2], device=DEV), lens[:, None] - count[:, None] + i
    seen = pos_k <= pos_q[..., None]
    if state["window"] >= 0:
        seen = seen & ((pos_q[..., None] - pos_k <= state["window"]) | (pos_k < state["prefix"]))
    s = torch.matmul(q, k.transpose(2, 3)).view(B, H, Hq // H, n, -1) * 0.125
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    alpha = torch.sigmoid(lse - state["sink"].view(1, H, Hq // H, 1, 1))
    o = torch.matmul((e / total.clamp(min=1e-30)).view(B, H, -1, e.shape[-1]), v).view(B, H, Hq // H, n, 64) * alpha
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, 64)[there].to(torch.bfloat16)
    return o, lse.permute(0, 3, 1, 2, 4).reshape(B, n, Hq)[there].t().contiguous()


def _softmax64(x, T):
    """Probabilities of rows x at temperatures T [rows, 1] in 64 bits, what belongs to them, and log-sums."""
    x = x.double()
    top = x.amax(-1, keepdim=True)
    z = (x - top) / T
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    return e / total, z - torch.log(total)


def _plain_verify(state):
    cu, draft, u = state["cu"].long(), state["drafts"].long(), state["u"].double()
    B, R, V = cu.numel() - 1, state["logits"].shape[0], state["logits"].shape[1]
    seq = torch.searchsorted(cu[1:], torch.arange(R, device=DEV), right=True)
    tested = torch.ones(R, dtype=torch.bool, device=DEV)
    tested[cu[1:] - 1] = False
    at = tested.nonzero().reshape(-1)  # the row that draft d is tested against
    greedy = state["temp"] == 0
    T = torch.where(greedy, torch.ones_like(state["temp"]), state["temp"]).double()
    p, logp = _softmax64(state["logits"], T[seq][:, None])
    best = (state["logits"] == state["logits"].amax(-1, keepdim=True)).to(torch.int8).argmax(-1)  # the first of equals
    px = p[at, draft]
    qx = torch.ones_like(px)
    if state["draft_logits"] is not None:
        q = _softmax64(state["draft_logits"], T[seq[at]][:, None])[0]
        qx = q.gather(1, draft[:, None])[:, 0]
    fine = torch.where(greedy[seq[at]], draft == best[at], u[at] * qx < px)
    # the first row whose draft is refused, or the sequence's last row
    stop = torch.arange(R, device=DEV)
    stop[at[fine]] = R
    first = torch.full((B,), R, device=DEV).scatter_reduce(0, seq, stop, "amin")
    accepted = first - cu[:-1]
    refused = first < cu[1:] - 1
    # what is left of the target's probabilities where a draft was refused; the target's own after the last draft
    w = p[first]
    d = (first - torch.arange(B, device=DEV))[refused]  # the refused drafts
    if state["draft_logits"] is not None:
        rest = (w[refused] - q[d]).clamp(min=0.0)
    else:
        rest = w[refused].scatter(1, draft[d][:, None], 0.0)
    w[refused] = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w[refused])
    run = torch.cumsum(w, -1)
    token = (run <= u[cu[1:] - 1][:, None] * run[:, -1:]).sum(-1)
    token = torch.minimum(token, V - 1 - (w > 0).to(torch.int8).flip(-1).argmax(-1))
    token = torch.where(greedy, best[first], token)
    tokens = torch.full((R,), -1, dtype=torch.int64, device=DEV)
    tokens[at] = torch.where(at < first[seq[at]], draft, tokens[at])
    tokens[first] = token
    out = torch.where(tokens >= 0, logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0], torch.zeros((), device=DEV).double())
    rejected = cu[1:] - 1 - first
    return tokens.to(torch.int32), out.float(), accepted.to(torch.int32), rejected.to(torch.int32)


# ---------------------------------------------------------------- 64 bits, apart from the above
def _exact_decode(case, state):
    H, Hq = case["kv_heads"], case["heads"]
    group, page = Hq // H, case["page"]
    cu, lens = state["cu"].cpu().tolist(), state["seqlens"].cpu().tolist()
    table, sink = state["block_table"].cpu().tolist(), state["sink"].double().view(H, group)
    o, lse = [], []
    for b in range(case["batch"]):
        L = lens[b]
        ids = torch.tensor(table[b][:-(-L // page)], device=DEV)
        k, v = (state[x][ids].double().reshape(-1, H, 64)[:L] for x in ("k_pages", "v_pages"))
        for r in range(cu[b], cu[b + 1]):
            at = L - (cu[b + 1] - r)
            j = torch.arange(max(at, -1) + 1, device=DEV)
            if case["window"] >= 0:
                j = j[(at - j <= case["window"]) | (j < case["prefix"])]
            s = torch.einsum("hgd,khd->hgk", state["q"][r].double().view(H, group, 64), k[j]) / 8.0
            l = torch.logsumexp(s, -1)
            o.append(torch.einsum("hgk,khd->hgd", torch.exp(s - torch.logaddexp(l, sink)[..., None]), v[j]).reshape(Hq, 64))
            lse.append(l.reshape(Hq))
    return torch.stack(o), torch.stack(lse, 1)


def _exact_verify(case, state):
    """The log-probabilities of the tokens given, sequence by sequence."""
    cu, u, temp = state["cu"].cpu().tolist(), state["u"].double().cpu().numpy(), state["temp"].double().cpu().tolist()
    draft = state["drafts"].cpu().tolist()
    out = np.zeros(cu[-1])
    for b in range(case["batch"]):
        T = temp[b] if temp[b] > 0 else 1.0
        for r in range(cu[b], cu[b + 1]):
            x = state["logits"][r].double() / T
            lp = x - torch.logsumexp(x, 0)
            w = torch.exp(lp)
            if r + 1 < cu[b + 1]:
                d = r - b
                if state["draft_logits"] is not None:
                    y = state["draft_logits"][d].double() / T
                    q = torch.exp(y - torch.logsumexp(y, 0))
                else:
                    q = torch.zeros_like(w)
                    q[draft[d]] = 1.0
                if temp[b] == 0:
                    fine = bool((x[:draft[d]] < x[draft[d]]).all() and (x[draft[d]:] <= x[draft[d]]).all())
                else:
                    fine = u[r] * float(q[draft[d]]) < float(w[draft[d]])
                if fine:
                    out[r] = float(lp[draft[d]])
                    continue
                rest = torch.clamp(w - q, min=0.0)
                w = rest if float(rest.sum()) > 0 else w
            if temp[b] == 0:
                out[r] = float(lp.max())
            else:
                run = torch.cumsum(w, 0).cpu().numpy()
                i = int(np.searchsorted(run, u[cu[b + 1] - 1] * run[-1], side="right"))
                out[r] = float(lp[min(i, int(w.nonzero()[-1]))])
            break
    return None, torch.from_numpy(out), None, None


def exact(case, seed):
    if case["op"] in ("plan", "write"):
        return None  # whole numbers, and copies
    state = prepare(case, seed)
    return _exact_decode(case, state) if case["op"] == "decode" else _exact_verify(case, state)
