"""The rollout-side operators as they are measured: cases, inputs, plain forms and 64-bit values.

A rollout of the training loop keeps its keys and values in a paged cache of
4-bit values, forks one prompt's pages into the rollouts of a group, attends
to the cache for each new token and samples the token together with the
log-probability that the GRPO loss takes as ``logp_old``.  Four kinds of case:

  append   writes new keys and values into the pages (4-bit quantisation) and reads them back
  decode   the last rows of each sequence against its 4-bit pages (sink, window, prefix)
  fork     frees a group's old rollouts, forks its prompts into new ones, reserves a token each
  compact  moves the live pages of a pool into another pool, tables and counts with them
  sample   temperature, top-k, top-p and min-p from given random numbers

The cache.  ``pages`` is uint8 [num_pages, kv_heads, page_size * 72]: blocks of
16 tokens, 1152 bytes each, one after the other.  In a block, with g = 0..7
and t = 0..3, lane = 4 g + t:
  bytes [0, 512)      keys' codes: per lane 8 bytes of token g, then 8 of token g + 8: dims 16 t .. 16 t + 15
  bytes [512, 1024)   values' codes: per lane 4 bytes each of tokens 2t, 2t+1, 2t+8, 2t+9: dims 8 g .. 8 g + 7
  bytes [1024, 1088)  keys' scales: per lane those of tokens g and g + 8, dims 16 t .. 16 t + 15
  bytes [1088, 1152)  values' scales: per (group of 16 dims, t) those of tokens 2t, 2t+1, 2t+8, 2t+9
A byte holds two codes, the lower dim in the low nibble.  A code is sign (8)
and magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale is e4m3 and serves 16 dims
of a token; a value is code * scale * (its head's float32 factor).
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 64
BLOCK = 16
BLOCK_BYTES = 1152
DEV = "cuda"
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the smallest step: one sequence that has just begun (latency counts)
        {"name": "decode_1x37", "op": "decode", "batch": 1, "len_lo": 37, "len_hi": 37, "heads": 64, "kv_heads": 8,
         "rows": 1, "window": -1, "prefix": 0, "page": 64},
        # an ordinary rollout step of 32 sequences
        {"name": "decode_32x8192", "op": "decode", "batch": 32, "len_lo": 8192, "len_hi": 8192, "heads": 64,
         "kv_heads": 8, "rows": 1, "window": -1, "prefix": 0, "page": 64},
        # several new rows per sequence (drafted tokens being checked)
        {"name": "decode_8x32768_n4", "op": "decode", "batch": 8, "len_lo": 32768, "len_hi": 32768, "heads": 64,
         "kv_heads": 8, "rows": 4, "window": -1, "prefix": 0, "page": 64},
        # trajectories of very different lengths under window and prefix, odd head counts, small pages
        {"name": "decode_200_ragged_w128", "op": "decode", "batch": 200, "len_lo": 3, "len_hi": 20001, "heads": 40,
         "kv_heads": 8, "rows": 1, "window": 128, "prefix": 4, "page": 16},
        # one new token for each of 64 sequences
        {"name": "append_64x1", "op": "append", "batch": 64, "len_lo": 33, "len_hi": 8192, "new_lo": 1, "new_hi": 1,
         "kv_heads": 8, "page": 64},
        # prompts and tool answers of unequal lengths being filled in
        {"name": "append_12_ragged_long", "op": "append", "batch": 12, "len_lo": 1201, "len_hi": 16384,
         "new_lo": 1001, "new_hi": 16001, "kv_heads": 8, "page": 64},
        # a group of 4 rollouts of one short prompt begins (latency counts)
        {"name": "fork_1x4", "op": "fork", "prompts": 1, "group": 4, "len_lo": 77, "len_hi": 77, "kv_heads": 8,
         "page": 16},
        # a batch of 64 prompts with 8 rollouts each begins: the old rollouts' pages go, the prompts are forked
        {"name": "fork_64x8", "op": "fork", "prompts": 64, "group": 8, "len_lo": 131, "len_hi": 2050, "kv_heads": 8,
         "page": 64},
        # what a few short sequences hold is moved out of a pool that is mostly empty
        {"name": "compact_5_slots", "op": "compact", "slots": 5, "len_lo": 20, "len_hi": 300, "kv_heads": 2,
         "page": 32, "spare": 4.0},
        # the cache is packed into a smaller pool before the trainer takes the memory
        {"name": "compact_96_slots", "op": "compact", "slots": 96, "len_lo": 100, "len_hi": 8000, "kv_heads": 8,
         "page": 64, "spare": 3.0},
        # one row of float32 logits over an odd vocabulary
        {"name": "sample_1x50257", "op": "sample", "batch": 1, "vocab": 50257, "dtype": "float32", "temperature": 0.8,
         "top_k": 50, "top_p": 0.95, "min_p": 0.0, "mixed": False},
        # a large batch whose rows ask for different things, some of them greedy, some masked
        {"name": "sample_256x201088_mixed", "op": "sample", "batch": 256, "vocab": 201088, "dtype": "bfloat16",
         "temperature": 0.9, "top_k": 200, "top_p": 0.95, "min_p": 0.02, "mixed": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fork", "compact", "sample", "sample"])
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        kv, group = rng.choice([(1, 8), (2, 8), (4, 4), (8, 8), (8, 1), (8, 5), (3, 7), (1, 32)])
        hi = _log_int(rng, 2, 100000)
        batch = max(1, min(_log_int(rng, 1, 256), (1 << 18) // hi))
        return {"op": op, "batch": batch, "len_lo": _log_int(rng, 1, hi), "len_hi": hi, "heads": kv * group,
                "kv_heads": kv, "rows": rng.choice([1, 1, 1, 2, 3, 4]), "window": rng.choice([-1, -1, 0, 128, 1000]),
                "prefix": rng.choice([0, 4, 100]), "page": page}
    if op == "append":
        hi = _log_int(rng, 1, 16000)
        batch = max(1, min(_log_int(rng, 1, 256), (1 << 16) // hi))
        lo = _log_int(rng, 1, hi)
        return {"op": op, "batch": batch, "len_lo": hi, "len_hi": hi + _log_int(rng, 1, 4000), "new_lo": lo,
                "new_hi": hi, "kv_heads": rng.choice([1, 2, 3, 4, 8]), "page": page}
    if op == "fork":
        hi = _log_int(rng, 2, 4000)
        return {"op": op, "prompts": _log_int(rng, 1, 64), "group": _log_int(rng, 1, 16), "len_lo": _log_int(rng, 1, hi),
                "len_hi": hi, "kv_heads": rng.choice([1, 2, 3, 8]), "page": page}
    if op == "compact":
        hi = _log_int(rng, 2, 8000)
        return {"op": op, "slots": _log_int(rng, 1, 96), "len_lo": _log_int(rng, 1, hi), "len_hi": hi,
                "kv_heads": rng.choice([1, 2, 3, 8]), "page": page, "spare": round(rng.uniform(1.0, 4.0), 2)}
    vocab = _log_int(rng, 100, 201088)
    return {"op": op, "batch": max(1, min(_log_int(rng, 1, 512), (256 * 201088) // vocab)), "vocab": vocab,
            "dtype": rng.choice(["float32", "bfloat16", "float16"]), "temperature": round(rng.uniform(0.3, 1.5), 3),
            "top_k": rng.choice([0, 1, 20, 1000]), "top_p": rng.choice([1.0, 0.95, 0.8, 0.3]),
            "min_p": rng.choice([0.0, 0.0, 0.05]), "mixed": rng.choice([True, False])}


def _lengths(n, lo, hi):
    """n lengths from lo to hi, evenly spread over their logarithm, in a fixed mixed order."""
    x = np.exp(np.linspace(math.log(lo), math.log(hi), n)).round().astype(np.int64)
    x[-1] = hi
    return np.random.RandomState(1).permutation(x)


def _visible_keys(length, rows, window, prefix):
    """Keys that at least one of the last `rows` positions sees."""
    first = max(0, length - rows)
    lo = 0 if window < 0 else max(0, first - window)
    return length - lo + min(prefix, lo)


def work(case):
    op = case["op"]
    if op == "decode":
        lens = _lengths(case["batch"], case["len_lo"], case["len_hi"])
        n, heads, kv = case["rows"], case["heads"], case["kv_heads"]
        keys = sum(_visible_keys(int(x), n, case["window"], case["prefix"]) for x in lens)
        rows = case["batch"] * n
        return {"bytes": keys * kv * 72 + rows * heads * (2 * 128 + 4) + heads * 4, "flops": 4 * 64 * heads * n * keys}
    if op == "append":
        tokens = int(_lengths(case["batch"], case["new_lo"], case["new_hi"]).sum())
        # in bf16, out in 4 bits, read from there, out in bf16
        return {"bytes": tokens * case["kv_heads"] * 2 * (128 + 36 + 36 + 128), "flops": tokens * case["kv_heads"] * 128 * 6}
    if op == "fork":
        lens = _lengths(case["prompts"], case["len_lo"], case["len_hi"])
        # each prompt's open page is read once and written for every rollout; the rollouts' tables are cleared and
        # written, their pages' counts taken down and up again
        part = (-(-(lens % case["page"]) // BLOCK)).sum() * BLOCK_BYTES * case["kv_heads"]
        table = (lens // case["page"] + 1).sum() * case["group"]
        return {"bytes": float(part * (1 + case["group"]) + table * 4 * 6 + len(lens) * case["group"] * 40), "flops": 0}
    if op == "compact":
        held = int((-(-_lengths(case["slots"], case["len_lo"], case["len_hi"]) // case["page"])).sum())
        pool = int(held * case["spare"]) + 1
        return {"bytes": 2 * held * case["page"] * 72 * case["kv_heads"] + 8 * held + 4 * pool, "flops": 0}
    size = 4 if case["dtype"] == "float32" else 2
    return {"bytes": case["batch"] * (case["vocab"] * size + 40), "flops": case["batch"] * case["vocab"] * 6}


# ---------------------------------------------------------------- the format, plainly
def _offsets():
    """[16, 72]: the place in a block of a token's 32 key bytes, 32 value bytes, 4 key scales, 4 value scales."""
    r = np.arange(16)[:, None]
    b = np.arange(32)[None, :]
    k = 16 * (4 * (r % 8) + b // 8) + 8 * (r // 8) + b % 8
    t, i = (r % 8) // 2, r % 2 + 2 * (r // 8)
    v = 512 + 16 * (4 * (b // 4) + t) + 4 * i + b % 4
    s = np.arange(4)[None, :]
    ks = 1024 + 2 * (4 * (r % 8) + s) + r // 8
    vs = 1088 + 4 * (4 * s + t) + i
    return torch.from_numpy(np.concatenate([k, v, ks, vs], axis=1)).to(DEV)


def _quantise(x, factor):
    """x [T, H, 64], factor [H] -> bytes [T, H, 32] and e4m3 scale bytes [T, H, 4]."""
    y = (x.float() / factor[None, :, None]).reshape(x.shape[0], x.shape[1], 4, 16)
    top = y.abs().amax(-1, keepdim=True)
    scale = (top / torch.tensor(6.0, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    z = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    a = z.abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; half ways go to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code | ((z < 0) & (code > 0)).to(torch.uint8) * 8).to(torch.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8).squeeze(-1)


def _values(codes, scales, factor):
    """bytes [..., H, 32], scale bytes [..., H, 4], factor [H] -> float32 [..., H, 64]."""
    lut = torch.tensor(LUT, dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 4, 16)
    y = lut[c.int()] * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return y.reshape(*codes.shape[:-1], 64) * factor[:, None]


def _places(state, cu, total):
    """For each of `total` rows: page, block in the page, row in the block."""
    table, lens, slots, page = state["page_table"], state["seqlens"], state["slots"], state["page"]
    rows = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu[1:].long(), rows, right=True)
    count = (cu[1:] - cu[:-1]).long()
    slot = slots.long()[b]
    pos = lens.long()[slot] - count[b] + rows - cu.long()[b]
    at = table.long()[slot, pos // page]
    return at, (pos % page) // BLOCK, pos % BLOCK


def _store(state, cu, k, v):
    T, H = k.shape[0], k.shape[1]
    kb, ks = _quantise(k, state["k_scale"])
    vb, vs = _quantise(v, state["v_scale"])
    at, block, r = _places(state, cu, T)
    pages = state["pages"].view(state["pages"].shape[0], H, state["page"] // BLOCK, BLOCK_BYTES)
    heads = torch.arange(H, device=DEV)
    pages[at[:, None, None], heads[None, :, None], block[:, None, None], _offsets()[r][:, None, :]] = torch.cat(
        (kb, vb, ks, vs), -1)


def _fetch(state, cu, total):
    H = state["pages"].shape[1]
    at, block, r = _places(state, cu, total)
    pages = state["pages"].view(state["pages"].shape[0], H, state["page"] // BLOCK, BLOCK_BYTES)
    heads = torch.arange(H, device=DEV)
    raw = pages[at[:, None, None], heads[None, :, None], block[:, None, None], _offsets()[r][:, None, :]]
    return (_values(raw[..., :32], raw[..., 64:68], state["k_scale"]),
            _values(raw[..., 32:64], raw[..., 68:72], state["v_scale"]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 31))


def _kv(T, H, g):
    """Keys with a few strong channels, values without, as trained models have them."""
    gain = 0.5 + 2.5 * torch.rand((1, H, HEAD_DIM), generator=g, device=DEV) ** 6
    shift = torch.randn((1, H, HEAD_DIM), generator=g, device=DEV) * 0.5
    k = torch.randn((T, H, HEAD_DIM), generator=g, device=DEV) * gain + shift
    v = torch.randn((T, H, HEAD_DIM), generator=g, device=DEV)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _cache(lens, page, kv_heads, g, pool=None, slots=None, columns=None):
    """A cache whose slots hold `lens` tokens in pages that lie in mixed order."""
    held = [-(-int(x) // page) for x in lens]
    used = sum(held)
    pool = used if pool is None else pool
    slots = len(lens) if slots is None else slots
    order = torch.randperm(pool, generator=g, device=DEV)[:used].to(torch.int32).cpu().numpy()
    table = np.full((slots, max(held) if columns is None else columns), -1, dtype=np.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    count = np.zeros(pool, dtype=np.int32)
    count[order] = 1
    sizes = np.zeros(slots, dtype=np.int32)
    sizes[:len(lens)] = lens
    return {"pages": torch.zeros((pool, kv_heads, page * 72), dtype=torch.uint8, device=DEV),
            "page_table": torch.from_numpy(table).to(DEV), "seqlens": torch.from_numpy(sizes).to(DEV),
            "refcount": torch.from_numpy(count).to(DEV), "page": page,
            "k_scale": (0.5 + torch.rand(kv_heads, generator=g, device=DEV)).float(),
            "v_scale": (0.5 + torch.rand(kv_heads, generator=g, device=DEV)).float()}


def _random_bytes(state, g):
    """Pages full of cache-like bytes: any code, scales of ordinary size."""
    pages = state["pages"]
    pages.random_(0, 256, generator=g)
    blocks = pages.view(pages.shape[0], pages.shape[1], state["page"] // BLOCK, BLOCK_BYTES)
    blocks[..., 1024:] = blocks[..., 1024:] % 48 + 24


def _offsets_of(counts):
    return torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "sample":
        return _prepare_sample(case, g)
    if op == "decode":
        lens = _lengths(case["batch"], case["len_lo"], case["len_hi"])
        state = _cache(lens, case["page"], case["kv_heads"], g)
        # filled through the same quantisation as the append does, a few sequences at a time
        step = max(1, (1 << 16) // int(lens.max()))
        for i in range(0, len(lens), step):
            part = dict(state, slots=torch.arange(i, min(len(lens), i + step), device=DEV, dtype=torch.int32))
            n = int(lens[i:i + step].sum())
            k, v = _kv(n, case["kv_heads"], g)
            _store(part, _offsets_of(lens[i:i + step]), k, v)
        rows = case["batch"] * case["rows"]
        state.update(case, slots=torch.arange(case["batch"], device=DEV, dtype=torch.int32),
                     q=(1.5 * torch.randn((rows, case["heads"], HEAD_DIM), generator=g, device=DEV)).to(torch.bfloat16),
                     sink=torch.randn(case["heads"], generator=g, device=DEV))
        return state
    if op == "append":
        new = _lengths(case["batch"], case["new_lo"], case["new_hi"])
        lens = np.maximum(_lengths(case["batch"], case["len_lo"], case["len_hi"]), new)
        state = _cache(lens, case["page"], case["kv_heads"], g)
        k, v = _kv(int(new.sum()), case["kv_heads"], g)
        state.update(case, slots=torch.randperm(case["batch"], generator=g, device=DEV).to(torch.int32), k=k, v=v)
        # entry b serves slot slots[b]: its share of the rows is that slot's
        state["cu"] = _offsets_of(new[state["slots"].cpu().numpy()])
        return state
    if op == "fork":
        P, G, page = case["prompts"], case["group"], case["page"]
        lens = _lengths(P, case["len_lo"], case["len_hi"])
        held = int((-(-lens // page)).sum())
        state = _cache(lens, page, case["kv_heads"], g, pool=held + 2 * P * G + 3, slots=P + P * G,
                       columns=-(-int(lens.max() + 1) // page))
        _random_bytes(state, g)
        state.update(case, src=torch.arange(P, device=DEV, dtype=torch.int32).repeat_interleave(G),
                     dst=(P + torch.randperm(P * G, generator=g, device=DEV)).to(torch.int32),
                     one=torch.ones(P * G, device=DEV, dtype=torch.int32))
        return state
    lens = _lengths(case["slots"], case["len_lo"], case["len_hi"])
    held = int((-(-lens // case["page"])).sum())
    state = _cache(lens, case["page"], case["kv_heads"], g, pool=int(held * case["spare"]) + 1)
    _random_bytes(state, g)
    small = {"pages": torch.zeros((held + 1,) + tuple(state["pages"].shape[1:]), dtype=torch.uint8, device=DEV),
             "page_table": torch.full_like(state["page_table"], -1), "seqlens": torch.zeros_like(state["seqlens"]),
             "refcount": torch.zeros(held + 1, dtype=torch.int32, device=DEV), "k_scale": state["k_scale"].clone(),
             "v_scale": state["v_scale"].clone()}
    state.update(case, small=small)
    return state


def _prepare_sample(case, g):
    B, V = case["batch"], case["vocab"]
    # a few likely tokens and a long tail, as language models give them
    rank = torch.rand((B, V), generator=g, device=DEV).clamp_(min=1e-7).mul_(V).add_(1.0)
    logits = 12.0 - 1.2 * torch.log(rank) + 0.8 * torch.randn((B, V), generator=g, device=DEV)
    full = lambda x, t: torch.full((B,), x, dtype=t, device=DEV)  # noqa: E731
    state = {"temperature": full(case["temperature"], torch.float32), "top_k": full(case["top_k"], torch.int32),
             "top_p": full(case["top_p"], torch.float32), "min_p": full(case["min_p"], torch.float32),
             "u": torch.rand(B, generator=g, device=DEV)}
    if case["mixed"]:
        i = torch.arange(B, device=DEV)
        state["temperature"][i % 7 == 1] = 0.0
        state["temperature"][i % 7 == 2] = 1.0
        state["top_k"][i % 5 == 3] = 0
        state["top_p"][i % 4 == 1] = 1.0
        state["min_p"][i % 3 == 2] = 0.0
        logits[i % 6 == 5, V // 50 + 1:] = -math.inf  # a grammar that allows the first tokens alone
    state["logits"] = logits.to(getattr(torch, case["dtype"]))
    state.update(case={k: v for k, v in case.items()}, op="sample")
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _own_cache(sa, state):
    """The framework's handle of a cache, kept as a user's program keeps it."""
    if "handle" not in state:
        state["handle"] = sa.KV4Cache(*(state[x] for x in ("pages", "page_table", "seqlens", "refcount", "k_scale",
                                                           "v_scale")))
    return state["handle"]


def _run_own(state):
    import sink_aware_masked_gb300 as sa

    op = state["op"]
    if op == "sample":
        return sa.sample_tokens(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                                top_p=state["top_p"], min_p=state["min_p"])
    cache = _own_cache(sa, state)
    if op == "decode":
        if "workspace" not in state:
            state["workspace"] = sa.kv4_decode_workspace(cache, state["q"])
        return sa.kv4_decode_fwd(cache, state["slots"], state["q"], state["sink"], q_per_seq=state["rows"],
                                 window=state["window"], prefix=state["prefix"], workspace=state["workspace"])
    if op == "append":
        sa.kv4_append(cache, state["slots"], state["k"], state["v"], cu_new=state["cu"])
        return sa.kv4_read(cache, state["slots"], state["k"].shape[0], cu=state["cu"])
    if op == "fork":
        sa.kv4_free(cache, state["dst"])
        forked = sa.kv4_fork(cache, state["src"], state["dst"])
        reserved = sa.kv4_reserve(cache, state["dst"], state["one"])
        return forked, reserved, state["page_table"], state["seqlens"], state["refcount"], state["pages"]
    small = state["small"]
    count = sa.kv4_compact(cache, _own_cache(sa, small))
    return count, small["page_table"], small["seqlens"], small["refcount"], small["pages"]


def _run_plain(state):
    op = state["op"]
    if op == "sample":
        return _plain_sample(state)
    if op == "decode":
        return _plain_decode(state)
    if op == "append":
        _store(state, state["cu"], state["k"], state["v"])
        k, v = _fetch(state, state["cu"], state["k"].shape[0])
        return k.to(torch.bfloat16), v.to(torch.bfloat16)
    if op == "fork":
        _plain_free(state, state["dst"])
        forked = _plain_fork(state, state["src"], state["dst"])
        reserved = _plain_reserve(state, state["dst"], state["one"])
        return forked, reserved, state["page_table"], state["seqlens"], state["refcount"], state["pages"]
    return _plain_compact(state, state["small"])


def _plain_decode(state):
    slots, page, n = state["slots"].long(), state["page"], state["rows"]
    B, Hq, H = slots.numel(), state["heads"], state["kv_heads"]
    table, lens = state["page_table"].long()[slots], state["seqlens"].long()[slots]
    raw = state["pages"][table.clamp(min=0)]  # [B, pages, H, bytes]
    raw = raw.view(B, table.shape[1], H, page // BLOCK, BLOCK_BYTES)[..., _offsets()]  # [B, pages, H, blocks, 16, 72]
    raw = raw.permute(0, 1, 3, 4, 2, 5).reshape(B, -1, H, 72)
    k = _values(raw[..., :32], raw[..., 64:68], state["k_scale"]).permute(0, 2, 1, 3)  # [B, H, L, 64]
    v = _values(raw[..., 32:64], raw[..., 68:72], state["v_scale"]).permute(0, 2, 1, 3)
    pos_k = torch.arange(k.shape[2], device=DEV)
    pos_q = lens[:, None] - n + torch.arange(n, device=DEV)  # [B, n]
    seen = pos_k <= pos_q[..., None]
    if state["window"] >= 0:
        seen = seen & ((pos_q[..., None] - pos_k <= state["window"]) | (pos_k < state["prefix"]))
    q = state["q"].float().view(B, n, H, Hq // H, 64).permute(0, 2, 3, 1, 4).reshape(B, H, -1, 64)
    s = torch.matmul(q, k.transpose(2, 3)).view(B, H, Hq // H, n, -1) * 0.125
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    alpha = torch.sigmoid(lse - state["sink"].view(1, H, Hq // H, 1, 1))
    o = torch.matmul((e / total.clamp(min=1e-30)).view(B, H, -1, e.shape[-1]), v).view(B, H, Hq // H, n, 64) * alpha
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, Hq, 64).to(torch.bfloat16)
    return o, lse.view(B, Hq, n).permute(1, 0, 2).reshape(Hq, B * n)


def _plain_free(state, slots):
    table, lens, count = state["page_table"], state["seqlens"], state["refcount"]
    s = slots.long()
    rows = table[s].long()
    held = (lens[s] + state["page"] - 1) // state["page"]
    mine = torch.arange(table.shape[1], device=DEV)[None, :] < held[:, None]
    count.index_add_(0, rows.clamp(min=0).reshape(-1), -mine.to(torch.int32).reshape(-1))
    table[s] = torch.where(mine, torch.full_like(table[s], -1), table[s])
    lens[s] = 0


def _hand_out(state, need):
    """The lowest free pages for requests in order: need [n] -> first place of each in the list, the list, who is served."""
    free = torch.nonzero(state["refcount"] == 0).reshape(-1)
    upto = torch.cumsum(need, 0)
    return upto - need, free, (upto <= free.numel()) | (need == 0)


def _plain_fork(state, src, dst):
    table, lens, count, page = state["page_table"], state["seqlens"], state["refcount"], state["page"]
    s, d = src.long(), dst.long()
    size = lens[s].long()
    need = (size % page != 0).long()
    first, free, ok = _hand_out(state, need)
    row = table[s].long()
    column = torch.arange(table.shape[1], device=DEV)[None, :]
    shared = (column < (size // page)[:, None]) & ok[:, None]
    count.index_add_(0, row.clamp(min=0).reshape(-1), shared.to(torch.int32).reshape(-1))
    fresh = (ok & (need > 0)).nonzero().reshape(-1)
    new = free[first[fresh]]
    count[new] = 1
    old = row[fresh, size[fresh] // page]
    out = torch.where(shared, row, table[d].long())
    out[fresh, size[fresh] // page] = new
    table[d] = out.to(torch.int32)
    lens[d] = torch.where(ok, size, lens[d].long()).to(torch.int32)
    # the last page's blocks that hold tokens
    P, H, nb = state["pages"].shape[0], state["pages"].shape[1], page // BLOCK
    pages = state["pages"].view(P, H, nb, BLOCK_BYTES)
    held = torch.arange(nb, device=DEV)[None, :] * BLOCK < (size[fresh] % page)[:, None]
    pages[new] = torch.where(held[:, None, :, None], pages[old], pages[new])
    return ok.to(torch.int32)


def _plain_reserve(state, slots, new):
    table, lens, count, page = state["page_table"], state["seqlens"], state["refcount"], state["page"]
    s = slots.long()
    size = lens[s].long()
    held, want = -(-size // page), -(-(size + new.long()) // page)
    first, free, ok = _hand_out(state, want - held)
    column = torch.arange(table.shape[1], device=DEV)[None, :]
    take = (column >= held[:, None]) & (column < want[:, None]) & ok[:, None]
    at = (first[:, None] + column - held[:, None]).clamp(0, max(0, free.numel() - 1))
    got = free[at] if free.numel() else torch.zeros_like(at)
    table[s] = torch.where(take, got, table[s].long()).to(torch.int32)
    count.index_add_(0, got.reshape(-1), take.to(torch.int32).reshape(-1))
    lens[s] = torch.where(ok, size + new.long(), size).to(torch.int32)
    return ok.to(torch.int32)


def _plain_compact(state, small):
    count = state["refcount"]
    live = (count > 0).nonzero().reshape(-1)
    place = torch.cumsum((count > 0).long(), 0) - 1
    small["pages"][:live.numel()] = state["pages"][live]
    small["refcount"].zero_()
    small["refcount"][:live.numel()] = count[live]
    table = state["page_table"].long()
    held = (state["seqlens"].long() + state["page"] - 1) // state["page"]
    mine = torch.arange(table.shape[1], device=DEV)[None, :] < held[:, None]
    small["page_table"].copy_(torch.where(mine, place[table.clamp(min=0)], torch.full_like(table, -1)))
    small["seqlens"].copy_(state["seqlens"])
    number = torch.tensor(live.numel(), dtype=torch.int32, device=DEV).reshape(1)
    return number, small["page_table"], small["seqlens"], small["refcount"], small["pages"]


def _plain_sample(state):
    x = state["logits"].double() + 0.0
    B, V = x.shape
    greedy = (state["temperature"] == 0)[:, None]
    T = torch.where(greedy, torch.ones_like(x[:, :1]), state["temperature"].double()[:, None])
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / T)
    whole = e.sum(-1, keepdim=True)
    order = torch.sort(state["logits"].float() + 0.0, dim=-1, descending=True, stable=True)[1]
    k = state["top_k"].long()[:, None]
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, V), k))
    es = e.gather(1, order) * (torch.arange(V, device=DEV)[None, :] < k)
    run = torch.cumsum(es, -1)
    p = state["top_p"].double()[:, None]
    keep = (run - es < p * run[:, -1:]) | (p >= 1.0)
    keep[:, 0] = True
    keep &= (es >= state["min_p"].double()[:, None].clamp(max=1.0)) & (es > 0)
    w = torch.zeros_like(e).scatter_(1, order, es * keep)
    run = torch.cumsum(w, -1)
    total = run[:, -1:]
    token = (run <= state["u"].double()[:, None] * total).sum(-1)
    last = V - 1 - (w > 0).to(torch.int32).flip(-1).argmax(-1)
    token = torch.minimum(token, last)
    mine = (x.gather(1, token[:, None]) - top) / T
    return (token.to(torch.int32), (mine - torch.log(whole)).float().reshape(-1),
            (mine - torch.log(total)).float().reshape(-1))


# ---------------------------------------------------------------- 64 bits, apart from the above
def _e2m1(code):
    sign = 1.0 - 2.0 * (code >> 3).double()
    ex, man = ((code >> 1) & 3).double(), (code & 1).double()
    return sign * torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2(ex - 1.0))


def _e4m3(code):
    c = code.long()
    ex, man = ((c >> 3) & 15).double(), (c & 7).double()
    return torch.where(ex == 0, man * 2.0 ** -9, (1.0 + man / 8.0) * torch.exp2(ex - 7.0))


def _sequence64(state, slot):
    """Keys and values [L, H, 64] of one slot in 64 bits, read from its bytes by the format's own words."""
    L, page = int(state["seqlens"][slot]), state["page"]
    ids = state["page_table"][slot][: -(-L // page)].long()
    raw = state["pages"][ids]  # [n, H, bytes]
    H = raw.shape[1]
    blk = raw.permute(1, 0, 2).reshape(H, -1, BLOCK_BYTES).long()  # [H, blocks, 1152]
    kc = blk[..., :512].reshape(H, -1, 8, 4, 2, 8)                  # g, t, half, byte
    kc = torch.stack((kc & 15, kc >> 4), -1).reshape(H, -1, 8, 4, 2, 16)
    ks = _e4m3(blk[..., 1024:1088]).reshape(H, -1, 8, 4, 2)
    k = (_e2m1(kc) * ks[..., None]).permute(0, 1, 4, 2, 3, 5).reshape(H, -1, 64)  # token = 8 half + g
    vc = blk[..., 512:1024].reshape(H, -1, 8, 4, 2, 2, 4)            # g, t, half, odd, byte
    vc = torch.stack((vc & 15, vc >> 4), -1).reshape(H, -1, 8, 4, 2, 2, 8)
    vs = _e4m3(blk[..., 1088:]).reshape(H, -1, 4, 4, 2, 2).repeat_interleave(2, dim=2)
    v = (_e2m1(vc) * vs[..., None]).permute(0, 1, 4, 3, 5, 2, 6).reshape(H, -1, 64)  # token = 8 half + 2 t + odd
    return (k[:, :L] * state["k_scale"].double()[:, None, None], v[:, :L] * state["v_scale"].double()[:, None, None])


def _exact_decode(case, state):
    n, H, Hq = case["rows"], case["kv_heads"], case["heads"]
    group = Hq // H
    q = state["q"].double().view(case["batch"], n, H, group, 64)
    o = torch.zeros((case["batch"], n, H, group, 64), dtype=torch.float64, device=DEV)
    lse = torch.full((case["batch"], n, H, group), -math.inf, dtype=torch.float64, device=DEV)
    sink = state["sink"].double().view(H, group)
    for b in range(case["batch"]):
        k, v = _sequence64(state, b)
        L = k.shape[1]
        for i in range(n):
            at = L - n + i
            if at < 0:
                continue
            j = torch.arange(at + 1, device=DEV)
            if case["window"] >= 0:
                j = j[(at - j <= case["window"]) | (j < case["prefix"])]
            s = torch.einsum("hgd,hkd->hgk", q[b, i], k[:, j]) / 8.0
            lse[b, i] = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.logaddexp(lse[b, i], sink)[..., None])
            o[b, i] = torch.einsum("hgk,hkd->hgd", p, v[:, j])
    return o.reshape(-1, Hq, 64), lse.reshape(-1, Hq).t().contiguous()


def _exact_quantised(x, factor):
    a = (x.double() / factor.double()[None, :, None]).reshape(x.shape[0], x.shape[1], 4, 16)
    scales = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    scales = torch.tensor(scales[:-1], dtype=torch.float64, device=DEV)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)

    def nearest(values, z):  # the even place of two that are as near
        hi = torch.searchsorted(values, z.contiguous()).clamp(1, len(values) - 1)
        below, above = z - values[hi - 1], values[hi] - z
        return values[torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)]

    s = nearest(scales, (a.abs().amax(-1) / 6.0).clamp(max=448.0))[..., None]
    y = nearest(grid, (a.abs() / torch.where(s > 0, s, torch.ones_like(s))).clamp(max=6.0)) * s * torch.sign(a)
    return y.reshape(x.shape) * factor.double()[None, :, None]


def _exact_sample(state):
    x = state["logits"].double().cpu().numpy()
    u, T, k, p, mp = (state[n].double().cpu().numpy() for n in ("u", "temperature", "top_k", "top_p", "min_p"))
    logp, logq = [], []
    for r in range(x.shape[0]):
        t = 1.0 if T[r] == 0 else T[r]
        z = (x[r] - x[r].max()) / t
        e = np.exp(z)
        order = np.argsort(-x[r], kind="stable")
        count = 1 if T[r] == 0 else int(k[r]) if 0 < k[r] < x.shape[1] else x.shape[1]
        order = order[:count]
        if p[r] < 1.0:
            run = np.cumsum(e[order])
            order = order[:max(1, int(np.searchsorted(run, p[r] * run[-1], side="left")) + 1)]
        chosen = np.sort(order[(e[order] >= min(1.0, mp[r])) & (e[order] > 0)])
        run = np.cumsum(e[chosen])
        i = chosen[min(int(np.searchsorted(run, u[r] * run[-1], side="right")), len(chosen) - 1)]
        logp.append(z[i] - np.log(e.sum()))
        logq.append(z[i] - np.log(run[-1]))
    return torch.tensor(logp, dtype=torch.float64), torch.tensor(logq, dtype=torch.float64)


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers alone
    state = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, state)
    if case["op"] == "append":
        return (_exact_quantised(state["k"], state["k_scale"]), _exact_quantised(state["v"], state["v_scale"]))
    return (None,) + _exact_sample(state)
