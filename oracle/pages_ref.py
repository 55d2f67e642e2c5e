"""CPU oracle of the rollout with drafted tokens: pages of bf16 keys and values, and the verification of drafts.

Plain loops over the definitions (include/sinkattn.h), float64 throughout;
shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


class Pages:
    """Tables and pools as numpy arrays; keys and values float64 (hold bf16 values in them)."""

    def __init__(self, num_pages, num_slots, max_pages, heads, page_size):
        self.k = np.zeros((num_pages, page_size, heads, 64))
        self.v = np.zeros((num_pages, page_size, heads, 64))
        self.table = np.full((num_slots, max_pages), -1, dtype=np.int32)
        self.lens = np.zeros(num_slots, dtype=np.int32)
        self.owner = np.full(num_pages, -1, dtype=np.int32)
        self.heads, self.page_size = heads, page_size

    def pages_of(self, tokens):
        return -(-int(tokens) // self.page_size)

    def place(self, slot, pos):
        return int(self.table[slot, pos // self.page_size]) * self.page_size + pos % self.page_size

    def plan(self, slots, drop, new, total):
        """(live, cu, slot_map, positions), request by request."""
        table_tokens = self.table.shape[1] * self.page_size
        valid = [0 <= s < len(self.lens) and s not in slots[:i] and new[i] >= 0 for i, s in enumerate(slots)]
        for s, d, ok in zip(slots, drop, valid):
            if not ok:
                continue
            left = max(int(self.lens[s]) - max(int(d), 0), 0)
            for col in range(self.pages_of(left), self.pages_of(self.lens[s])):
                page = self.table[s, col]
                if 0 <= page < len(self.owner) and self.owner[page] == s:
                    self.owner[page] = -1
                self.table[s, col] = -1
            self.lens[s] = left
        free = list(np.flatnonzero(self.owner == -1))
        live, slot_map, positions, out_of_pages = [], [], [], False
        for s, n, ok in zip(slots, new, valid):
            left = int(self.lens[s]) if ok else 0
            ok = ok and left + n <= table_tokens
            need = self.pages_of(left + n) - self.pages_of(left) if ok else 0
            if need > 0 and (out_of_pages or need > len(free)):
                out_of_pages, ok = True, False
            if ok:
                for col in range(self.pages_of(left), self.pages_of(left) + need):
                    self.table[s, col] = free.pop(0)
                    self.owner[self.table[s, col]] = s
                self.lens[s] = left + n
            live.append(s if ok else -1)
            slot_map += [self.place(s, left + i) if ok else -1 for i in range(max(n, 0))]
            positions += [left + i if ok else -1 for i in range(max(n, 0))]
        cu = np.concatenate(([0], np.cumsum([max(n, 0) for n in new]))).astype(np.int32)
        pad = [-1] * max(total - len(slot_map), 0)
        return (np.array(live, dtype=np.int32), cu, np.array((slot_map + pad)[:total], dtype=np.int32),
                np.array((positions + pad)[:total], dtype=np.int32))

    def write(self, slot_map, k, v):
        for r, place in enumerate(slot_map):
            if 0 <= place < self.k.shape[0] * self.page_size:
                page, row = divmod(int(place), self.page_size)
                self.k[page, row], self.v[page, row] = k[r], v[r]

    def sequence(self, slot):
        """Keys and values [len, heads, 64] of a slot; NaN where its page is not in the pool."""
        L = int(self.lens[slot])
        k, v = (np.full((L, self.heads, 64), np.nan) for _ in range(2))
        for pos in range(L):
            page = self.table[slot, pos // self.page_size] if pos // self.page_size < self.table.shape[1] else -1
            if 0 <= page < len(self.owner):
                k[pos], v[pos] = self.k[page, pos % self.page_size], self.v[page, pos % self.page_size]
        return k, v


def softmax(x, temperature):
    """(probabilities, their logarithms) of one row, or a NaN or -inf for a row that has none."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.nan
    if np.isneginf(x).all():
        return -np.inf
    with np.errstate(divide="ignore"):
        z = (x - x.max()) / temperature
        logp = z - np.log(np.exp(z).sum())
    return np.exp(logp), logp


def verify(x, y, drafts, u, temperature):
    """One entry: x [n, V] target logits, y [n - 1, V] draft logits or None, drafts [n - 1], u [n].

    Returns (tokens [n], logp [n], accepted, weights, border): the weights the
    last token was drawn from (None where it was not drawn), and the smallest
    distance of a test from equality, |u q - p|.
    """
    n = len(x)
    tokens, logp = np.full(n, -1), np.zeros(n)
    greedy, border, weights = temperature == 0, np.inf, None
    T = 1.0 if greedy else temperature
    clamp = lambda t: 0.0 if np.isnan(t) else min(max(t, 0.0), float(np.float32(0.99999994)))  # noqa: E731
    if np.isnan(temperature) or temperature < 0 or temperature > 1e36:
        logp[0] = np.nan
        return tokens, logp, 0, None, border
    for i in range(n):
        p = softmax(x[i], T)
        q = None
        if not isinstance(p, tuple):
            logp[i] = p
            return tokens, logp, i, None, border
        if i < n - 1:
            d = int(drafts[i])
            inside = 0 <= d < x.shape[1]
            if greedy:
                stands = inside and d == int(np.argmax(x[i]))
            else:
                q = np.zeros(x.shape[1])
                if y is not None:
                    q = softmax(y[i], T)
                    if not isinstance(q, tuple):
                        logp[i] = np.nan
                        return tokens, logp, i, None, border
                    q = q[0]
                elif inside:
                    q[d] = 1.0
                stands = inside and clamp(u[i]) * q[d] < p[0][d]
                if inside and p[0][d] > 0:  # (what the target never gives never stands)
                    border = min(border, abs(clamp(u[i]) * q[d] - p[0][d]))
            if stands:
                tokens[i], logp[i] = d, p[1][d]
                continue
        if greedy:
            tokens[i] = int(np.argmax(x[i]))
        else:
            weights = p[0] if q is None else np.maximum(p[0] - q, 0.0)
            if y is None and q is not None and inside:
                weights[d] = 0.0
            if not weights.sum() > 0:
                weights = p[0]
            run = np.cumsum(weights)
            tokens[i] = min(int(np.searchsorted(run, clamp(u[n - 1]) * run[-1], side="right")),
                            int(np.flatnonzero(weights)[-1]))
        logp[i] = p[1][tokens[i]]
        return tokens, logp, i, weights, border
