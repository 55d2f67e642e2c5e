"""CPU oracle of the rollout-side operators: the 4-bit paged cache, its page handling and token sampling.

Plain loops over the definitions (include/sinkattn.h), float64 throughout;
shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values():
    """The value of each of the 256 bytes (0x7f and 0xff are NaN)."""
    b = np.arange(256)
    e, m, s = (b >> 3) & 15, b & 7, np.where(b >= 128, -1.0, 1.0)
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))
    v[(b & 127) == 127] = np.nan
    return s * v


E4M3 = e4m3_values()


def _nearest_even(values, x):
    """Index of the nearest of ascending `values` (even index of two as near), saturating."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    below, above = x - values[hi - 1], values[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, factor):
    """x [..., 64] -> (codes uint8 [..., 64], scale bytes uint8 [..., 4])."""
    y = (np.asarray(x, dtype=np.float64) / factor).reshape(*x.shape[:-1], 4, 16)
    finite = np.isfinite(y).all(-1)
    y = np.where(finite[..., None], y, 0.0)
    scale = _nearest_even(E4M3[:127], np.minimum(np.abs(y).max(-1) / 6, 448.0))
    s = E4M3[scale][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s > 0, np.abs(y) / s, 0.0)
    code = _nearest_even(CODES[:8], np.minimum(z, 6.0)) + np.where((y < 0), 8, 0)
    scale = np.where(finite, scale, 0x7F)
    return code.astype(np.uint8).reshape(x.shape), scale.astype(np.uint8)


def values(codes, scales, factor):
    """The values the codes stand for, [..., 64]."""
    y = CODES[codes].reshape(*codes.shape[:-1], 4, 16) * E4M3[scales][..., None]
    return y.reshape(codes.shape) * factor


class Cache:
    """The cache as numpy arrays of its bytes and tables."""

    def __init__(self, num_pages, num_slots, max_pages, heads, page_size, k_scale=None, v_scale=None):
        self.pages = np.zeros((num_pages, heads, page_size * 72), dtype=np.uint8)
        self.table = np.full((num_slots, max_pages), -1, dtype=np.int32)
        self.lens = np.zeros(num_slots, dtype=np.int32)
        self.ref = np.zeros(num_pages, dtype=np.int32)
        self.heads, self.page_size = heads, page_size
        self.k_scale = np.ones(heads, dtype=np.float32) if k_scale is None else k_scale
        self.v_scale = np.ones(heads, dtype=np.float32) if v_scale is None else v_scale

    # ---- bytes of one token: (page, offset of its block, row in the block)
    def _block(self, slot, pos):
        page = self.table[slot, pos // self.page_size]
        return page, (pos % self.page_size) // 16 * 1152, pos % 16

    def write(self, slot, pos, head, k_codes, k_scales, v_codes, v_scales):
        page, base, r = self._block(slot, pos)
        mem = self.pages[page, head]
        kb, vb = k_codes[0::2] | (k_codes[1::2] << 4), v_codes[0::2] | (v_codes[1::2] << 4)
        g, half = r % 8, r // 8
        t, i = (r % 8) // 2, r % 2 + 2 * half
        for lane_t in range(4):
            at = base + 16 * (4 * g + lane_t) + 8 * half
            mem[at:at + 8] = kb[8 * lane_t:8 * lane_t + 8]
            mem[base + 1024 + 2 * (4 * g + lane_t) + half] = k_scales[lane_t]
            mem[base + 1088 + 4 * (4 * lane_t + t) + i] = v_scales[lane_t]
        for lane_g in range(8):
            at = base + 512 + 16 * (4 * lane_g + t) + 4 * i
            mem[at:at + 4] = vb[4 * lane_g:4 * lane_g + 4]

    def token(self, slot, pos, head):
        """(k [64], v [64]) float64."""
        page, base, r = self._block(slot, pos)
        mem = self.pages[page, head]
        g, half = r % 8, r // 8
        t, i = (r % 8) // 2, r % 2 + 2 * half
        kb = np.concatenate([mem[base + 16 * (4 * g + x) + 8 * half:][:8] for x in range(4)])
        vb = np.concatenate([mem[base + 512 + 16 * (4 * x + t) + 4 * i:][:4] for x in range(8)])
        ks = np.array([mem[base + 1024 + 2 * (4 * g + x) + half] for x in range(4)])
        vs = np.array([mem[base + 1088 + 4 * (4 * x + t) + i] for x in range(4)])
        nibbles = lambda b: np.stack([b & 15, b >> 4], -1).reshape(-1)  # noqa: E731
        return (values(nibbles(kb), ks, float(self.k_scale[head])), values(nibbles(vb), vs, float(self.v_scale[head])))

    def fill(self, slot, k, v, first=0):
        """Quantises k, v [n, heads, 64] into positions first .. of a slot whose pages are there."""
        for h in range(self.heads):
            kc, ks = quantise(k[:, h], float(self.k_scale[h]))
            vc, vs = quantise(v[:, h], float(self.v_scale[h]))
            for j in range(k.shape[0]):
                self.write(slot, first + j, h, kc[j], ks[j], vc[j], vs[j])

    def sequence(self, slot):
        """Keys and values [len, heads, 64] float64 of a slot."""
        L = int(self.lens[slot])
        k, v = np.zeros((L, self.heads, 64)), np.zeros((L, self.heads, 64))
        for pos in range(L):
            for h in range(self.heads):
                k[pos, h], v[pos, h] = self.token(slot, pos, h)
        return k, v

    # ---- page handling, one request after the other
    def _pages_of(self, tokens):
        return -(-int(tokens) // self.page_size)

    def _in_order(self, needs):
        """Which requests get their pages: in order, until one does not fit."""
        free = int((self.ref == 0).sum())
        total, out = 0, []
        for need in needs:
            total += need
            out.append(need == 0 or total <= free)
        return out

    def _take(self, count):
        pages = np.nonzero(self.ref == 0)[0][:count]
        self.ref[pages] = 1
        return pages

    def reserve(self, slots, new):
        S, seen, needs, valid = len(self.lens), set(), [], []
        for s, n in zip(slots, new):
            ok = 0 <= s < S and s not in seen and n >= 0
            ok = ok and int(self.lens[s]) + int(n) <= self.table.shape[1] * self.page_size
            seen.add(int(s))
            valid.append(ok)
            needs.append(self._pages_of(self.lens[s] + n) - self._pages_of(self.lens[s]) if ok else 0)
        served = self._in_order(needs)
        done = [int(a and b) for a, b in zip(valid, served)]
        for s, n, need, ok in zip(slots, new, needs, done):
            if ok:
                held = self._pages_of(self.lens[s])
                self.table[s, held:held + need] = self._take(need)
                self.lens[s] += n
        return np.array(done, dtype=np.int32)

    def fork(self, src, dst):
        S, seen, needs, valid = len(self.lens), set(), [], []
        before = self.lens.copy()
        for a, b in zip(src, dst):
            ok = 0 <= a < S and 0 <= b < S and b not in seen and before[b] == 0
            seen.add(int(b))
            valid.append(ok)
            needs.append(int(ok and before[a] % self.page_size != 0))
        done = [int(a and b) for a, b in zip(valid, self._in_order(needs))]
        for a, b, need, ok in zip(src, dst, needs, done):
            if not ok:
                continue
            full = int(before[a]) // self.page_size
            self.table[b, :full] = self.table[a, :full]
            for p in self.table[a, :full]:
                self.ref[p] += 1
            if need:
                page, old = self._take(1)[0], self.table[a, full]
                self.table[b, full] = page
                used = -(-(int(before[a]) % self.page_size) // 16) * 1152
                self.pages[page, :, :used] = self.pages[old, :, :used]
            self.lens[b] = before[a]
        return np.array(done, dtype=np.int32)

    def free(self, slots):
        for s in slots:
            if 0 <= s < len(self.lens):
                held = self._pages_of(self.lens[s])
                for p in self.table[s, :held]:
                    self.ref[p] -= 1
                self.table[s, :held] = -1
                self.lens[s] = 0


def kept_tokens(x, u, temperature, top_k, top_p, min_p):
    """One valid row in float64: (z, sum of all e, kept indices ascending, their cumulated masses, u times the kept
    mass), with z the scaled logits less their largest."""
    x = np.asarray(x, dtype=np.float64) + 0.0
    z = (x - x.max()) / (1.0 if temperature == 0 else temperature)
    e = np.exp(z)
    order = np.argsort(-x, kind="stable")
    if temperature == 0 or top_p <= 0:
        order = order[:1]
    elif 0 < top_k < len(x):
        order = order[:top_k]
    if 0 < top_p < 1:
        run = np.cumsum(e[order])
        order = order[:min(len(order), int(np.searchsorted(run, top_p * run[-1])) + 1)]
    kept = np.sort(order[(e[order] >= min(min_p, 1.0)) & (e[order] > 0)])
    run = np.cumsum(e[kept])
    return z, e.sum(), kept, run, min(max(u, 0.0), 1.0 - 2.0 ** -24) * run[-1]


def sample_invalid(x, u, temperature, top_k, top_p, min_p):
    """What an invalid row gives for logp and logq (token -1): NaN, or -inf where nothing is allowed; None if valid."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan([u, temperature, top_p, min_p]).any() or not 0 <= temperature <= 1e36:
        return float("nan")
    if np.isnan(x).any() or np.isposinf(x).any():
        return float("nan")
    return -np.inf if np.isneginf(x).all() else None


def sample(x, u, temperature, top_k, top_p, min_p):
    """One row: (token, logp, logq)."""
    bad = sample_invalid(x, u, temperature, top_k, top_p, min_p)
    if bad is not None:
        return -1, bad, bad
    z, total, kept, run, at = kept_tokens(x, u, temperature, top_k, top_p, min_p)
    i = min(int(np.searchsorted(run, at, side="right")), len(kept) - 1)
    return int(kept[i]), z[kept[i]] - np.log(total), z[kept[i]] - np.log(run[-1])
