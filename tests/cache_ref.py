"""Plain 64-bit references of the cache operators, lane by lane and slot by
slot, written from their definitions (numpy, no code of the library)."""
import numpy as np


def bf16_bits(x):
    """float -> bf16 bit patterns, round to nearest even."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32)


class RefCache:
    """Tables, lengths, references and bf16 bit patterns of a paged cache."""

    def __init__(self, k, v, table, length, ref):
        self.k, self.v = k.copy(), v.copy()
        self.table, self.len, self.ref = table.copy(), length.copy(), ref.copy()
        self.page = k.shape[3]

    def where(self, lane, slot):
        return self.table[lane, slot // self.page], slot % self.page

    def fork(self, parent):
        old, length = self.table.copy(), self.len.copy()
        for i, p in enumerate(parent):
            self.table[i] = old[p] if p >= 0 else -1
            self.len[i] = length[p] if p >= 0 else 0
        for e in old[old >= 0]:
            self.ref[e] -= 1
        for e in self.table[self.table >= 0]:
            self.ref[e] += 1

    def reserve(self, want):
        saved = (self.table.copy(), self.ref.copy())
        copies = []

        taken = set()  # a page freed by nothing here: each taken page is a new one

        def take():
            free = [p for p in np.flatnonzero(self.ref == 0) if p not in taken]
            if not free:
                raise MemoryError
            taken.add(free[0])
            return free[0]
        try:
            for b, w in enumerate(want):
                if w <= 0:
                    continue
                n = int(self.len[b])
                # the pages under the slots n .. n + w - 1
                for col in range(n // self.page, -(-(n + int(w)) // self.page)):
                    if col >= self.table.shape[1]:
                        raise MemoryError
                    p = self.table[b, col]
                    if p >= 0 and self.ref[p] <= 1:
                        continue  # the lane's own already
                    d = take()
                    if p >= 0:
                        if n > col * self.page:
                            copies.append((p, d, n - col * self.page))
                        self.ref[p] -= 1
                    self.ref[d] = 1
                    self.table[b, col] = d
        except MemoryError:
            self.table, self.ref = saved
            return False
        for p, d, n in copies:
            self.k[:, d, :, :n] = self.k[:, p, :, :n]
            self.v[:, d, :, :n] = self.v[:, p, :, :n]
        return True

    def release(self, b, n):
        for col in range(-(-n // self.page), self.table.shape[1]):
            if self.table[b, col] >= 0:
                self.ref[self.table[b, col]] -= 1
                self.table[b, col] = -1

    def trim(self, new_len):
        for b, n in enumerate(new_len):
            self.len[b] = min(self.len[b], max(int(n), 0))
            self.release(b, int(self.len[b]))

    def compact(self, count, path=None):
        for b, n in enumerate(count):
            base = int(self.len[b])
            if path is not None:
                moved = []
                for j in range(int(n)):
                    p, r = self.where(b, base + int(path[b][j]))
                    moved.append((self.k[:, p, :, r].copy(), self.v[:, p, :, r].copy()))
                for j, (k, v) in enumerate(moved):
                    p, r = self.where(b, base + j)
                    self.k[:, p, :, r], self.v[:, p, :, r] = k, v
            self.len[b] = base + int(n)
            self.release(b, int(self.len[b]))


def rope(y, heads, dim, positions, pair_axis, inv_freq, style):
    """Rotated rows [rows][heads][dim] of y in 64 bits, and |x| + |y| of each value's pair."""
    x = y.astype(np.float64).reshape(-1, heads, dim)
    out, mag = x.copy(), np.abs(x)
    half = len(inv_freq)
    for i in range(half):
        a, b = (i, i + half) if style == 0 else (2 * i, 2 * i + 1)
        ang = positions[pair_axis[i]].astype(np.float64) * inv_freq[i]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    return out, mag


def attention(ref, layer, q, scale, row_start, mask):
    """(out, lse, weighted |v|, score error bound) of rows q [rows][heads][dim] (float), each row's slots one by one.

    The score's 32-bit error: D products and sums of |q k| magnitude, each within 2^-24 of it, then the scaling."""
    rows, heads, dim = q.shape
    hkv = ref.k.shape[2]
    out = np.zeros((rows, heads, dim))
    lse = np.full((rows, heads), -np.inf)
    wabs = np.zeros((rows, heads, dim))
    err = np.zeros((rows, heads))
    seen = np.zeros(rows, int)
    for b in range(len(row_start) - 1):
        lo, hi = int(row_start[b]), int(row_start[b + 1])
        for r in range(lo, hi):
            n = int(ref.len[b])
            bits = (1 << (r - lo + 1)) - 1 if mask is None else int(mask[r])
            slots = list(range(n)) + [n + j for j in range(hi - lo) if bits >> j & 1]
            slots = [s for s in slots if s // ref.page < ref.table.shape[1] and
                     0 <= ref.table[b, s // ref.page] < ref.k.shape[1]]
            seen[r] = len(slots)
            if not slots:
                continue
            pg = np.array([ref.where(b, s)[0] for s in slots])
            of = np.array([s % ref.page for s in slots])
            k = bf16_value(ref.k[layer][pg, :, of]).astype(np.float64)  # [slots][kv heads][dim]
            v = bf16_value(ref.v[layer][pg, :, of]).astype(np.float64)
            for h in range(heads):
                kh = h // (heads // hkv)
                with np.errstate(all="ignore"):
                    s = scale * (k[:, kh] @ q[r, h])
                    top = s.max()
                    p = np.exp(s - top)
                    tot = p.sum()
                    lse[r, h] = top + np.log(tot)
                    out[r, h] = (p / tot) @ v[:, kh]
                    wabs[r, h] = (p / tot) @ np.abs(v[:, kh])
                    err[r, h] = (dim + 4) * 2.0**-24 * np.max(abs(scale) * (np.abs(k[:, kh]) @ np.abs(q[r, h])))
    return out, lse, wabs, err, seen


def beam(logits, scores, finished, eos):
    """(scores, parent, token, finished) of each group, candidates listed and sorted."""
    groups, beams = scores.shape
    V = logits.shape[1]
    o_s = np.full((groups, beams), -np.inf)
    o_p, o_t = np.full((groups, beams), -1), np.full((groups, beams), -1)
    o_f = np.zeros((groups, beams), np.uint8)
    for g in range(groups):
        key, place = [], []
        for w in range(beams):
            m = g * beams + w
            cum = float(scores[g, w])
            if finished is not None and finished[g, w]:
                key.append(np.array([cum]))
                place.append(np.array([w * V + eos]))
                continue
            x = logits[m].astype(np.float64)
            with np.errstate(all="ignore"):
                top = x.max()
                c = cum + (x - (top + np.log(np.exp(x - top).sum())))
            key.append(c)
            place.append(w * V + np.arange(V))
        key, place = np.concatenate(key), np.concatenate(place)
        ok = key > -np.inf
        key, place = key[ok], place[ok]
        order = np.lexsort((place, -key))[:beams]
        n = len(order)
        o_s[g, :n] = key[order]
        o_p[g, :n] = g * beams + place[order] // V
        o_t[g, :n] = place[order] % V
        for j in range(n):
            par = o_p[g, j] - g * beams
            o_f[g, j] = o_t[g, j] == eos or (finished is not None and finished[g, par] != 0)
    return o_s, o_p, o_t, o_f
