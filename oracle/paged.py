"""Oracle of the paged 4-bit memory: page tables, quantised rows, page selection and decode
attention over requests of different lengths, row by row in plain numpy.

Quantisation is part of the definition, in correctly rounded 32-bit arithmetic; everything
after it is fp64."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["round_bf16", "quantise_row", "row_values", "strip_image", "PagedModel"]


def round_bf16(x):
    """fp32 values rounded to the nearest bf16 (ties to even), as fp32."""
    x = np.asarray(x, np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, x).astype(np.float32)


def quantise_row(row):
    """(codes int [D], scales fp32 [groups]) of one row of fp32 values, groups of 32 dims."""
    row = np.asarray(row, np.float32)
    codes, scales = np.zeros(len(row), int), []
    for a in range(0, len(row), 32):
        x = row[a:a + 32]
        if not np.isfinite(x).all():
            scales.append(np.float32(np.nan))
            continue
        s = round_bf16(np.float32(np.abs(x).max()) / np.float32(7))
        if s < np.float32(2.0 ** -100):
            scales.append(np.float32(0))
            continue
        scales.append(np.float32(s))
        inv = np.float32(1) / np.float32(s)
        codes[a:a + 32] = np.clip(np.rint(x * inv), -7, 7).astype(int)
    return codes, np.array(scales, np.float32)


def row_values(codes, scales):
    """fp64 values that codes and scales stand for."""
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32)[:len(codes)]


def strip_image(k_rows, v_rows, P):
    """Bytes of a strip from its rows' (codes, scales), None for a row not written: (bytes, mask
    of the bits that the rows determine)."""
    G = P // 32
    n = 16 * P + 64 * G
    image, mask = np.zeros(n, np.uint8), np.zeros(n, np.uint8)

    def nibble(bit, value):
        image[bit // 8] |= value << (bit % 8)
        mask[bit // 8] |= 15 << (bit % 8)

    for which, rows in enumerate((k_rows, v_rows)):
        for t, row in enumerate(rows):
            if row is None:
                continue
            codes = np.zeros(P, int)
            codes[:len(row[0])] = row[0]
            scales = np.zeros(G, np.float32)
            scales[:len(row[1])] = row[1]
            for d in range(P):
                g = d // 32
                if which == 0:
                    c, j = d % 32 // 8, d % 8
                    bit = 32 * ((4 * t + c) * G + g) + 4 * j
                else:
                    lane, j = d % 32 // 4, d % 4
                    unit = ((8 * (t // 8) + lane) * 4 + t % 8 // 2) * 2 * G + 2 * g + t % 2
                    bit = 8 * 8 * P + 16 * unit + 4 * j
                nibble(bit, codes[d] + 8)
            for g in range(G):
                at = 16 * P + (t * 2 * G + which * G + g) * 2
                bits = 0x7FFF if np.isnan(scales[g]) else int(scales[g].view(np.uint32) >> 16)
                image[at], image[at + 1] = bits & 255, bits >> 8
                mask[at] = mask[at + 1] = 255
    return image, mask


class PagedModel:
    """The memory as lists: a free stack, a table and a length per request, rows per slot."""

    def __init__(self, heads, dim, page, n_pages, requests, columns):
        self.heads, self.dim, self.page, self.columns = heads, dim, page, columns
        self.n_pages = n_pages
        self.free = list(range(n_pages - 1, -1, -1))
        self.tables = [[] for _ in range(requests)]
        self.lens = [0] * requests
        self.rows = {}  # slot -> (k [heads][dim], v [heads][dim]) as stored values, fp64
        self.reps = {}  # page -> [heads][dim] mean of its stored keys

    def extend(self, new, n_slots):
        """Slots of the new tokens, or None (and no change) where the call is refused."""
        if min(new, default=0) < 0 or sum(new) > n_slots:
            return None
        pages = [-(-(self.lens[r] + n) // self.page) for r, n in enumerate(new)]
        need = sum(p - len(self.tables[r]) for r, p in enumerate(pages))
        if need > len(self.free) or max(pages, default=0) > self.columns:
            return None
        slots = []
        for r, n in enumerate(new):
            for pos in range(self.lens[r], self.lens[r] + n):
                if pos // self.page == len(self.tables[r]):
                    self.tables[r].append(self.free.pop())
                slots.append(self.tables[r][pos // self.page] * self.page + pos % self.page)
            self.lens[r] += n
        return slots

    def truncate(self, keep):
        back = []
        for r, n in enumerate(keep):
            self.lens[r] = min(self.lens[r], n)
            held = -(-self.lens[r] // self.page)
            back += self.tables[r][held:]
            self.tables[r] = self.tables[r][:held]
        self.free += back[::-1]

    def append(self, slots, k, v):
        """k, v [n][heads][dim] fp32."""
        for i, s in enumerate(slots):
            if s < 0 or s // self.page >= self.n_pages:
                continue
            self.rows[s] = tuple(
                np.stack([row_values(*quantise_row(x[i, h])) for h in range(self.heads)])
                for x in (k, v))
        for s in slots:
            if s >= 0 and s // self.page < self.n_pages and s % self.page == self.page - 1:
                p = s // self.page
                self.reps[p] = np.mean([self.rows[p * self.page + i][0]
                                        for i in range(self.page)], axis=0)

    def parts(self, r, sink, window):
        """(sink end, first window token, candidate pages) of request r."""
        T, full = self.lens[r], self.lens[r] // self.page
        w0 = min(max(T - window, 0), full * self.page)
        cand = [j for j in range(full) if (j + 1) * self.page > sink and j * self.page < w0]
        return min(sink, w0), w0, cand

    def select(self, q, k, sink, window):
        """q [R][Hq][dim] -> idx [R][heads][k]; scores rounded once to fp32."""
        R, group = len(q), q.shape[1] // self.heads
        idx = np.full((R, self.heads, k), -1)
        for r in range(R):
            cand = self.parts(r, sink, window)[2]
            for h in range(self.heads):
                s = q[r, h * group:(h + 1) * group].astype(np.float64).sum(0)
                score = [np.float32((s * self.reps[self.tables[r][j]][h]).sum()) for j in cand]
                best = sorted(range(len(cand)), key=lambda i: (-score[i], i))[:k]
                got = sorted(cand[i] for i in best)
                idx[r, h, :len(got)] = got
        return idx

    def attend(self, q, idx, sink, window, scale):
        """(out [R][Hq][dim], lse [R][Hq], largest |v|, bound of the logits' error in units of
        2^-24) in fp64."""
        R, Hq = q.shape[:2]
        group = Hq // self.heads
        out, lse = np.zeros((R, Hq, self.dim)), np.full((R, Hq), -np.inf)
        vmax, unit = 0.0, 0.0
        for r in range(R):
            end, w0, cand = self.parts(r, sink, window)
            for h in range(self.heads):
                seen = set(range(end)) | set(range(w0, self.lens[r]))
                for j in [] if idx is None else idx[r, h][:len(cand)]:
                    seen |= {t for t in range(j * self.page, (j + 1) * self.page) if end <= t < w0}
                if not seen:
                    continue
                rows = [self.rows[self.tables[r][t // self.page] * self.page + t % self.page]
                        for t in sorted(seen)]
                K, V = (np.stack([x[i][h] for x in rows]) for i in (0, 1))
                vmax = max(vmax, np.abs(V).max())
                Q = q[r, h * group:(h + 1) * group].astype(np.float64)
                x = scale * Q @ K.T
                # the products run over codes 1 .. 15 times the scale: at most 15 / 7 of the
                # group's largest key
                top = np.repeat([np.abs(K[:, a:a + 32]).max(1) for a in range(0, self.dim, 32)],
                                32, axis=0)[:self.dim]
                unit = max(unit, (scale * np.abs(Q) @ top).max() * 15 / 7, np.abs(x).max())
                m = x.max(1, keepdims=True)
                w = np.exp(x - m)
                out[r, h * group:(h + 1) * group] = w @ V / w.sum(1, keepdims=True)
                lse[r, h * group:(h + 1) * group] = (m + np.log(w.sum(1, keepdims=True)))[:, 0]
        return out, lse, vmax, unit
