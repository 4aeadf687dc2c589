"""CPU oracle of the paged 3-bit KV cache: the block layout, the page calls
served one entry after the other, and the attention in fp64. Plain numpy,
written from the definitions; shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

from oracle import bitlinear_oracle as O

PAGE = 64


def block_bytes(D: int) -> int:
    return PAGE * (2 * (3 * D // 8) + 8)


def append(pages, codes4, k_bits, v_bits, slots, row4=None):
    """Write tokens (bf16 bits [n x H x D]) into the slots of `pages`
    [n_pages x H x block] (and `codes4` [n_pages x H x C4 x D]), in place."""
    n, H, D = k_bits.shape
    rb = 3 * D // 8
    keep = np.flatnonzero(np.asarray(row4) >= 0) if row4 is not None else np.zeros(0, np.int64)
    stores = [O.kv_quant_3bit(x, keep) for x in (k_bits, v_bits)]
    rank = {int(t): j for j, t in enumerate(keep)}
    for i in range(n):
        if slots[i] < 0:
            continue
        p, o = divmod(int(slots[i]), PAGE)
        four = i in rank
        for h in range(H):
            blk = pages[p, h]
            kr, vr = stores[0][0][i, h].copy(), stores[1][0][i, h]
            ks, vs = stores[0][2][i, h], stores[1][2][i, h]
            if four:
                kr[0] = row4[i]
                codes4[p, h, row4[i], :D // 2] = stores[0][1][rank[i], h]
                codes4[p, h, row4[i], D // 2:] = stores[1][1][rank[i], h]
                ks = -ks
            blk[o * rb:(o + 1) * rb] = kr
            at = PAGE * rb + (o // 4) * 4 * rb + o % 4
            blk[at:at + 4 * rb:4] = vr
            s = blk[2 * PAGE * rb:].view(np.float32)
            s[o], s[PAGE + o] = ks, vs


def read(pages, codes4, page, o, D):
    """(k, v) [H x D] in fp64 of token o of a page."""
    rb = 3 * D // 8
    H = pages.shape[1]
    out = np.zeros((2, H, D))
    for h in range(H):
        blk = pages[page, h]
        at = PAGE * rb + (o // 4) * 4 * rb + o % 4
        rows = (blk[o * rb:(o + 1) * rb], blk[at:at + 4 * rb:4])
        s = blk[2 * PAGE * rb:].view(np.float32).astype(np.float64)
        four = np.signbit(s[o])
        for w in range(2):
            scale = abs(s[w * PAGE + o])
            if four:
                b = codes4[page, h, rows[0][0], w * D // 2:(w + 1) * D // 2]
                c = np.stack([b & 15, b >> 4], 1).reshape(-1).astype(np.int64) - 8
            else:
                bits = np.unpackbits(rows[w], bitorder="little").reshape(D, 3)
                c = bits @ np.array([1, 2, 4]) - 4
            out[w, h] = c * scale
    return out[0], out[1]


def pages_of(n: int) -> int:
    return -(-n // PAGE)


class Tables:
    """Sequences' tables, lengths and reference counts, with the page calls."""

    def __init__(self, R, W, n_pages, pages, codes4=None):
        self.tables = np.full((R, W), -1, np.int32)
        self.lens = np.zeros(R, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.pages, self.codes4 = pages, codes4  # [L x n_pages x ...]

    def copy(self, src, dst):
        self.pages[:, dst] = self.pages[:, src]
        if self.codes4 is not None:
            self.codes4[:, dst] = self.codes4[:, src]

    def fork(self, parents, children):
        for p, c in zip(parents, children):
            m = pages_of(int(self.lens[p]))
            self.tables[c, :m] = self.tables[p, :m]
            for page in self.tables[p, :m]:
                self.refs[page] += 1
            self.lens[c] = self.lens[p]

    def free(self, rows, keep=None):
        for i, r in enumerate(rows):
            k = 0 if keep is None else int(keep[i])
            if k >= self.lens[r]:
                continue
            for page in self.tables[r, pages_of(k):pages_of(int(self.lens[r]))]:
                self.refs[page] -= 1
            self.lens[r] = k

    def grow(self, rows, n_new, max_new):
        """Slots [n x max_new]; None if the pool has too few free pages. The free pages
        are those of before the call: a page that an entry leaves is still the others'."""
        free = list(np.flatnonzero(self.refs == 0))
        state = (self.tables.copy(), self.lens.copy(), self.refs.copy())
        slots = np.full((len(rows), max_new), -1, np.int32)
        copies = []
        for i, (r, add) in enumerate(zip(rows, n_new)):
            n, have = int(self.lens[r]), pages_of(int(self.lens[r]))
            want = pages_of(n + int(add)) - have
            cow = add > 0 and n % PAGE != 0 and self.refs[self.tables[r, have - 1]] > 1
            if want + cow > len(free):
                self.tables, self.lens, self.refs = state
                return None
            if cow:
                old, new = self.tables[r, have - 1], free.pop(0)
                copies.append((old, new))
                self.refs[old] -= 1
                self.refs[new] = 1
                self.tables[r, have - 1] = new
            for j in range(want):
                self.tables[r, have + j] = free.pop(0)
                self.refs[self.tables[r, have + j]] = 1
            for u in range(int(add)):
                slots[i, u] = self.tables[r, (n + u) // PAGE] * PAGE + (n + u) % PAGE
            self.lens[r] = n + int(add)
        for s, d in copies:
            self.copy(s, d)
        return slots

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        for s, d in zip(movers, holes):
            self.copy(s, d)
            self.refs[d], self.refs[s] = self.refs[s], 0
            for r in range(len(self.lens)):
                m = pages_of(int(self.lens[r]))
                t = self.tables[r, :m]
                t[t == s] = d
        return live

    def held(self):
        """The tables' entries that say something, the others -1."""
        t = np.full_like(self.tables, -1)
        for r, n in enumerate(self.lens):
            t[r, :pages_of(int(n))] = self.tables[r, :pages_of(int(n))]
        return t


def attention(q_bits, pages, codes4, tables, lens, shared=()):
    """(o, A): the fp64 attention of q [B x Sq x Hq x D] (bf16 bits) over one layer's
    pages, and A = sum_t p_t |v_t|."""
    q = O.bf16_to_f32(q_bits).astype(np.float64)
    B, Sq, Hq, D = q.shape
    H = pages.shape[1]
    o, A = np.zeros(q.shape), np.zeros(q.shape)
    known = {}

    def rows(page, m):  # its first m tokens
        if (page, m) not in known:
            kv = [read(pages, codes4, page, i, D) for i in range(m)]
            known[page, m] = np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv])
        return known[page, m]

    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        ids = (list(shared) + list(tables[b]))[:pages_of(n)]
        kv = [rows(int(p), min(PAGE, n - PAGE * j)) for j, p in enumerate(ids)]
        k, v = (np.concatenate([x[w] for x in kv]) for w in range(2))
        for i in range(Sq):
            m = n - Sq + 1 + i
            if m <= 0:
                continue
            for hq in range(Hq):
                h = hq // (Hq // H)
                s = k[:m, h] @ q[b, i, hq] / np.sqrt(D)
                p = np.exp(s - s.max())
                p /= p.sum()
                o[b, i, hq] = p @ v[:m, h]
                A[b, i, hq] = p @ np.abs(v[:m, h])
    return o, A
