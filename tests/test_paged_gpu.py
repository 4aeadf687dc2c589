"""The paged 3-bit cache on the GPU against the oracle: stored bytes, tables and
counts equal; attention within the tolerance that tolerance() derives."""
import numpy as np
import pytest
import torch

import bit_quantised_gemm_b200 as B
from bit_quantised_gemm_b200 import _lib
from oracle import bitlinear_oracle as O
from oracle import paged_oracle as P
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def up(bits):
    return W.bf16_bits_to_torch(bits).to(DEV)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def fresh():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,n", [(1, 1), (3, 7), (4, 64), (5, 201), (32, 33)])
def test_append(D, H, n):
    """Consecutive slots from an odd place on, over page borders, every fifth token left
    out; k and v slices of one projection's output; the other bytes stay."""
    rng = np.random.default_rng(100 * D + 10 * H + n)
    qkv = W.normal_bf16(rng, (n, (1 + 2 * H) * D))
    k, v = qkv[:, D:(1 + H) * D].reshape(n, H, D), qkv[:, (1 + H) * D:].reshape(n, H, D)
    n_pages = (n + 13) // 64 + 2
    order = rng.permutation(n_pages)
    slots = np.array([order[(13 + i) // 64] * 64 + (13 + i) % 64 for i in range(n)])
    slots[4::5] = -1
    row4 = np.full(n, -1)
    row4[::9] = (np.arange(n)[::9] // 9) % 3  # nine tokens apart: at most 8 a page, rows repeat only across pages
    seen = set()
    for i in range(n):  # distinct rows within a page
        if row4[i] >= 0 and slots[i] >= 0:
            if (slots[i] // 64, row4[i]) in seen:
                row4[i] = -1
            seen.add((slots[i] // 64, row4[i]))
    want, want4 = np.full((n_pages, H, P.block_bytes(D)), 0x5A, np.uint8), np.full((n_pages, H, 3, D), 0x5A, np.uint8)
    pages, codes4 = torch.from_numpy(want.copy()).to(DEV), torch.from_numpy(want4.copy()).to(DEV)
    P.append(want, want4, k, v, slots, row4)
    t = up(qkv)
    st = fresh()
    B.kv_append_3bit(t[:, D:(1 + H) * D].unflatten(1, (H, D)), t[:, (1 + H) * D:].unflatten(1, (H, D)), ints(slots), pages,
                     row4=ints(row4), codes4=codes4, status=st)
    assert np.array_equal(pages.cpu().numpy(), want)
    assert np.array_equal(codes4.cpu().numpy(), want4)
    assert st.item() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_aligned_run(D):
    """Whole pages in order, then the same tokens backwards: the slots decide, not the tokens' order."""
    rng = np.random.default_rng(D)
    n, H = 192, 2
    k, v = W.normal_bf16(rng, (n, H, D)), W.normal_bf16(rng, (n, H, D))
    for slots in (np.arange(n), np.arange(n)[::-1].copy(), np.arange(n) // 64 * 64 + (np.arange(n) * 5 + 2) % 64):
        want = np.zeros((3, H, P.block_bytes(D)), np.uint8)
        P.append(want, None, k, v, slots)
        pages, _ = B.kv_page_pool(3, H, D, device=DEV)
        B.kv_append_3bit(up(k), up(v), ints(slots), pages)
        assert np.array_equal(pages.cpu().numpy(), want)


@pytest.mark.parametrize("D,H", [(64, 3), (128, 2), (256, 5)])
@pytest.mark.parametrize("first", [0, 4, 13, 60])
def test_append_prompt(D, H, first):
    """A prompt from some place of a page on, with padding behind it, then with one token at 4 bits in its middle:
    whole runs of tokens, runs cut by page borders, and tokens alone at both ends."""
    rng = np.random.default_rng(D + first)
    n = 150
    k, v = W.normal_bf16(rng, (n, H, D)), W.normal_bf16(rng, (n, H, D))
    n_pages = (first + n + 63) // 64
    order = rng.permutation(n_pages)
    slots = np.array([order[(first + i) // 64] * 64 + (first + i) % 64 for i in range(n)])
    slots[n - 5:] = -1
    for row4 in (np.full(n, -1), np.where(np.arange(n) == 70, 1, -1)):
        want, want4 = np.full((n_pages, H, P.block_bytes(D)), 0x5A, np.uint8), np.full((n_pages, H, 2, D), 0x5A, np.uint8)
        pages, codes4 = torch.from_numpy(want.copy()).to(DEV), torch.from_numpy(want4.copy()).to(DEV)
        P.append(want, want4, k, v, slots, row4)
        B.kv_append_3bit(up(k), up(v), ints(slots), pages, row4=ints(row4), codes4=codes4)
        assert np.array_equal(pages.cpu().numpy(), want) and np.array_equal(codes4.cpu().numpy(), want4)


def test_append_values_at_borders():
    """Zero rows (the scale's floor), tiny and large rows, exact ties of the codes."""
    D, H = 128, 2
    x = np.zeros((6, H, D), np.float32)
    x[1] = 1e-6
    x[2] = 3e38
    x[3, :, :8] = [3, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -3]
    x[4, :, :4] = [7, 0.5, 3.5, -6.5]
    x[5] = -2.0
    k = O.f32_to_bf16(x)
    want, want4 = np.zeros((1, H, P.block_bytes(D)), np.uint8), np.zeros((1, H, 1, D), np.uint8)
    row4 = np.array([-1, -1, -1, -1, 0, -1])
    P.append(want, want4, k, k, np.arange(6), row4)
    pages, codes4 = B.kv_page_pool(1, H, D, rows4=1, device=DEV)
    B.kv_append_3bit(up(k), up(k), ints(np.arange(6)), pages, row4=ints(row4), codes4=codes4)
    assert np.array_equal(pages.cpu().numpy(), want) and np.array_equal(codes4.cpu().numpy(), want4)


def test_append_leaves_bad_indexes_out():
    rng = np.random.default_rng(0)
    D, H, n = 64, 2, 6
    k = W.normal_bf16(rng, (n, H, D))
    slots, row4 = np.array([5, 128, 7, 1 << 30, 9, 10]), np.array([-1, -1, 2, -1, -1, 0])
    want, want4 = np.zeros((2, H, P.block_bytes(D)), np.uint8), np.zeros((2, H, 2, D), np.uint8)
    good = np.array([0, 4, 5])
    P.append(want, want4, k[good], k[good], slots[good], row4[good])
    pages, codes4 = B.kv_page_pool(2, H, D, rows4=2, device=DEV)
    st = fresh()
    B.kv_append_3bit(up(k), up(k), ints(slots), pages, row4=ints(row4), codes4=codes4, status=st)
    assert np.array_equal(pages.cpu().numpy(), want) and np.array_equal(codes4.cpu().numpy(), want4)
    with pytest.raises(B.BitlinearError) as e:
        B.check_status(st)
    assert e.value.code == _lib.ERR_INDEX


# -------------------------------------------------------------- page calls
class Both:
    """The oracle's tables and the device's, through the same calls."""

    def __init__(self, R, W_, n_pages, L=2, H=2, D=64, C4=1, seed=0, lead=0):
        rng = np.random.default_rng(seed)
        pages = rng.integers(0, 256, (L, n_pages, H, P.block_bytes(D)), np.uint8)
        codes4 = rng.integers(0, 256, (L, n_pages, H, C4, D), np.uint8) if C4 else None
        self.o = P.Tables(R, W_, n_pages, pages, codes4)
        self.pages = torch.from_numpy(pages.copy()).to(DEV)
        self.codes4 = torch.from_numpy(codes4.copy()).to(DEV) if C4 else None
        self.wide = torch.full((R, W_ + lead), -7, dtype=torch.int32, device=DEV)
        self.tables = self.wide[:, :W_]  # rows W + lead apart
        self.lens, self.refs = ints(self.o.lens), ints(self.o.refs)
        self.st = fresh()

    def same(self, status=0):
        assert np.array_equal(self.lens.cpu().numpy(), self.o.lens)
        assert np.array_equal(self.refs.cpu().numpy(), self.o.refs)
        got, held = self.tables.cpu().numpy(), self.o.held()
        assert np.array_equal(np.where(held < 0, -1, got), held)
        assert np.array_equal(self.pages.cpu().numpy(), self.o.pages)
        if self.codes4 is not None:
            assert np.array_equal(self.codes4.cpu().numpy(), self.o.codes4)
        assert (self.wide[:, self.tables.shape[1]:] == -7).all()
        assert self.st.item() == status
        self.st.zero_()

    def grow(self, rows, n_new, max_new=None):
        max_new = max(n_new) if max_new is None else max_new
        want = self.o.grow(rows, n_new, max_new)
        got = B.kv_pages_grow(self.pages, self.tables, self.lens, self.refs, ints(rows), ints(n_new), max_new,
                              codes4=self.codes4, status=self.st)
        assert np.array_equal(got.cpu().numpy(), np.full((len(rows), max_new), -1) if want is None else want)
        self.same(_lib.STATUS_NO_PAGES if want is None else 0)

    def fork(self, parents, children):
        self.o.fork(parents, children)
        B.kv_pages_fork(self.tables, self.lens, self.refs, ints(parents), ints(children), status=self.st)
        self.same()

    def free(self, rows, keep=None):
        self.o.free(rows, keep)
        B.kv_pages_free(self.tables, self.lens, self.refs, ints(rows), keep=None if keep is None else ints(keep),
                        status=self.st)
        self.same()

    def compact(self):
        want = self.o.compact()
        got = B.kv_pages_compact(self.pages, self.tables, self.lens, self.refs, codes4=self.codes4, status=self.st)
        assert got.item() == want
        self.same()


@pytest.mark.parametrize("seed", range(4))
def test_page_calls_in_a_run(seed):
    """Random calls, the pool sometimes too small, against the oracle after every one."""
    rng = np.random.default_rng(seed)
    R = 12
    b = Both(R, 6, int(rng.integers(20, 40)), C4=seed % 2, seed=seed, lead=seed)
    for _ in range(40):
        live = np.flatnonzero(b.o.lens > 0)
        empty = np.flatnonzero(b.o.lens == 0)
        what = rng.integers(0, 5)
        if what == 0 and len(live) and len(empty):
            kids = rng.permutation(empty)[:rng.integers(1, 4)]
            b.fork(rng.choice(live, len(kids)), kids)
        elif what in (1, 2):
            rows = rng.permutation(R)[:rng.integers(1, R + 1)]
            room = 6 * 64 - b.o.lens[rows]
            add = np.minimum(rng.choice([0, 1, 1, 5, 64, 100], len(rows)), room)
            b.grow(rows, add, max(1, int(add.max())))
        elif what == 3 and len(live):
            rows = rng.permutation(live)[:rng.integers(1, 4)]
            b.free(rows, rng.integers(0, 200, len(rows)) if rng.random() < 0.5 else None)
        elif what == 4:
            b.compact()


def test_grow_many_on_one_page():
    """A parent and 40 children leave one partly filled page: all but the last copy it."""
    b = Both(64, 3, 140)
    b.grow([3], [70])
    b.fork([3] * 40, list(range(4, 44)))
    b.grow(list(range(43, 2, -1)), [1, 59, 0, 60] * 10 + [2], 60)
    b.free(list(range(10, 30)))
    b.compact()


def test_grow_the_largest_call():
    """1024 entries, a pool of more pages than one walk's step."""
    b = Both(1024, 2, 20000, L=1, H=1, C4=0)
    b.o.refs[:18000] = 1
    b.refs[:18000] = 1
    b.grow(list(range(1024)), [1 + (i % 100) for i in range(1024)])
    b.grow(list(range(1024)), [1] * 1024)


def test_page_calls_leave_bad_entries_out():
    b = Both(6, 2, 12)
    b.grow([0, 1], [100, 64])
    tables = b.tables.clone()
    # a row twice, a row that is none, a length behind the table's end, too many tokens
    got = B.kv_pages_grow(b.pages, b.tables, b.lens, b.refs, ints([2, 2, 6, -1, 0, 3]), ints([5, 6, 1, 1, 29, 30]), 29,
                          codes4=b.codes4, status=b.st).cpu().numpy()
    want = b.o.grow([2], [5], 29)
    assert np.array_equal(got[0], want[0]) and (got[1:] == -1).all()
    b.same(_lib.STATUS_BAD_INDEX)
    # children: named twice, holding tokens, a parent too, no row; parents: no row
    B.kv_pages_fork(b.tables, b.lens, b.refs, ints([0, 1, 1, 3, 0, 9]), ints([3, 3, 0, 4, 6, 5]), status=b.st)
    b.same(_lib.STATUS_BAD_INDEX)  # row 0 is a child here, so the first entry is left out as well
    B.kv_pages_fork(b.tables, b.lens, b.refs, ints([0, 1, 1]), ints([3, 3, 4]), status=b.st)
    b.o.fork([0, 1], [3, 4])
    b.same(_lib.STATUS_BAD_INDEX)
    # freed twice in a call: once; rows that are none
    B.kv_pages_free(b.tables, b.lens, b.refs, ints([0, 0, 7, -3]), status=b.st)
    b.o.free([0])
    b.same(_lib.STATUS_BAD_INDEX)
    # a table entry outside the pool is passed over
    b.tables[1, 0] = 99
    B.kv_pages_free(b.tables, b.lens, b.refs, ints([1]), status=b.st)
    assert b.st.item() == _lib.STATUS_BAD_INDEX and b.refs.min().item() >= 0
    st = fresh()
    before = b.pages.clone()
    B.kv_pages_copy(b.pages, ints([0, 12, -1, -1]), ints([12, 1, 3, -1]), codes4=b.codes4, status=st)
    assert st.item() == _lib.STATUS_BAD_INDEX and torch.equal(before, b.pages)
    assert tables.shape == b.tables.shape


@pytest.mark.parametrize("L,H,D,C4", [(1, 1, 64, 0), (3, 5, 128, 2), (2, 8, 256, 1)])
def test_copy(L, H, D, C4):
    rng = np.random.default_rng(L)
    b = Both(1, 1, 23, L, H, D, C4)
    at = rng.permutation(23)
    src, dst = at[:11].copy(), at[11:22].copy()
    b.o.copy(src, dst)
    B.kv_pages_copy(b.pages, ints(src), ints(dst), codes4=b.codes4, status=b.st)
    b.same()
    if L == 1:
        B.kv_pages_copy(b.pages[0], ints(dst[:1]), ints(at[22:]))
        b.o.copy(dst[:1], at[22:])
        b.same()


# --------------------------------------------------------------- attention
def tolerance(o, A, n=1024):
    """bf16's rounding, half a step: 2^-8 |o|. The sums: scores, weights and values are
    formed in 32 bits: 2^-16 (A + |o|) with A = sum p |v| (as for the contiguous
    cache's attention). Weights as 16-bit floats, where a kernel takes them so: half a
    step of fp16, 2^-11 of each weight, so at most 2^-11 A. Weights as whole numbers,
    where a kernel takes them so: the largest is 2^29 at least, so half a unit is 2^-30 of
    it; times codes of up to 8 for each of n tokens. A row's largest code is 3 or more, so
    the largest weight is at most a third of A's largest value: n 2^-30 8/3 max A < n 2^-28 max A."""
    return (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -16) * (A + np.abs(o))
            + n * 2.0 ** -28 * A.max(-1, keepdims=True, initial=0))


def pool(rng, n_pages, H, D, C4, spread=1.0):
    """Random pages, all slots filled; with C4, some tokens of each page at 4 bits."""
    pages = np.zeros((n_pages, H, P.block_bytes(D)), np.uint8)
    codes4 = np.zeros((n_pages, H, C4, D), np.uint8) if C4 else None
    n = n_pages * 64
    x = rng.standard_normal((2, n, H, D), np.float32) * np.exp(spread * rng.standard_normal((2, n, H, 1), np.float32) / 2)
    row4 = np.full(n, -1)
    for j in range(C4):
        row4[np.arange(n_pages) * 64 + rng.permutation(64)[j]] = j
    P.append(pages, codes4, O.f32_to_bf16(x[0]), O.f32_to_bf16(x[1]), np.arange(n), row4)
    return pages, codes4


def check(q, pages, codes4, tables, lens, shared, **kw):
    B_, Sq = q.shape[:2]
    st = fresh()
    got = B.kv_attention_3bit_paged(up(q), torch.from_numpy(pages).to(DEV), ints(tables), ints(lens), shared=ints(shared),
                                    codes4=None if codes4 is None else torch.from_numpy(codes4).to(DEV), status=st, **kw)
    o, A = P.attention(q, pages, codes4, tables, lens, shared)
    err = np.abs(O.bf16_to_f32(bits(got)).astype(np.float64) - o)
    assert st.item() == 0
    bound = tolerance(o, A, max(lens)) + 1e-30
    assert (err <= bound).all(), (err / bound).max()
    return got


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,Sq,C4,shared", [(1, 1, 1, 0, 0), (2, 1, 1, 1, 2), (3, 2, 1, 0, 1), (2, 4, 1, 2, 3), (1, 8, 2, 0, 2),
                                              (2, 3, 5, 1, 0), (1, 1, 7, 0, 1)])
def test_attention(D, H, G, Sq, C4, shared):
    """Lengths around page borders, none, fewer tokens than queries, inside the shared pages; the
    places behind the last token and the unused table entries hold rubbish."""
    rng = np.random.default_rng(D + 7 * H + G + Sq)
    own = [0, 1, 63, 64, 65, 130, 2, 190]
    lens = np.array([0 if n == 0 else 64 * shared + n for n in own])
    if shared:
        lens[6] = 64 * shared - 5  # ends inside the shared pages
    Bn, W_ = len(own), 4
    mine = [max(0, P.pages_of(int(n)) - shared) for n in lens]
    n_pages = shared + sum(mine) + 2
    pages, codes4 = pool(rng, n_pages, H, D, C4)
    order = rng.permutation(n_pages)
    head, tables, at = order[:shared], np.full((Bn, W_), 1 << 30), shared
    rb = 3 * D // 8
    for b, m in enumerate(mine):
        tables[b, :m] = order[at:at + m]
        at += m
        if m and lens[b] % 64:  # what no token has written
            blk, n = pages[tables[b, m - 1]], int(lens[b]) % 64
            for o in range(n, 64):
                blk[:, o * rb:(o + 1) * rb] = 0xFF
                v = 64 * rb + (o // 4) * 4 * rb + o % 4
                blk[:, v:v + 4 * rb:4] = 0xFF
                blk[:, 2 * 64 * rb + 4 * o:2 * 64 * rb + 4 * o + 4] = 0xFF        # NaN
                blk[:, 2 * 64 * rb + 256 + 4 * o:2 * 64 * rb + 256 + 4 * o + 4] = [0, 0, 0x80, 0x7F]  # infinity
    q = W.normal_bf16(rng, (Bn, Sq, H * G, D))
    got = check(q, pages, codes4, tables, lens, head)
    assert (got[0] == 0).all()  # no token: zeros


@pytest.mark.parametrize("Bn,G,Sq", [(12, 1, 1), (33, 1, 1), (130, 1, 1), (20, 4, 1), (9, 8, 2), (40, 2, 3)])
@pytest.mark.parametrize("D,shared", [(64, 5), (128, 1), (128, 6), (256, 3)])
def test_attention_many_rows_on_a_prefix(Bn, G, Sq, D, shared):
    """Row counts on both sides of the tiles' sizes, odd and even numbers of shared pages."""
    rng = np.random.default_rng(Bn + G + Sq + D + shared)
    H = 2
    own = rng.integers(Sq, 80, Bn)
    own[1], own[Bn // 2] = 0, 64
    lens = 64 * shared + own
    lens[2], lens[3] = 0, 64 * shared - 63
    tables = np.zeros((Bn, 2), np.int64)
    pages, codes4 = pool(rng, shared + 4, H, D, 1)
    tables[:] = shared + rng.integers(0, 4, (Bn, 2))  # sequences may share any page
    q = W.normal_bf16(rng, (Bn, Sq, H * G, D))
    check(q, pages, codes4, tables, lens, rng.permutation(shared))


@pytest.mark.parametrize("D,shared,C4", [(64, 7, 0), (64, 2, 5), (128, 9, 0), (128, 1, 1), (128, 5, 6), (256, 3, 0), (256, 6, 4)])
@pytest.mark.parametrize("Bn", [17, 128, 260, 300])
def test_attention_tiles_on_a_prefix(D, shared, C4, Bn):
    """One tile of rows, two, and an odd one beside a pair; odd and even numbers of pages, one page; more 4-bit
    rows a page than travel with it; sequences that end before, inside and at the end of the prefix."""
    rng = np.random.default_rng(D + shared + Bn)
    pages, codes4 = pool(rng, shared + 2, 1, D, C4)
    lens = 64 * shared + rng.integers(0, 40, Bn)
    lens[0], lens[5], lens[6], lens[Bn // 2] = 0, 64 * shared - 1, 1, 64 * shared
    tables = shared + rng.integers(0, 2, (Bn, 1))
    q = W.normal_bf16(rng, (Bn, 1, 1, D))
    got = check(q, pages, codes4, tables, lens, rng.permutation(shared))
    assert (got[0] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_tiles_unwritten_and_bad(D):
    """What no token has written behind the last one of the prefix counts for nothing, and a page that is none is
    passed over, 4-bit rows out of range are left out; both are reported."""
    rng = np.random.default_rng(D)
    Bn, shared = 40, 4
    pages, codes4 = pool(rng, 6, 2, D, 1)
    rb = 3 * D // 8
    blk = pages[3]
    for o in range(20, 64):  # page 3, the prefix's last: 20 tokens
        blk[:, o * rb:(o + 1) * rb] = 0xFF
        at = 64 * rb + (o // 4) * 4 * rb + o % 4
        blk[:, at:at + 4 * rb:4] = 0xFF
        blk[:, 128 * rb + 4 * o:128 * rb + 4 * o + 4] = 0xFF
        blk[:, 128 * rb + 256 + 4 * o:128 * rb + 256 + 4 * o + 4] = [0, 0, 0x80, 0x7F]
    q = W.normal_bf16(rng, (Bn, 1, 2, D))
    lens = rng.integers(1, 64 * 3 + 20, Bn)
    lens[3] = 64 * 3 + 20
    none = np.zeros((Bn, 0), np.int64)
    check(q, pages, codes4, none, lens, [0, 1, 2, 3])
    # a page that is none: as if its tokens were not there
    dev = (up(q), torch.from_numpy(pages).to(DEV), ints(none).view(Bn, 0), ints(np.full(Bn, 64 * 3)))
    c4 = torch.from_numpy(codes4).to(DEV)
    st = fresh()
    got = B.kv_attention_3bit_paged(*dev, shared=ints([0, 6, 2]), codes4=c4, status=st)
    assert st.item() == _lib.STATUS_BAD_INDEX
    want, A = P.attention(q, pages, codes4, none, np.full(Bn, 128), [0, 2])
    err = np.abs(O.bf16_to_f32(bits(got)).astype(np.float64) - want)
    assert (err <= tolerance(want, A)).all()
    # the 4-bit token of each page without its row: left out
    st = fresh()
    got = B.kv_attention_3bit_paged(*dev[:3], ints(np.full(Bn, 64)), shared=ints([1]), status=st)
    assert st.item() == _lib.STATUS_BAD_INDEX
    o4 = int(np.flatnonzero(np.signbit(pages[1, 0, 128 * rb:].view(np.float32)[:64]))[0])
    keep = np.array([o for o in range(64) if o != o4])
    kv = [P.read(pages, codes4, 1, o, D) for o in keep]
    k, v = (np.stack([x[i] for x in kv]) for i in range(2))
    for h in range(2):
        s = np.einsum("bd,td->bt", O.bf16_to_f32(q[:, 0, h]).astype(np.float64), k[:, h]) / np.sqrt(D)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want, A = p @ v[:, h], p @ np.abs(v[:, h])
        err = np.abs(O.bf16_to_f32(bits(got))[:, 0, h].astype(np.float64) - want)
        assert (err <= tolerance(want, A)).all()


@pytest.mark.parametrize("G", [1, 4, 8])
def test_attention_one_page_many_times(G):
    """A table that names one page 1.25 million times, more than 500 times for each warp: the answer is the page's own."""
    rng = np.random.default_rng(G)
    D, W_ = 64, 148 * 2 * 8 * 530
    pages, _ = pool(rng, 1, 1, D, 0)
    q = W.normal_bf16(rng, (1, 1, G, D))
    st = fresh()
    got = B.kv_attention_3bit_paged(up(q), torch.from_numpy(pages).to(DEV), torch.zeros(1, W_, dtype=torch.int32, device=DEV),
                                    ints([64 * W_]), status=st)
    o, A = P.attention(q, pages, None, np.zeros((1, 1), int), [64])
    # 530 pages of 4 steps, each rounding a sum of up to 7/4 of 4/3 A by 2^-23: 2120 * 7/3 * 2^-23 < 2^-10
    bound = tolerance(o, A) + 2.0 ** -10 * A.max(-1, keepdims=True)
    assert st.item() == 0 and (np.abs(O.bf16_to_f32(bits(got)) - o) <= bound).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_one_shared_page_many_times(D):
    """The same for the tiles: a prefix that is one page 20000 times."""
    rng = np.random.default_rng(D)
    pages, _ = pool(rng, 1, 2, D, 0)
    n, Bn = 20000, 40
    q = W.normal_bf16(rng, (Bn, 1, 2, D))
    st = fresh()
    got = B.kv_attention_3bit_paged(up(q), torch.from_numpy(pages).to(DEV), torch.zeros(Bn, 0, dtype=torch.int32, device=DEV),
                                    ints(np.full(Bn, 64 * n)), shared=ints(np.zeros(n)), status=st)
    o, A = P.attention(q, pages, None, np.zeros((Bn, 1), int), np.full(Bn, 64))
    # up to 20000 / 18 pages a stream, 4 steps each, as above
    bound = tolerance(o, A) + 2.0 ** -9 * A.max(-1, keepdims=True)
    assert st.item() == 0 and (np.abs(O.bf16_to_f32(bits(got)) - o) <= bound).all()


def test_attention_more_sequences_than_threads():
    """Lengths are summed by chunks of sequences, and a warp finds its place between them."""
    rng = np.random.default_rng(14)
    D, Bn = 64, 700
    pages, _ = pool(rng, 6, 1, D, 0)
    lens = np.where(rng.integers(0, 3, Bn) == 0, 0, rng.integers(0, 130, Bn))
    q = W.normal_bf16(rng, (Bn, 1, 1, D))
    check(q, pages, None, rng.integers(0, 6, (Bn, 3)), lens, [])


@pytest.mark.parametrize("D,G", [(64, 1), (128, 1), (128, 4), (256, 2)])
def test_attention_long(D, G):
    """Long enough that one sequence's pages go to many warps, two lengths far apart."""
    rng = np.random.default_rng(D + G)
    pages, codes4 = pool(rng, 6, 1, D, 1)
    lens = np.array([64 * 230 + 17, 9])
    tables = rng.integers(0, 6, (2, 231))
    q = W.normal_bf16(rng, (2, 1, G, D))
    check(q, pages, codes4, tables, lens, [])


def test_attention_sharp_and_flat():
    """Scores so large that one token takes all, values of very different sizes, and scores of zero (the mean)."""
    rng = np.random.default_rng(5)
    D, H = 128, 2
    pages, codes4 = pool(rng, 8, H, D, 0, spread=6.0)
    tables, lens = rng.permutation(8).reshape(2, 4), np.array([256, 201])
    q = W.normal_bf16(rng, (2, 1, H, D))
    big = O.f32_to_bf16(O.bf16_to_f32(q) * 64)
    check(big, pages, codes4, tables, lens, [])
    check(np.zeros_like(q), pages, codes4, tables, lens, [])


def test_attention_strided_queries_and_given_output():
    rng = np.random.default_rng(6)
    D, H, G, Bn = 128, 2, 2, 5
    pages, _ = pool(rng, 6, H, D, 0)
    tables, lens = rng.integers(0, 6, (Bn, 3)), np.array([100, 0, 192, 64, 1])
    qkv = up(W.normal_bf16(rng, (Bn, 8, D)))
    p, wide = torch.from_numpy(pages).to(DEV), ints(np.concatenate([tables, tables + 100], 1))
    out = torch.full((Bn, 1, H * G, D), 7.0, dtype=torch.bfloat16, device=DEV)
    got = B.kv_attention_3bit_paged(qkv[:, None, 2:6], p, wide[:, :3], ints(lens), out=out)
    assert got.data_ptr() == out.data_ptr()
    want = B.kv_attention_3bit_paged(qkv[:, None, 2:6].contiguous(), p, ints(tables), ints(lens))
    assert torch.equal(got, want)


def test_attention_leaves_bad_indexes_out():
    """Pages outside the pool are passed over and reported; lengths are cut to the table."""
    rng = np.random.default_rng(7)
    D, H = 128, 2
    pages, _ = pool(rng, 5, H, D, 0)
    p = torch.from_numpy(pages).to(DEV)
    q = up(W.normal_bf16(rng, (3, 1, H, D)))
    for shared in (None, ints([4])):
        base = 0 if shared is None else 64
        st = fresh()
        got = B.kv_attention_3bit_paged(q, p, ints([[0, 5, 1], [2, 3, -9], [2, 1, 0]]), ints([base + 192, base + 150, base + 500]),
                                        shared=shared, status=st)
        assert st.item() == _lib.STATUS_BAD_INDEX
        st = fresh()
        want = B.kv_attention_3bit_paged(q, p, ints([[0, 1, 1], [2, 3, 0], [2, 1, 0]]), ints([base + 128, base + 128, base + 192]),
                                         shared=shared, status=st)
        assert st.item() == 0
        assert (got.float() - want.float()).abs().max().item() <= 2.0 ** -6 * want.float().abs().max().item()
    # a negative length is an empty sequence
    st = fresh()
    got = B.kv_attention_3bit_paged(q, p, ints([[0], [1], [2]]), ints([-5, 3, 0]), status=st)
    assert st.item() == _lib.STATUS_BAD_INDEX and (got[0] == 0).all() and (got[2] == 0).all() and (got[1] != 0).any()


def test_attention_without_pages():
    q = up(W.normal_bf16(np.random.default_rng(8), (2, 1, 4, 64)))
    pages, _ = B.kv_page_pool(1, 2, 64, device=DEV)
    none = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    assert (B.kv_attention_3bit_paged(q, pages, none, ints([0, 0])) == 0).all()
    assert B.kv_attention_3bit_paged(q[:0], pages, none[:0], ints([])).shape == (0, 1, 4, 64)


def test_offsets_beyond_32_bits():
    """A pool of more than 4 GB: its last pages are appended to, copied and attended to."""
    D, H = 64, 64
    n_pages = (1 << 32) // (P.block_bytes(D) * H) + 9
    pages = torch.empty(n_pages, H, P.block_bytes(D), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(9)
    n = 70
    k, v, q = W.normal_bf16(rng, (n, H, D)), W.normal_bf16(rng, (n, H, D)), W.normal_bf16(rng, (1, 1, H, D))
    last = [n_pages - 1, n_pages - 3]
    slots = [last[i // 64] * 64 + i % 64 for i in range(n)]
    B.kv_append_3bit(up(k), up(v), ints(slots), pages)
    small = np.zeros((2, H, P.block_bytes(D)), np.uint8)
    P.append(small, None, k, v, np.arange(n))
    o, A = P.attention(q, small, None, [[0, 1]], [n])
    for table in (last, [n_pages - 2, 0]):
        got = B.kv_attention_3bit_paged(up(q), pages, ints([table]), ints([n]))
        assert (np.abs(O.bf16_to_f32(bits(got)) - o) <= tolerance(o, A)).all()
        B.kv_pages_copy(pages, ints(last), ints([n_pages - 2, 0]))


# -------------------------------------------------------------- a run of all
def decode_run(H, D, G, steps, stream=None, graph=False, seed=11):
    """A prompt, its forks, some steps of every sequence, one sequence given up, the pool compacted: each
    step's attention against the oracle's on the oracle's own pages."""
    rng = np.random.default_rng(seed)
    L, R, W_, n_pages, C4 = 2, 5, 5, 24, 1
    sim = P.Tables(R, W_, n_pages, np.zeros((L, n_pages, H, P.block_bytes(D)), np.uint8),
                   np.zeros((L, n_pages, H, C4, D), np.uint8))
    pages, codes4 = B.kv_page_pool(n_pages, H, D, layers=L, rows4=C4, device=DEV)
    tables = torch.full((R, W_), -1, dtype=torch.int32, device=DEV)
    lens, refs = ints(np.zeros(R)), ints(np.zeros(n_pages))
    st = fresh()
    kw = dict(status=st, stream=stream)

    def append(slots, flat, row4):
        for layer in range(L):
            k, v = W.normal_bf16(rng, (len(flat), H, D)), W.normal_bf16(rng, (len(flat), H, D))
            P.append(sim.pages[layer], sim.codes4[layer], k, v, flat, row4)
            B.kv_append_3bit(up(k), up(v), slots, pages[layer], row4=ints(row4), codes4=codes4[layer], **kw)

    prompt = 130
    rows = ints([0])
    slots = B.kv_pages_grow(pages, tables, lens, refs, rows, ints([prompt]), prompt, codes4=codes4, **kw)
    flat = sim.grow([0], [prompt], prompt).reshape(-1)
    append(slots.view(-1), flat, np.where(np.arange(prompt) == 0, 0, -1))
    B.kv_pages_fork(tables, lens, refs, ints([0] * 4), ints([1, 2, 3, 4]), **kw)
    sim.fork([0] * 4, [1, 2, 3, 4])
    every, ones = np.arange(R), ints(np.ones(R))
    q = up(W.normal_bf16(rng, (R, 1, H * G, D)))
    shared = tables[0, :2].clone()
    step = None
    for s in range(steps):
        slots = B.kv_pages_grow(pages, tables, lens, refs, ints(every), ones, 1, codes4=codes4, **kw)
        flat = sim.grow(every, np.ones(R, int), 1).reshape(-1)
        append(slots.view(-1), flat, np.full(R, -1))
        q.copy_(up(W.normal_bf16(rng, (R, 1, H * G, D))))
        for layer in range(L):
            o, A = P.attention(bits(q), sim.pages[layer], sim.codes4[layer], sim.tables, sim.lens)
            args = (q, pages[layer], tables[:, 2:], lens)
            if graph and layer == 1:
                if step is None:  # captured once, replayed with the tables, lengths and pages of each step
                    side = torch.cuda.Stream()
                    side.wait_stream(torch.cuda.current_stream())
                    with torch.cuda.stream(side):
                        B.kv_attention_3bit_paged(*args, shared=shared, codes4=codes4[layer], status=st)
                    torch.cuda.current_stream().wait_stream(side)
                    step = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(step):
                        caught = B.kv_attention_3bit_paged(*args, shared=shared, codes4=codes4[layer], status=st)
                step.replay()
                got = caught
            else:
                got = B.kv_attention_3bit_paged(*args, shared=shared, codes4=codes4[layer], **kw)
            if stream is not None:
                stream.synchronize()
            err = np.abs(O.bf16_to_f32(bits(got)).astype(np.float64) - o)
            assert (err <= tolerance(o, A)).all(), (s, layer, (err / tolerance(o, A)).max())
    B.kv_pages_free(tables, lens, refs, ints([3, 1]), keep=ints([0, 140]), **kw)
    sim.free([3, 1], [0, 140])
    live = B.kv_pages_compact(pages, tables, lens, refs, codes4=codes4, **kw)
    if stream is not None:
        stream.synchronize()
    assert live.item() == sim.compact()
    assert np.array_equal(refs.cpu().numpy(), sim.refs) and np.array_equal(lens.cpu().numpy(), sim.lens)
    held = sim.held()
    assert np.array_equal(np.where(held < 0, -1, tables.cpu().numpy()), held)
    for layer in range(L):
        o, A = P.attention(bits(q), sim.pages[layer], sim.codes4[layer], sim.tables, sim.lens)
        got = B.kv_attention_3bit_paged(q, pages[layer], tables, lens, codes4=codes4[layer], **kw)
        if stream is not None:
            stream.synchronize()
        assert (np.abs(O.bf16_to_f32(bits(got)).astype(np.float64) - o) <= tolerance(o, A)).all()
    assert st.item() == 0


def test_run_together():
    decode_run(2, 128, 2, 4)


def test_run_captured():
    decode_run(1, 64, 1, 4, graph=True)


def test_run_on_a_stream_of_its_own():
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        decode_run(2, 128, 1, 3, stream=s)
    s.synchronize()


def tile_calls(n):
    rng = np.random.default_rng(12)
    pages, _ = pool(rng, 40, 4, 128, 0)
    p = torch.from_numpy(pages).to(DEV)
    calls = []
    for i in range(n):
        q = up(W.normal_bf16(rng, (24, 1, 8, 128)))
        lens = ints(64 * 8 + rng.integers(1, 100, 24))
        calls.append((q, p, ints(rng.integers(0, 40, (24, 2))), lens, ints(rng.permutation(40)[:8])))
    return calls


def test_run_overlapped():
    """Every kernel may start before the one ahead of it in the stream has ended."""
    B.set_launch_overlap(True)
    try:
        decode_run(2, 128, 2, 4)
        decode_run(1, 64, 1, 3, seed=12)
        calls = tile_calls(3)
        want = [B.kv_attention_3bit_paged(*c[:4], shared=c[4]) for c in calls]
        torch.cuda.synchronize()
        for _ in range(10):
            got = [B.kv_attention_3bit_paged(*c[:4], shared=c[4]) for c in calls]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    finally:
        B.set_launch_overlap(False)


def test_two_graphs_and_a_workspace():
    """Two captured calls that use one workspace, replayed in turn, after the tables, lengths and queries have changed."""
    rng = np.random.default_rng(15)
    D, H = 128, 2
    pages, codes4 = pool(rng, 12, H, D, 1)
    p, c4 = torch.from_numpy(pages).to(DEV), torch.from_numpy(codes4).to(DEV)
    Bn, shared = 20, 3
    sets = []
    for i in range(2):
        q = up(W.normal_bf16(rng, (Bn, 1, H, D)))
        sets.append(dict(q=q, tables=ints(rng.integers(0, 12, (Bn, 2))), lens=ints(64 * shared + rng.integers(1, 120, Bn)),
                         shared=ints(rng.permutation(12)[:shared])))
    work = B.kv_attention_3bit_paged_workspace(sets[0]["q"], p, sets[0]["tables"], sets[0]["shared"])

    def call(s, **kw):
        return B.kv_attention_3bit_paged(s["q"], p, s["tables"], s["lens"], shared=s["shared"], codes4=c4, **kw)

    call(sets[0], workspace=work)
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(s, workspace=work)
        graphs.append((g, out))
    for _ in range(3):
        for s in sets:
            s["q"].copy_(up(W.normal_bf16(rng, (Bn, 1, H, D))))
            s["lens"].copy_(ints(rng.integers(0, 64 * shared + 128, Bn)))
            s["tables"].copy_(ints(rng.integers(0, 12, (Bn, 2))))
        for (g, out), s in zip(graphs, sets):
            g.replay()
            assert torch.equal(out, call(s))


def test_two_calls_at_once():
    """Two streams, a workspace each, the same pool: what one call after the other gives."""
    calls = tile_calls(2)
    want = [B.kv_attention_3bit_paged(*c[:4], shared=c[4]) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [B.kv_attention_3bit_paged(*c[:4], shared=c[4], stream=s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_contiguous_cache_agrees():
    """One sequence without 4-bit tokens: the paged attention and kv_attention_3bit read the same codes."""
    rng = np.random.default_rng(13)
    T, H, D = 300, 4, 128
    k, v, q = W.normal_bf16(rng, (T, H, D)), W.normal_bf16(rng, (T, H, D)), W.normal_bf16(rng, (1, H, D))
    pages, _ = B.kv_page_pool(5, H, D, device=DEV)
    B.kv_append_3bit(up(k), up(v), ints(np.arange(T)), pages)
    got = B.kv_attention_3bit_paged(up(q)[:, None], pages, ints([np.arange(5)]), ints([T]))
    want = B.kv_attention_3bit(up(q), *B.kv_quant_3bit_kv(up(k), up(v), None), None)
    assert (got[:, 0].float() - want.float()).abs().max().item() <= 2.0 ** -7 * want.float().abs().max().item()
