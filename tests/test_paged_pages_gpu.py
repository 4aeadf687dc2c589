"""The page calls of the paged 3-bit cache on the GPU: pools without layers or pages, a
prefix whose pages compaction moves, bad entries alone."""
import numpy as np
import pytest
import torch

import bit_quantised_gemm_b200 as B
from bit_quantised_gemm_b200 import _lib
from oracle import paged_oracle as P
from test_paged_gpu import DEV, Both, ints
import workloads as W

pytestmark = pytest.mark.gpu


def test_a_pool_without_layers():
    """Tables, lengths and references of pages that hold nothing: grown, forked, copied on write, freed, compacted."""
    b = Both(6, 3, 20, L=0)
    b.grow([0, 1], [70, 3])
    b.fork([0], [2])
    b.grow([2, 0, 1], [1, 60, 64])
    b.free([1, 2], [0, 64])
    b.grow([1], [1])
    b.free([1])
    b.compact()
    b.grow([3], [130])


@pytest.mark.parametrize("L,C4", [(2, 1), (0, 0)])
def test_a_pool_without_pages(L, C4):
    b = Both(4, 2, 0, L=L, C4=C4)
    b.compact()
    b.grow([1, 2], [1, 0])  # too few free pages
    b.grow([3], [0])
    b.free([0])
    b.compact()


@pytest.mark.parametrize("kids,D", [(3, 128), (18, 64)])
def test_a_prefix_after_compaction(kids, D):
    """The prefix's pages move; its list, taken again from a row that holds it, names them: the same answer."""
    b = Both(kids + 7, 6, 80, L=1, H=2, D=D, C4=0)
    rng = np.random.default_rng(D)
    k, v = (W.normal_bf16(rng, (80 * 64, 2, D)) for _ in range(2))
    P.append(b.o.pages[0], None, k, v, np.arange(80 * 64))
    b.pages.copy_(torch.from_numpy(b.o.pages))
    others, first = list(range(kids + 1, kids + 7)), list(range(kids + 1))
    b.grow(others + [0], [330] * 6 + [260])  # 36 pages, then the prefix's
    b.fork([0] * kids, first[1:])
    b.grow(first, [1 + i % 50 for i in first])
    q = W.bf16_bits_to_torch(W.normal_bf16(rng, (kids + 1, 1, 4, D))).to(DEV)

    def attention(shared):
        return B.kv_attention_3bit_paged(q, b.pages[0], b.tables[:kids + 1, 4:], b.lens[:kids + 1].contiguous(), shared=shared, status=b.st)

    before = b.tables[0, :4].clone()
    want = attention(before)
    b.free(others)
    b.compact()
    after = b.tables[0, :4].clone()
    assert not torch.equal(before, after)
    assert torch.equal(attention(after), want) and b.st.item() == 0


def test_bad_entries_change_nothing():
    """Calls of bad entries alone: every table, length, count and page stays, what unused entries hold too."""
    b = Both(6, 2, 12)
    b.grow([0, 1], [100, 64])
    b.fork([1], [4])
    kept = [t.clone() for t in (b.wide, b.lens, b.refs, b.pages, b.codes4)]

    def same():
        assert b.st.item() == _lib.STATUS_BAD_INDEX
        b.st.zero_()
        assert all(torch.equal(x, y) for x, y in zip(kept, (b.wide, b.lens, b.refs, b.pages, b.codes4)))

    tables = (b.tables, b.lens, b.refs)
    for row, n in ((6, 1), (-1, 1), (0, 29), (3, 30), (2, -1)):  # no row, too many for a row, for the call, none
        got = B.kv_pages_grow(b.pages, *tables, ints([row]), ints([n]), 29, codes4=b.codes4, status=b.st)
        assert (got == -1).all()
        same()
    for parent, child in ((0, 1), (0, 6), (9, 5), (-1, 5), (5, 5)):  # a child with tokens, no row, its own parent
        B.kv_pages_fork(*tables, ints([parent]), ints([child]), status=b.st)
        same()
    for row, keep in ((7, 0), (-3, 0), (0, -1)):
        B.kv_pages_free(*tables, ints([row]), keep=ints([keep]), status=b.st)
        same()
    for src, dst in ((0, 12), (12, 1), (-1, 3), (3, -1)):
        B.kv_pages_copy(b.pages, ints([src]), ints([dst]), codes4=b.codes4, status=b.st)
        same()
