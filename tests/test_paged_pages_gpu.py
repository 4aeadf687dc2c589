"""The page calls of the paged 3-bit cache on the GPU: pools without layers or pages."""
from test_paged_gpu import Both

import pytest

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
