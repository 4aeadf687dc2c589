"""The 64-bit attention that the paged kernels are held against, on the CPU: against
the oracle's token by token, and that its bound sees a page that is left out."""
import numpy as np
import pytest

import paged_cases as C
import paged_reference as R
from oracle import paged_oracle as P
import workloads as W


@pytest.mark.parametrize("D,C4", [(64, 0), (128, 2), (256, 1)])
def test_against_the_oracle(D, C4):
    rng = np.random.default_rng(D)
    H, G, Sq = 2, 2, 3
    pages, codes4 = C.pool(rng, 5, H, D, C4)
    kv = R.dequant(pages, codes4)
    for o in (0, 13, 63):
        for w, x in enumerate(P.read(pages, codes4, 3, o, D)):
            assert np.array_equal(kv[w][3, :, o], x)
    q = W.normal_bf16(rng, (4, Sq, H * G, D))
    tables, lens = rng.integers(0, 5, (4, 3)), np.array([64 * 3, 0, 64 + 2, 2])
    for shared in ([], [2]):
        o, (A, _, L) = R.attention(q, kv, tables, lens, shared)
        want, want_A = P.attention(q, pages, codes4, tables, lens, shared)
        assert np.allclose(o, want, rtol=1e-12, atol=1e-13) and np.allclose(A, want_A, rtol=1e-12, atol=1e-13)
        assert (A.max(-1) <= L[..., 0] * (8 if C4 else 4)).all()


def moved(case, skip):
    """Rows of a case that a page left out at place `skip` moves beyond twice the bound."""
    kv = R.dequant(case.pages, case.codes4)
    args = (case.q, kv, case.tables, case.lens, case.shared)
    o, E = R.attention(*args)
    lost = R.attention(*args, skip=skip)[0]
    return (np.abs(lost - o) > 2 * R.bound(o, E, case.steps)).any(-1)


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2)])
def test_the_bound_sees_a_page(D, G):
    case = C.many_sequences(D, G, 0, B=30, H=2)
    full = case.lens >= 64 * 4
    assert full.any() and moved(case, 2)[full].mean() > 0.95
    case = C.long_sequences(D, G, B=3, H=2)
    assert moved(case, 21).mean() > 0.6
    case = C.long_prefix(D, 40)
    sees = case.lens >= 64 * 31
    assert moved(case, 30)[sees].mean() > 0.5
