"""The paged attention on the GPU against 64 bits, to half a step of its output: its weights'
bits and range, and what a warp or a CTA carries from page to page."""
import numpy as np
import pytest
import torch

import bit_quantised_gemm_b200 as B
import paged_cases as C
import paged_reference as R
from oracle import bitlinear_oracle as O
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def up(bits):
    return W.bf16_bits_to_torch(bits).to(DEV)


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def fresh():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def run(pages, codes4, q, tables, lens, shared=(), status=0, **kw):
    st = fresh()
    got = B.kv_attention_3bit_paged(up(q), torch.from_numpy(pages).to(DEV), ints(tables), ints(lens),
                                    shared=ints(shared), codes4=None if codes4 is None else torch.from_numpy(codes4).to(DEV),
                                    status=st, **kw)
    assert st.item() == status
    return O.bf16_to_f32(got.view(torch.int16).cpu().numpy().view(np.uint16)).astype(np.float64)


def check(pages, codes4, q, tables, lens, shared=(), steps=64):
    got = run(pages, codes4, q, tables, lens, shared)
    o, E = R.attention(q, R.dequant(pages, codes4), tables, lens, shared)
    err, most = np.abs(got - o), R.bound(o, E, steps) + 1e-37
    worst = (int((err > most).sum()), err.size, float((err / most).max()))
    assert worst[0] == 0, worst


# how rows of a head come together: (sequences, query heads a cache head, queries, pages in front)
OWN = [(24, 1, 1, 0), (24, 2, 1, 0), (24, 3, 1, 0), (24, 4, 1, 0), (24, 5, 1, 0), (24, 8, 1, 0), (8, 4, 3, 0)]
FEW = [(2, 1, 1, 1), (4, 1, 1, 1), (3, 2, 1, 1), (16, 1, 1, 1)]
TILES = [(17, 1, 1, 1), (40, 4, 1, 1), (20, 4, 4, 1)]


# ------------------------------------------------------- bits of the weights
def few_tokens(D, form):
    """A few tokens a row: a weight's rounding is not averaged away."""
    Bn, G, Sq, front = form
    rng = np.random.default_rng(D + Bn + G + Sq)
    H = 4
    pages, codes4 = C.pool(rng, 6, H, D, 2)
    q = W.normal_bf16(rng, (Bn, Sq, H * G, D))
    lens = rng.integers(1, 10, Bn)
    if front:
        check(pages, codes4, q, np.zeros((Bn, 0), int), lens, [3])
        lens[::3] += 64
        check(pages, codes4, q, rng.integers(0, 6, (Bn, 1)), lens, [3])
    else:
        check(pages, codes4, q, rng.integers(0, 6, (Bn, 2)), lens)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", OWN + FEW)
def test_weights_to_half_a_step(D, form):
    few_tokens(D, form)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", TILES)
def test_tile_weights_to_half_a_step(D, form):
    few_tokens(D, form)
