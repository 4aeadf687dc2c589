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


def check_case(c):
    check(c.pages, c.codes4, c.q, c.tables, c.lens, c.shared, c.steps)


# how rows of a head come together: (sequences, query heads a cache head, queries, pages in front)
OWN = [(24, 1, 1, 0), (24, 2, 1, 0), (24, 3, 1, 0), (24, 4, 1, 0), (24, 5, 1, 0), (24, 8, 1, 0), (8, 4, 3, 0)]
FEW = [(2, 1, 1, 1), (4, 1, 1, 1), (3, 2, 1, 1), (16, 1, 1, 1), (32, 1, 1, 1)]
TILES = [(17, 1, 1, 1), (33, 1, 1, 1), (40, 4, 1, 1), (20, 4, 4, 1)]


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


# ------------------------------------------------------ range of the weights
def lopsided(rng, n_pages, H, D, at, k_at, v_exp):
    """Pages in which the tokens `at` have a key whose only large value is k_at, and values 2^v_exp in size."""
    x = C.normal(rng, n_pages, H, D)
    x[0, :, :, 0] = 0
    for t in at:
        x[0, t] = 0
        x[0, t, :, 0] = k_at
        x[1, t] *= np.float32(2.0 ** v_exp)
    return C.write(rng, x[0], x[1], n_pages, 2, plain=[t % 64 for t in at])


def lopsided_sets(D, form, at, k_at, v_exp):
    """Every row's query is 8 in dimension 0, which the other keys leave at zero: the tokens `at` have scores of
    8 k_at / sqrt(D). 4 pages in order, in front or not."""
    Bn, G, Sq, front = form
    rng = np.random.default_rng(D + Bn + G + Sq + abs(v_exp))
    H = 2
    pages, codes4 = lopsided(rng, 4, H, D, at, k_at, v_exp)
    x = rng.standard_normal((Bn, Sq, H * G, D), np.float32)
    x[..., 0] = 8
    q = O.f32_to_bf16(x)
    lens = rng.integers(Sq, 256, Bn)
    lens[0], lens[1] = 256, 150
    if front:
        check(pages, codes4, q, np.zeros((Bn, 0), int), lens, [0, 1, 2, 3])
        check(pages, codes4, q, np.tile([2, 3], (Bn, 1)), lens, [0, 1])
    else:
        check(pages, codes4, q, np.tile([0, 1, 2, 3], (Bn, 1)), lens)


RANGES = [([5], -4096.0, 28), ([5], -4096.0, 40), ([70, 140], -4096.0, 60), ([0, 63, 128], -65536.0, 100),
          ([0], 30.0, -60), ([70], 60.0, -60), ([0, 100], 12.0, 20), ([3, 190], 200.0, -30)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", OWN + FEW)
@pytest.mark.parametrize("at,k_at,v_exp", RANGES)
def test_range_of_weights(D, form, at, k_at, v_exp):
    """Tokens without weight and with large values, or that take nearly all and have values of nearly nothing."""
    lopsided_sets(D, form, at, k_at, v_exp)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", TILES)
@pytest.mark.parametrize("at,k_at,v_exp", RANGES)
def test_tile_range_of_weights(D, form, at, k_at, v_exp):
    lopsided_sets(D, form, at, k_at, v_exp)


def spread_values(D, form):
    """Values between 2^-13 and 2^13 in size, sharp and flat scores."""
    Bn, G, Sq, front = form
    rng = np.random.default_rng(D + Bn + G + Sq)
    H = 2
    x = C.normal(rng, 4, H, D)
    x[1] *= np.exp(3 * rng.standard_normal((256, H, 1), np.float32))
    pages, codes4 = C.write(rng, x[0], x[1], 4, 1)
    lens = rng.integers(Sq, 257, Bn)
    for gain in (0, 1, 8):
        q = O.f32_to_bf16(gain * rng.standard_normal((Bn, Sq, H * G, D), np.float32))
        check(pages, codes4, q, np.tile([0, 1, 2, 3][2 * front:], (Bn, 1)), lens, [0, 1][:2 * front])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", OWN + FEW)
def test_spread_values(D, form):
    spread_values(D, form)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", TILES)
def test_tile_spread_values(D, form):
    spread_values(D, form)


def unwritten_pages(D, Bn, n):
    """Pages of a new pool (scales of zero) counted among the tokens: scores of zero, values of zero."""
    rng = np.random.default_rng(D + Bn)
    H = 2
    pages, codes4 = C.pool(rng, 6, H, D, 1)
    pages[0], codes4[0] = 0, 0
    shared = np.zeros(n, int)
    shared[10::25] = 1 + rng.integers(0, 5, len(shared[10::25]))
    q = W.normal_bf16(rng, (Bn, 1, H, D))
    lens = rng.integers(64 * 40, 64 * n, Bn)
    kv = R.dequant(pages, codes4)
    o, E = R.attention(q, kv, np.zeros((Bn, 0), int), lens, shared)
    got = run(pages, codes4, q, np.zeros((Bn, 0), int), lens, shared)
    # a piece has n / 18 pages at most where there are tiles, n / 100 in a walk
    err, most = np.abs(got - o), R.bound(o, E, 8 * n // 18 + 160)
    worst = (int((err > most).sum()), err.size, float((err / most).max()))
    assert worst[0] == 0, worst


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Bn", [2, 4, 16])
def test_unwritten_pages(D, Bn):
    unwritten_pages(D, Bn, 400)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Bn", [17, 40, 200])
def test_tile_unwritten_pages(D, Bn):
    unwritten_pages(D, Bn, 900)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", OWN + FEW + TILES)
@pytest.mark.parametrize("e", [96, -12])
def test_keys_and_queries_of_far_sizes(D, form, e):
    """Keys of 2^e and queries of 2^-e: scores of ordinary size."""
    Bn, G, Sq, front = form
    rng = np.random.default_rng(D + Bn + G + Sq)
    H = 2
    x = C.normal(rng, 4, H, D)
    pages, codes4 = C.write(rng, x[0] * np.float32(2.0 ** e), x[1], 4, 1)
    q = O.f32_to_bf16(np.float32(2.0 ** -e) * rng.standard_normal((Bn, Sq, H * G, D), np.float32))
    lens = rng.integers(Sq, 257, Bn)
    check(pages, codes4, q, np.tile([0, 1, 2, 3][2 * front:], (Bn, 1)), lens, [0, 1][:2 * front])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", OWN + FEW + TILES)
@pytest.mark.parametrize("e", [4, 16, 28, 40])
def test_scores_far_out(D, form, e):
    """Scores up to 2^(e + 17): the token of the largest one, twice the next, takes all, and the row is its value to
    half a step and 2^-16, with nothing lost of the score's own weight."""
    Bn, G, Sq, front = form
    rng = np.random.default_rng(D + Bn + G + Sq + e)
    H = 2
    x = C.normal(rng, 4, H, D)
    x[0] = 0
    x[0, :, :, 0] = 2.0 ** 13 * rng.uniform(1, 2, (256, H))
    x[0, 100, :, 0] = 2.0 ** 15
    pages, codes4 = C.write(rng, x[0], x[1], 4)
    q = np.zeros((Bn, Sq, H * G, D), np.float32)
    q[..., 0] = 2.0 ** e
    lens = rng.integers(120, 257, Bn)
    want = R.dequant(pages)[1][1, :, 36].repeat(G, 0)  # [Hq, D]
    most = np.abs(want) * 2.0 ** -16 + 2.0 ** (np.frexp(np.abs(want) + 2.0 ** -60)[1] - 9.0)
    sets = [(np.tile([0, 1, 2, 3], (Bn, 1)), [])]
    if front:
        sets = [(np.zeros((Bn, 0), int), [0, 1, 2, 3]), (np.tile([2, 3], (Bn, 1)), [0, 1]), (np.tile([1, 2, 3], (Bn, 1)), [0])]
    for tables, shared in sets:
        got = run(pages, codes4, O.f32_to_bf16(q), tables, lens, shared)
        assert (np.abs(got - want) <= most).all()


# ------------------------------------------------- several pages to a warp
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Sq,C4", [(1, 1, 0), (1, 1, 1), (2, 1, 5), (3, 1, 1), (4, 1, 5), (5, 1, 0), (8, 1, 5), (2, 3, 1)])
def test_many_sequences(D, G, Sq, C4):
    """Shares of several pages that begin and end inside sequences and hold several of them; 4-bit rows that
    travel with their pages and rows that do not."""
    check_case(C.many_sequences(D, G, C4, Sq=Sq))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("graded", [False, True])
def test_long_sequences(D, G, graded):
    """24 x 8 heads of 40 to 60 pages: about 4 pages a warp (8 with D = 256), all of one segment; largest score
    and largest weight moving with every page."""
    check_case(C.long_sequences(D, G, graded=graded))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [2, 4, 7, 16, 32])
@pytest.mark.parametrize("graded", [False, True])
def test_long_prefix_walks(D, rows, graded):
    """A prefix of 500 pages x 8 heads for few rows: 3 to 7 pages a warp."""
    check_case(C.long_prefix(D, rows, n=500, H=8, graded=graded))
    check_case(C.long_prefix(D, rows, n=300, H=16, own=3, graded=graded, C4=5))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [17, 40, 128, 200, 300])
@pytest.mark.parametrize("graded", [False, True])
def test_long_prefix_tiles(D, rows, graded):
    """Tiles over 3 to 8 pages each, a single tile, a pair, and a pair with a single one; with D = 256 one by one."""
    check_case(C.long_prefix(D, rows, n=300, graded=graded))
    check_case(C.long_prefix(D, rows, n=301, own=2, graded=graded, C4=0 if graded else 5))


@pytest.mark.parametrize("G", [4, 8])
@pytest.mark.parametrize("D,shared", [(64, 0), (128, 0), (256, 0), (128, 2)])
def test_many_rows_of_4_bits_in_small_groups(D, G, shared):
    """Five tokens of a page at 4 bits, more than travel with it, for 4 and 8 rows a head."""
    rng = np.random.default_rng(D + G + shared)
    H, Bn = 2, 2 if shared else 6
    pages, codes4 = C.pool(rng, 8, H, D, 5)
    lens = 64 * shared + rng.integers(1, 180, Bn)
    q = W.normal_bf16(rng, (Bn, 1, H * G, D))
    check(pages, codes4, q, rng.integers(0, 8, (Bn, 3)), lens, rng.permutation(8)[:shared])
