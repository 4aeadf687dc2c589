"""Pools, sequences and queries for the paged attention's tests."""
from types import SimpleNamespace

import numpy as np

from oracle import bitlinear_oracle as O
from oracle import paged_oracle as P
import workloads as W


def write(rng, k, v, n_pages, C4=0, plain=()):
    """Pages of the tokens k, v (fp32 [64 n_pages x H x D]) in order, C4 of each page, none of the
    places `plain` in it, at 4 bits."""
    H, D = k.shape[1:]
    pages = np.zeros((n_pages, H, P.block_bytes(D)), np.uint8)
    codes4 = np.zeros((n_pages, H, C4, D), np.uint8) if C4 else None
    row4 = np.full(64 * n_pages, -1)
    free = np.setdiff1d(np.arange(64), plain)
    for p in range(n_pages):
        for j, o in enumerate(rng.permutation(free)[:C4]):
            row4[64 * p + o] = j
    P.append(pages, codes4, O.f32_to_bf16(k), O.f32_to_bf16(v), np.arange(64 * n_pages), row4)
    return pages, codes4


def normal(rng, n_pages, H, D):
    return rng.standard_normal((2, 64 * n_pages, H, D), np.float32)


def pool(rng, n_pages, H, D, C4=0):
    return write(rng, *normal(rng, n_pages, H, D), n_pages, C4)


def graded_pool(rng, n_pages, H, D, C4=0, k_top=3.0, v_top=8.0):
    """Later pages hold larger keys and, in an order of their own, larger values: the largest score so far and the
    largest weight so far move from page to page, together and apart."""
    x = normal(rng, n_pages, H, D)
    x[0] *= np.repeat(np.linspace(0.25, k_top, n_pages), 64)[:, None, None].astype(np.float32)
    x[1] *= np.repeat(2.0 ** rng.uniform(-v_top, v_top, n_pages), 64)[:, None, None].astype(np.float32)
    return write(rng, *x, n_pages, C4)


def case(pages, codes4, q, tables, lens, shared, steps):
    return SimpleNamespace(pages=pages, codes4=codes4, q=q, tables=tables, lens=lens, shared=shared, steps=steps)


def many_sequences(D, G, C4, B=250, H=8, Sq=1, seed=0):
    """Short sequences of up to 6 pages, some empty: several of them, and parts of them, to a warp."""
    rng = np.random.default_rng(1000 * seed + D + G)
    pages, codes4 = pool(rng, 40, H, D, C4)
    lens = rng.integers(1, 64 * 6 + 1, B)
    lens[rng.integers(0, B, B // 10)] = 0
    lens[rng.integers(0, B, B // 10)] = 64 * rng.integers(1, 7)
    q = W.normal_bf16(rng, (B, Sq, H * G, D))
    return case(pages, codes4, q, rng.integers(0, 40, (B, 6)), lens, [], 8 * 6 + 8)


def long_sequences(D, G, B=24, H=8, graded=False, seed=0):
    """Sequences of up to 60 pages. Graded: from small to large keys in even sequences, the other way in odd ones."""
    rng = np.random.default_rng(2000 + 1000 * seed + D + G)
    pages, codes4 = (graded_pool if graded else pool)(rng, 40, H, D, 1)
    lens = rng.integers(64 * 40, 64 * 60 + 1, B)
    tables = rng.integers(0, 40, (B, 60))
    if graded:
        tables.sort(1)
        tables[1::2] = tables[1::2, ::-1]
    q = W.normal_bf16(rng, (B, 1, H * G, D))
    return case(pages, codes4, q, tables, lens, [], 8 * 60 + 60)


def long_prefix(D, rows, n=300, H=1, own=0, graded=False, C4=1, seed=0):
    """`rows` sequences behind n shared pages of 40 distinct ones; some end inside the prefix."""
    rng = np.random.default_rng(3000 + 1000 * seed + D + rows + n)
    pages, codes4 = (graded_pool if graded else pool)(rng, 40, H, D, C4)
    shared = rng.integers(0, 40, n)
    if graded:
        shared.sort()
    lens = 64 * n + rng.integers(0, 64 * own + 1, rows)
    lens[::5] = rng.integers(1, 64 * n, len(lens[::5]))
    lens[rows // 2] = 0
    q = W.normal_bf16(rng, (rows, 1, H, D))
    return case(pages, codes4, q, rng.integers(0, 40, (rows, max(own, 1)))[:, :own], lens, shared, 8 * 40 + 160)
