"""The paged cache's attention in 64 bits, a pool's pages taken apart once, and
how far 32-bit arithmetic and one rounding to bf16 may lie from it."""
import numpy as np

from oracle import bitlinear_oracle as O
from oracle import paged_oracle as P


def dequant(pages, codes4=None):
    """K, V [n_pages x H x 64 x D] in fp64 of all of a layer's pages, and V's scales [n_pages x H x 64 x 1]."""
    n, H, block = pages.shape
    D = (block // 64 - 8) * 4 // 3
    rb = 3 * D // 8
    scale = pages[..., 128 * rb:].copy().view(np.float32).astype(np.float64).reshape(n, H, 2, 64)
    k = pages[..., :64 * rb].reshape(n, H, 64, rb)
    v = pages[..., 64 * rb:128 * rb].reshape(n, H, 16, rb, 4).swapaxes(-1, -2).reshape(n, H, 64, rb)
    four = np.signbit(scale[:, :, 0])
    out = []
    for w, rows in enumerate((k, v)):
        bits = np.unpackbits(rows, axis=-1, bitorder="little").reshape(n, H, 64, D, 3)
        c = (bits @ np.array([1, 2, 4])).astype(np.float64) - 4
        if codes4 is not None:
            j = np.where(four, k[..., 0], 0)
            b = np.take_along_axis(codes4, j[..., None].astype(np.int64), 2)[..., w * D // 2:(w + 1) * D // 2]
            c4 = np.stack([b & 15, b >> 4], -1).reshape(n, H, 64, D).astype(np.float64) - 8
            c = np.where(four[..., None], c4, c)
        out.append(c * np.abs(scale[:, :, w])[..., None])
    return *out, scale[:, :, 1, :, None]


def attention(q_bits, kv, tables, lens, shared=(), skip=None):
    """(o, E) of q [B x Sq x Hq x D]: the attention, and what bound() takes its allowances from. `skip`: a
    place (in pages) of the sequences that is passed over."""
    q = O.bf16_to_f32(q_bits).astype(np.float64)
    B, Sq, Hq, D = q.shape
    H = kv[0].shape[1]
    o, A = np.zeros(q.shape), np.zeros(q.shape)
    T, L = np.zeros(q.shape[:3] + (1,)), np.zeros(q.shape[:3] + (1,))
    known = {}

    def taken(u):  # the distinct pages u: K, |K|, V, |V| [H x 64 len(u) x D], V's scales [H x len(u) x 64]
        if u.tobytes() not in known:
            k, v, sc = (x[u].swapaxes(0, 1).reshape(H, -1, x.shape[-1]) for x in kv)
            known.clear()
            known[u.tobytes()] = k, np.abs(k), v, np.abs(v), sc.reshape(H, len(u), 64)
        return known[u.tobytes()]

    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        ids = np.concatenate([np.asarray(shared, np.int64), np.asarray(tables[b], np.int64)])[:P.pages_of(n)]
        u, place = np.unique(ids, return_inverse=True)
        k, k_abs, v, v_abs, sc = taken(u)
        qb = q[b].reshape(Sq, H, Hq // H, D).transpose(1, 0, 2, 3).reshape(H, -1, D)  # rows (i, g)
        at = np.arange(64 * len(ids)).reshape(-1, 64)
        see = at < (n - Sq + 1 + np.arange(Sq).repeat(Hq // H))[:, None, None]  # [rows, pages, 64]
        if skip is not None:
            see[:, skip:skip + 1] = False
        every = lambda x, y: (x @ y.swapaxes(1, 2) / np.sqrt(D)).reshape(H, -1, len(u), 64)[:, :, place]  # noqa: E731
        s, t = every(qb, k), every(np.abs(qb), k_abs)
        top = np.where(see, s, -np.inf).max((2, 3), keepdims=True)
        p = np.where(see, np.exp(np.where(see, s, -np.inf) - np.where(np.isfinite(top), top, 0)), 0)
        l = p.sum((2, 3), keepdims=True)
        p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
        largest = (p * sc[:, None, place]).max((2, 3))[..., None]
        order = np.argsort(place, kind="stable")  # what each distinct page's tokens weigh in all its places
        w = np.add.reduceat(p[:, :, order], np.searchsorted(place[order], np.arange(len(u))), axis=2).reshape(H, p.shape[1], -1)
        for x, y in ((o, w @ v), (A, w @ v_abs), (T, np.where(p >= 2.0 ** -100, t, 0).max((2, 3))[..., None]), (L, n * largest)):
            x[b] = y.reshape(H, Sq, Hq // H, -1).transpose(1, 0, 2, 3).reshape(Sq, Hq, -1)
    return o, (A, T, L)


def bound(o, E, steps=64):
    """How far the kernels' bf16 outputs may be from o. E = (A, T, L): sum_t p_t |v_t|; the largest
    sum_d |q_d k_td| / sqrt(D) of the tokens with p_t of 2^-100 or more (the others' scores may be off by
    much); the number of tokens times the largest weight p_t x (V scale).
      * bf16's rounding: half a step, of the binade that the unrounded value may lie in;
      * scores: sums of D products in 32 bits. At most 2^-19 of the sum of their sizes (16 steps of an
        MMA, each off by 2^-23; the queries' fields of the integer form lose less), and a score off
        by e moves its weight by e and the output by at most e (A + |o|);
      * weights, exponentials, factors: 2^-16 (A + |o|) as for the contiguous cache;
      * weights have no exponents of their own: they are whole numbers of which the largest is 2^29 or more, or two
        fp16 numbers where the largest is 2^7 or more and 2^-24 is lost. So 2^-30 of the largest
        weight or less is lost of each token's, times a code of up to 4: 2^-28 L;
      * `steps` additions one behind the other, each off by 2^-23 of what may be in the sum."""
    A, T, L = E
    s = (2.0 ** -16 + 2.0 ** -19 * T + steps * 2.0 ** -23) * (A + np.abs(o)) + 2.0 ** -28 * L
    half = 2.0 ** (np.frexp(np.maximum(np.abs(o) + s, 2.0 ** -126))[1] - 9.0)
    return half + s
