"""The paged 3-bit cache without a GPU: the oracle's layout and page calls
against hand-worked cases, and the calls' refusals."""
import numpy as np
import pytest
import torch

import bit_quantised_gemm_b200 as B
from bit_quantised_gemm_b200 import _lib
from oracle import bitlinear_oracle as O
from oracle import paged_oracle as P
import workloads as W

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced on a host-side error


# ------------------------------------------------------------- the oracle
@pytest.mark.parametrize("D", [64, 128, 256])
def test_block_bytes(D):
    assert B.kv_page_block_bytes(D) == P.block_bytes(D) == 64 * (3 * D // 4 + 8)


def test_block_bytes_refuses():
    assert B.lib().kv_page_block_bytes(96) == 0
    with pytest.raises(ValueError):
        B.kv_page_block_bytes(32)


def test_oracle_places_a_token():
    """One token at place 6 of page 1: K row at 6 * 24, V bytes 4 apart from
    64 * 24 + 1 * 96 + 2, scales at words 6 and 70."""
    D = 64
    k = np.zeros((1, 1, D), np.float32)
    k[0, 0, :3] = [3.0, -3.0, 1.0]  # absmax 3: scale 1, codes 3, -3, 1 -> 7, 1, 5, then 4s
    v = -k
    pages = np.full((2, 1, P.block_bytes(D)), 0xA5, np.uint8)
    P.append(pages, None, O.f32_to_bf16(k), O.f32_to_bf16(v), [70])
    blk = pages[1, 0]
    word = 7 | (1 << 3) | (5 << 6) | sum(4 << (3 * i) for i in range(3, 8))
    assert [int(x) for x in blk[144:147]] == [word & 255, (word >> 8) & 255, word >> 16]
    word = 1 | (7 << 3) | (3 << 6) | sum(4 << (3 * i) for i in range(3, 8))
    assert [int(x) for x in blk[1634:1634 + 12:4]] == [word & 255, (word >> 8) & 255, word >> 16]
    s = blk[2 * 64 * 24:].view(np.float32)
    assert s[6] == 1.0 and s[70] == 1.0
    assert (pages[0] == 0xA5).all() and (blk == 0xA5).sum() >= blk.size - 24 - 24 - 8


def test_oracle_reads_what_it_wrote():
    rng = np.random.default_rng(3)
    D, H = 128, 2
    k, v = W.normal_bf16(rng, (5, H, D)), W.normal_bf16(rng, (5, H, D))
    pages, codes4 = np.zeros((2, H, P.block_bytes(D)), np.uint8), np.zeros((2, H, 3, D), np.uint8)
    row4 = np.array([-1, 2, -1, 0, -1])
    slots = [3, 7, 64, 127, 66]
    P.append(pages, codes4, k, v, slots, row4)
    for x, w in ((k, 0), (v, 1)):
        want = O.kv_dequant(*O.kv_quant_3bit(x, (1, 3)), (1, 3), D)
        for i, s in enumerate(slots):
            assert np.array_equal(P.read(pages, codes4, s // 64, s % 64, D)[w], want[i])


def test_oracle_page_calls():
    t = P.Tables(4, 4, 8, np.arange(8, dtype=np.uint8).reshape(1, 8, 1, 1).copy())
    assert t.grow([0], [70], 70)[0, [0, 63, 64, 69]].tolist() == [0, 63, 64, 69]
    t.fork([0, 0], [1, 2])
    assert t.refs[:2].tolist() == [3, 3]
    s = t.grow([1, 0, 2], [1, 1, 60], 60)
    # row 1 copies page 1 to page 2, row 0 copies it to page 3, row 2 is alone on it and needs a page more
    assert s[0, 0] == 2 * 64 + 6 and s[1, 0] == 3 * 64 + 6 and s[2, 0] == 64 + 6 and s[2, 58] == 4 * 64
    assert t.refs.tolist() == [3, 1, 1, 1, 1, 0, 0, 0]
    assert t.pages[0, :4, 0, 0].tolist() == [0, 1, 1, 1]
    assert t.grow([3], [64 * 4], 256) is None
    t.free([1], [64])
    t.free([0])
    assert t.refs.tolist() == [2, 1, 0, 0, 1, 0, 0, 0] and t.lens.tolist() == [0, 64, 130, 0]
    assert t.compact() == 3
    assert t.refs.tolist() == [2, 1, 1, 0, 0, 0, 0, 0] and t.tables[2, :3].tolist() == [0, 1, 2]


# ------------------------------------------------------ refusals of the ABI
def _append(**kw):
    a = dict(k=FAKE, ldk=256, v=FAKE, ldv=256, n=4, H=2, D=128, slots=FAKE, row4=None, pages=FAKE, n_pages=8,
             codes4=None, C4=0)
    a.update(kw)
    return B.lib().kv_append_3bit(*a.values(), None, None)


def test_append_refusals():
    assert _append(n=0) == _lib.OK
    assert _append(D=96) == _lib.ERR_UNSUPPORTED
    assert _append(H=0) == _lib.ERR_INVALID_ARG
    assert _append(n=-1) == _lib.ERR_INVALID_ARG
    assert _append(ldk=255) == _lib.ERR_INVALID_ARG
    assert _append(ldv=260) == _lib.ERR_INVALID_ARG
    assert _append(k=None) == _lib.ERR_INVALID_ARG
    assert _append(slots=None) == _lib.ERR_INVALID_ARG
    assert _append(pages=None) == _lib.ERR_INVALID_ARG
    assert _append(k=FAKE + 2) == _lib.ERR_ALIGNMENT
    assert _append(pages=FAKE + 8) == _lib.ERR_ALIGNMENT
    assert _append(C4=2) == _lib.ERR_INVALID_ARG        # no codes4
    assert _append(C4=65, codes4=FAKE) == _lib.ERR_INVALID_ARG
    assert _append(n_pages=1 << 25) == _lib.ERR_INVALID_ARG


def _attention(**kw):
    a = dict(q=FAKE, ldq=512, B=2, Sq=1, Hq=4, H=2, D=128, pages=FAKE, n_pages=8, codes4=None, C4=0, shared=None,
             n_shared=0, tables=FAKE, W=4, ldt=4, lens=FAKE, out=FAKE, work=FAKE, work_bytes=1 << 30)
    a.update(kw)
    return B.lib().kv_attention_3bit_paged(*a.values(), None, None)


def test_attention_refusals():
    assert _attention(B=0) == _lib.OK
    assert _attention(D=96) == _lib.ERR_UNSUPPORTED
    assert _attention(Hq=3) == _lib.ERR_INVALID_ARG
    assert _attention(Sq=0) == _lib.ERR_INVALID_ARG
    assert _attention(Sq=129) == _lib.ERR_UNSUPPORTED
    assert _attention(B=65536) == _lib.ERR_UNSUPPORTED
    assert _attention(ldq=504) == _lib.ERR_INVALID_ARG
    assert _attention(ldt=3) == _lib.ERR_INVALID_ARG
    assert _attention(n_shared=1) == _lib.ERR_INVALID_ARG   # no list
    assert _attention(tables=None) == _lib.ERR_INVALID_ARG
    assert _attention(lens=None) == _lib.ERR_INVALID_ARG
    assert _attention(W=1 << 25, ldt=1 << 25) == _lib.ERR_UNSUPPORTED
    assert _attention(q=FAKE + 8) == _lib.ERR_ALIGNMENT
    assert _attention(work=FAKE + 4) == _lib.ERR_ALIGNMENT
    need = B.lib().kv_attention_3bit_paged_workspace(2, 1, 4, 2, 128, 0, 4)
    assert need >= 0
    if need:
        assert _attention(work_bytes=need - 1) == _lib.ERR_INVALID_ARG
        assert _attention(work=None) == _lib.ERR_INVALID_ARG
    assert B.lib().kv_attention_3bit_paged_workspace(2, 1, 3, 2, 128, 0, 4) == _lib.ERR_INVALID_ARG


def test_page_call_refusals():
    L = B.lib()
    copy = lambda pb=1024, c4=None, pb4=0, n=2, src=FAKE, pages=FAKE: L.kv_pages_copy(  # noqa: E731
        pages, pb, c4, pb4, 2, 8, src, FAKE, n, None, None)
    assert copy(n=0) == _lib.OK
    assert copy(pb=1000) == _lib.ERR_INVALID_ARG
    assert copy(pb4=64) == _lib.ERR_INVALID_ARG
    assert copy(n=-1) == _lib.ERR_INVALID_ARG
    assert copy(src=None) == _lib.ERR_INVALID_ARG
    assert copy(pages=FAKE + 8) == _lib.ERR_ALIGNMENT
    fork = lambda R=4, W_=4, ldt=4, n=2, parents=FAKE, refs=FAKE: L.kv_pages_fork(  # noqa: E731
        FAKE, R, W_, ldt, FAKE, refs, 8, parents, FAKE, n, None, None)
    assert fork(n=0) == _lib.OK
    assert fork(ldt=3) == _lib.ERR_INVALID_ARG
    assert fork(R=-1) == _lib.ERR_INVALID_ARG
    assert fork(n=65536) == _lib.ERR_UNSUPPORTED
    assert fork(parents=None) == _lib.ERR_INVALID_ARG
    assert fork(refs=None) == _lib.ERR_INVALID_ARG
    free = lambda n=2, rows=FAKE: L.kv_pages_free(FAKE, 4, 4, 4, FAKE, FAKE, 8, rows, None, n, None, None)  # noqa: E731
    assert free(n=0) == _lib.OK
    assert free(n=-2) == _lib.ERR_INVALID_ARG
    assert free(rows=None) == _lib.ERR_INVALID_ARG
    grow = lambda n=2, m=1, rows=FAKE, slots=FAKE, work=FAKE: L.kv_pages_grow(  # noqa: E731
        FAKE, 1024, None, 0, 1, 8, FAKE, 4, 4, 4, FAKE, FAKE, rows, FAKE, n, m, slots, work, None, None)
    assert grow(n=0) == _lib.OK
    assert grow(n=1025) == _lib.ERR_UNSUPPORTED
    assert grow(m=-1) == _lib.ERR_INVALID_ARG
    assert grow(rows=None) == _lib.ERR_INVALID_ARG
    assert grow(slots=None) == _lib.ERR_INVALID_ARG
    assert grow(work=None) == _lib.ERR_INVALID_ARG
    compact = lambda n_live=FAKE, work=FAKE, pb=1024: L.kv_pages_compact(  # noqa: E731
        FAKE, pb, None, 0, 1, 8, FAKE, 4, 4, 4, FAKE, FAKE, n_live, work, None, None)
    assert compact(n_live=None) == _lib.ERR_INVALID_ARG
    assert compact(work=None) == _lib.ERR_INVALID_ARG
    assert compact(pb=8) == _lib.ERR_INVALID_ARG


# -------------------------------------------------- refusals of the binding
def test_binding_refusals():
    """CPU tensors: a well-formed call gets as far as the CUDA-tensor check."""
    H, D, n = 2, 128, 5
    i32 = dict(dtype=torch.int32)
    pages, codes4 = B.kv_page_pool(6, H, D, rows4=2, device="cpu")
    assert pages.shape == (6, H, B.kv_page_block_bytes(D)) and codes4.shape == (6, H, 2, D)
    k = torch.zeros(n, H, D, dtype=torch.bfloat16)
    slots = torch.zeros(n, **i32)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_append_3bit(k, k, slots, pages, codes4=codes4)
    with pytest.raises(ValueError, match="k: dtype"):
        B.kv_append_3bit(k.float(), k, slots, pages)
    with pytest.raises(ValueError, match="k: shape"):
        B.kv_append_3bit(k[:, :1], k, slots, pages)
    with pytest.raises(ValueError, match="k: shape"):
        B.kv_append_3bit(torch.zeros(n, D, H, dtype=torch.bfloat16).transpose(1, 2), k, slots, pages)
    with pytest.raises(ValueError, match="v: 4 tokens"):
        B.kv_append_3bit(k, k[:4], slots, pages)
    with pytest.raises(ValueError, match="slots: 5 values"):
        B.kv_append_3bit(k[:4], k[:4], slots, pages)
    with pytest.raises(ValueError, match="slots: dtype"):
        B.kv_append_3bit(k, k, slots.long(), pages)
    with pytest.raises(ValueError, match="row4: 4 values"):
        B.kv_append_3bit(k, k, slots, pages, row4=slots[:4], codes4=codes4)
    with pytest.raises(ValueError, match="codes4: shape"):
        B.kv_append_3bit(k, k, slots, pages, codes4=codes4[:5])
    with pytest.raises(ValueError, match="pages: blocks"):
        B.kv_append_3bit(k, k, slots, pages[..., :-16].contiguous())
    with pytest.raises(ValueError, match="pages: must be"):
        B.kv_append_3bit(k, k, slots, pages[None])

    tables, lens, refs = torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.zeros(6, **i32)
    q = torch.zeros(3, 1, 4, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_attention_3bit_paged(q, pages, tables, lens, codes4=codes4)
    with pytest.raises(ValueError, match="CUDA"):  # slices of a fused projection's output
        B.kv_attention_3bit_paged(torch.zeros(3, 1, 8, D, dtype=torch.bfloat16)[:, :, :4], pages, tables, lens)
    with pytest.raises(ValueError, match="q: head dimension"):
        B.kv_attention_3bit_paged(q[..., :64], pages, tables, lens)
    with pytest.raises(ValueError, match="q: strides"):
        B.kv_attention_3bit_paged(torch.zeros(3, 1, D, 4, dtype=torch.bfloat16).transpose(2, 3), pages, tables, lens)
    with pytest.raises(ValueError, match="tables: 2 rows"):
        B.kv_attention_3bit_paged(q, pages, tables[:2], lens[:2])
    with pytest.raises(ValueError, match="lens: 2 values"):
        B.kv_attention_3bit_paged(q, pages, tables, lens[:2])
    with pytest.raises(ValueError, match="shared: dtype"):
        B.kv_attention_3bit_paged(q, pages, tables, lens, shared=lens.long())
    with pytest.raises(ValueError, match="out: shape"):
        B.kv_attention_3bit_paged(q, pages, tables, lens, out=q[:2])
    with pytest.raises(ValueError, match="must be a"):
        B.kv_attention_3bit_paged_workspace(q[0], pages, tables)

    with pytest.raises(ValueError, match="CUDA"):
        B.kv_pages_copy(pages[None], lens, lens, codes4=codes4[None])
    with pytest.raises(ValueError, match="dst: 2 values"):
        B.kv_pages_copy(pages, lens, lens[:2])
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_pages_fork(tables, lens, refs, lens, lens)
    with pytest.raises(ValueError, match="tables: must be"):
        B.kv_pages_fork(tables[:, ::2], lens, refs, lens, lens)
    with pytest.raises(ValueError, match="children: 2 values"):
        B.kv_pages_fork(tables, lens, refs, lens, lens[:2])
    with pytest.raises(ValueError, match="refs: 3 values"):
        B.kv_pages_grow(pages, tables, lens, lens, lens, lens, 1)
    with pytest.raises(ValueError, match="n_new: 2 values"):
        B.kv_pages_grow(pages, tables, lens, refs, lens, lens[:2], 1)
    with pytest.raises(ValueError, match="max_new"):
        B.kv_pages_grow(pages, tables, lens, refs, lens, lens, -1)
    with pytest.raises(ValueError, match="keep: 2 values"):
        B.kv_pages_free(tables, lens, refs, lens, keep=lens[:2])
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_pages_compact(pages, tables, lens, refs, codes4=codes4)
