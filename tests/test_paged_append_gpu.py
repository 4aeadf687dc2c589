"""Appending several sequences' tokens in one call: the stored bytes are the oracle's."""
import numpy as np
import pytest
import torch

import bit_quantised_gemm_b200 as B
from oracle import paged_oracle as P
from test_paged_gpu import DEV, fresh, ints, up
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H", [(64, 3), (128, 2), (256, 2)])
@pytest.mark.parametrize("lengths,padding", [([61, 70, 3, 129], 0), ([33, 64, 31], 5), ([1, 1, 130, 1], 3), ([8, 16, 4, 64, 7], 1)])
def test_packed_prompts(D, H, lengths, padding):
    """Prompts of odd lengths one behind the other, each from another place of a page on, with padding before each:
    runs that begin anywhere in the call and anywhere in a page; the other bytes stay."""
    rng = np.random.default_rng(D + sum(lengths) + padding)
    slots, row4, page = [], [], 0
    for i, n in enumerate(lengths):
        first = 5 * i
        at = np.arange(n) + first
        slots += [-1] * padding + list((page + at // 64) * 64 + at % 64)
        row4 += [-1] * padding + [0] + [-1] * (n - 1)  # each prompt's first token at 4 bits
        page += (first + n + 63) // 64
    n = len(slots)
    k, v = W.normal_bf16(rng, (n, H, D)), W.normal_bf16(rng, (n, H, D))
    for four in (np.full(n, -1), np.array(row4)):
        want, want4 = np.full((page, H, P.block_bytes(D)), 0x5A, np.uint8), np.full((page, H, 1, D), 0x5A, np.uint8)
        pages, codes4 = torch.from_numpy(want.copy()).to(DEV), torch.from_numpy(want4.copy()).to(DEV)
        P.append(want, want4, k, v, np.array(slots), four)
        st = fresh()
        B.kv_append_3bit(up(k), up(v), ints(slots), pages, row4=ints(four), codes4=codes4, status=st)
        assert np.array_equal(pages.cpu().numpy(), want) and np.array_equal(codes4.cpu().numpy(), want4)
        assert st.item() == 0
