"""More refusals of the paged-cache calls' binding, on CPU tensors."""
import pytest
import torch

import bit_quantised_gemm_b200 as B


@pytest.mark.parametrize("status", [torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64),
                                    torch.zeros(0, dtype=torch.int32)])
def test_status_words_of_another_type_or_size(status):
    """A kernel writes 4 bytes of it."""
    i32 = dict(dtype=torch.int32)
    pages, _ = B.kv_page_pool(6, 2, 128, device="cpu")
    tables, lens, refs = torch.zeros(3, 4, **i32), torch.zeros(3, **i32), torch.zeros(6, **i32)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    calls = (lambda s: B.kv_append_3bit(k, k, lens, pages, status=s), lambda s: B.kv_pages_copy(pages, lens, lens, status=s),
             lambda s: B.kv_pages_fork(tables, lens, refs, lens, lens, status=s),
             lambda s: B.kv_pages_free(tables, lens, refs, lens, status=s),
             lambda s: B.kv_pages_grow(pages, tables, lens, refs, lens, lens, 1, status=s),
             lambda s: B.kv_pages_compact(pages, tables, lens, refs, status=s),
             lambda s: B.kv_attention_3bit_paged(k[:, None], pages, tables, lens, status=s))
    for call in calls:
        with pytest.raises(ValueError, match="status"):
            call(status)
        with pytest.raises(ValueError, match="CUDA|status: on cpu"):
            call(torch.zeros(1, **i32))
