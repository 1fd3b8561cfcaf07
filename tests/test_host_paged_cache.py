"""SfaPagedCache's refusals on the host."""
import pytest
import torch

import indexer_selected_sparse_block_gb300 as sfa


@pytest.mark.parametrize("rows", [dict(V=torch.zeros(4, 1, 64)), dict(X=torch.zeros(4, 16))])
def test_rows_for_a_cache_that_holds_none(rows):
    c = sfa.SfaPagedCache(n_seq=1, n_pages=2, page_size=4, max_pages=2, n_tok_cap=4, h_kv=1, dkq=64, dv=64,
                          device="cpu")
    with pytest.raises(ValueError, match="holds none"):
        c.step(torch.zeros(1, dtype=torch.int32), torch.zeros(4, 1, 64), **rows)
