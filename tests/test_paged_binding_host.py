"""Arguments that the binding refuses before it computes with them, without a GPU."""
import pytest
import torch

from tests.test_paged_host import tq  # noqa: F401


def test_a_cache_without_heads(tq):  # noqa: F811
    q, v = tq.tq_codebook_host(128, 4), tq.tq_codebook_mse_host(128, 4)
    y, start = torch.zeros(4, 256, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    kc, vc = q.empty_paged(3, 0, 16, device="cpu"), v.empty_paged(3, 0, 16, device="cpu")
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([4], dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.tq_attend_paged(q, v, y, start, kc, vc, table, lens, 4, 0.1)
