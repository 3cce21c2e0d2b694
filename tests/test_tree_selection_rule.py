"""Drafted trees on both sides of the choice between a tree's own top-k and the
prefill's: up to and above 296 rows, 1024 and 8192 candidates, block sizes that
the prefill's row kernel takes and that it does not."""
import pytest

from test_tree import Case


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [37, 38])  # 296 and 304 rows
@pytest.mark.parametrize("B,m,k", [(64, 16, 200), (64, 17, 200), (64, 128, 700), (100, 20, 333), (128, 65, 700),
                                   (256, 64, 1500), (64, 300, 900)])
def test_rows_and_candidates(hsa, batch, B, m, k):
    import torch
    top = (m + 6) * B
    c = Case(hsa, ctx=[top - 11 * b for b in range(batch)], T=8, capacity=top + 2 * B, B=B, m=m, k=k, d_idx=64, H=2,
             d=64, n_nodes=[8 - b % 3 for b in range(batch)])
    O, idx = c.run()
    c.check(O, idx, {(b, (3 * b) % 8) for b in range(0, batch, 4)} | {(batch - 1, 5)})
    O2, idx2 = c.run()
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(idx, idx2)
