"""A lost hand-off in the drafted tree's attention alone: below 128 MB of kept
blocks the token scores run on CUDA cores and wait for nothing, so the attention
is the only kernel of the step that loses one. Its bounded waits give up, the call
returns, hsa_device_status reports it, and a clean rerun gives the earlier results.
Runs, as its neighbours do, after the check that no wait gave up during the other
GPU tests."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["rows_200", "many_heads"])
def test_lost_arrival_in_the_attention(name):
    import torch
    import hierarchical_sparse_attention_hisa_b200 as hsa
    from hierarchical_sparse_attention_hisa_b200._lib import HSA_ERR_TIMEOUT, HSA_OK
    from test_tree import STEP_CASES, Case
    hsa.build()
    c = Case(hsa, **STEP_CASES[name])
    assert c.batch * c.T * c.m * c.B * c.d_idx * 2 <= 128 << 20
    O, idx = c.run()
    torch.cuda.synchronize()
    assert hsa.hsa_device_status(reset=True) == HSA_OK
    try:
        hsa.hsa_debug_inject_lost_arrival(True)
        _, idx1 = c.run()
        status = hsa.hsa_device_status(reset=True)
    finally:
        hsa.hsa_debug_inject_lost_arrival(False)
        hsa.hsa_device_status(reset=True)
    assert status == HSA_ERR_TIMEOUT
    assert torch.equal(idx1, idx)  # the selection lost nothing
    O2, idx2 = c.run()
    torch.cuda.synchronize()
    assert hsa.hsa_device_status(reset=False) == HSA_OK
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(idx, idx2)
