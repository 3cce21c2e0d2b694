"""The module's forms on a stream of the caller's while the current stream is
behind or ahead: their own allocations and fills are ordered with their kernels,
and nothing of theirs is handed out again while those run."""
import pytest

import synth
from helpers import dev

SLEEP = 200_000_000  # clock cycles, about a tenth of a second


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


def poison(torch, *tensors):
    """Memory of these sizes from the current stream's pool, overwritten."""
    keep = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda") for t in tensors]
    for t in keep:
        t.fill_(0xFF)
    return keep


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_norm_rope_while_the_current_stream_is_busy(hsa, handle):
    import torch
    L, H, d = 500, 6, 64
    Q, K = dev(synth.normal_bf16((L, H, d), 4, 1)), dev(synth.normal_bf16((L, d), 4, 2))
    inv = (10000.0 ** (-torch.arange(0, d, 2, device="cuda").float() / d)).contiguous()
    pos = torch.arange(L, dtype=torch.int32, device="cuda") * 3
    pos[::7] = -1
    want = hsa.qk_norm_rope(Q, K, inv_freq=inv, positions=pos)
    assert (want[0][::7] == 0).all() and (want[0][1] != 0).any()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)  # fills on the current stream come after this
    got = hsa.qk_norm_rope(Q, K, inv_freq=inv, positions=pos, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_index_and_attention_on_a_stream_that_is_behind(hsa, handle):
    import torch
    w = synth.WORKLOADS["tiny_prefill_2k"]
    x = synth.prefill_inputs(w)
    q, k, Q, K, V = (dev(x[n]) for n in ("q_idx", "k_idx", "Q", "K", "V"))
    idx = hsa.index(q, k, w.B, w.m, w.k)
    O = hsa.sparse_attn(Q, K, V, idx)
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    ws = hsa.hsa_index_workspace_size(hsa.params(B=w.B, m=w.m, k=w.k, d_idx=q.shape[1]), len(q), len(k))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)  # the calls' kernels run after the fills below
    got_idx = hsa.index(q, k, w.B, w.m, w.k, stream=s)
    keep = poison(torch, torch.empty(ws, dtype=torch.uint8, device="meta"), idx)
    got_O = hsa.sparse_attn(Q, K, V, got_idx, stream=s)
    keep += poison(torch, O)
    torch.cuda.synchronize()
    assert torch.equal(got_idx, idx) and torch.equal(got_O.view(torch.int16), O.view(torch.int16))
    assert all((t == 0xFF).all() for t in keep)
