"""A decode batch of 300 sequences whose candidate rows (m * B = 21 keys) do not
all start on 16 bytes: such rows must not go through the selection that loads
them 16 bytes at a time."""
import numpy as np
import pytest

import oracle
import synth
from helpers import assert_attn_close, dev, host_bits


@pytest.mark.gpu
def test_decode_many_odd_rows():
    import torch
    import hierarchical_sparse_attention_hisa_b200 as hsa
    hsa.build()
    batch, B, m, k, di, H, d, cap, seed = 300, 7, 3, 11, 64, 2, 64, 98, 12
    p = hsa.params(B=B, m=m, k=k, d_idx=di, H=H, d=d)
    kc = synth.int_bf16((batch, cap, di), seed, 2)
    Kc, Vc = synth.normal_bf16((batch, cap, d), seed, 4), synth.normal_bf16((batch, cap, d), seed, 5)
    q, kn = synth.int_bf16((batch, di), seed, 30), synth.int_bf16((batch, di), seed, 31)
    Q = synth.normal_bf16((batch, H, d), seed, 33)
    Kn, Vn = synth.normal_bf16((batch, d), seed, 34), synth.normal_bf16((batch, d), seed, 35)
    lens = (np.arange(batch) * 7) % 97
    g_kc = dev(kc)
    ks = torch.zeros((batch, cap // B, di), device="cuda")
    for b in range(batch):
        if lens[b] >= B:
            hsa.hsa_block_sums(p, int(lens[b]), g_kc[b], ks[b])
    ctx = torch.from_numpy(lens.astype(np.int32)).cuda()
    ws = torch.empty(hsa.hsa_decode_workspace_size(p, batch, cap), dtype=torch.uint8, device="cuda")
    O = torch.empty((batch, H, d), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((batch, k), dtype=torch.int32, device="cuda")
    hsa.hsa_decode_step(p, batch, cap, ctx, g_kc, dev(Kc), dev(Vc), ks, dev(q), dev(kn), dev(Q), dev(Kn), dev(Vn), O, idx,
                        ws)
    got_idx, got_O = idx.cpu().numpy(), host_bits(O)
    for b in range(batch):
        t = int(lens[b])
        seq = lambda cache, new: np.concatenate([cache[b, :t], new[b][None]])  # noqa: E731
        want = oracle.index(q[b][None], seq(kc, kn), B, m, k)
        assert np.array_equal(got_idx[b], want[0]), b
        assert_attn_close(got_O[b][None], oracle.sparse_attn(Q[b][None], seq(Kc, Kn), seq(Vc, Vn), want), f"sequence {b}")
