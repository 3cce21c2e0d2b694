"""NaN and infinity in V rows that a query keeps: softmax(q K^T) V has them in the
same value of every head's output."""
import numpy as np
import pytest

import synth
from helpers import assert_attn_close, dev, host_bits
from test_tree import SMALL, Case

NAN_AT, INF_AT = 5, 7


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


def split(O, what):
    """The poisoned values are as they must be; returns the others."""
    assert O[..., NAN_AT].isnan().all(), what
    assert (O[..., INF_AT] == float("inf")).all(), what
    keep = [c for c in range(O.shape[-1]) if c not in (NAN_AT, INF_AT)]
    return O[..., keep]


@pytest.mark.gpu
@pytest.mark.parametrize("H,d", [(4, 64), (70, 128)])
def test_decode_step(hsa, H, d):
    import torch
    c = Case(hsa, **dict(SMALL, ctx=[900, 700], T=1, capacity=1024, m=16, k=1024, H=H, d=d))
    g = c.g
    g["Vc"][:, 3, NAN_AT] = float("nan")
    g["Vc"][:, 130, INF_AT] = float("inf")
    ws = torch.empty(hsa.hsa_decode_workspace_size(c.p, 2, 1024), dtype=torch.uint8, device="cuda")
    O = torch.empty((2, H, d), dtype=torch.bfloat16, device="cuda")
    hsa.hsa_decode_step(c.p, 2, 1024, g["ctx"], g["kc"], g["Kc"], g["Vc"], g["ksum"], g["q"], g["kn"], g["Q"],
                        g["Kn"], g["Vn"], O, None, ws)
    assert split(O, "decode").isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("H,d", [(4, 64), (70, 128)])
def test_sparse_attn(hsa, H, d):
    import torch
    import oracle
    Lq, Lk, k = 40, 600, 256
    Q, K, V = (synth.normal_bf16(s, 8, t) for s, t in (((Lq, H, d), 1), ((Lk, d), 2), ((Lk, d), 3)))
    idx = np.tile(np.arange(0, 2 * k, 2, dtype=np.int32), (Lq, 1))
    ref = oracle.sparse_attn(Q, K, V, idx)
    Vg = dev(V)
    Vg[4, NAN_AT] = float("nan")
    Vg[300, INF_AT] = float("inf")
    O = hsa.sparse_attn(dev(Q), dev(K), Vg, torch.from_numpy(idx).cuda())
    rest = split(O, "prefill")
    assert_attn_close(host_bits(rest), np.delete(ref, (NAN_AT, INF_AT), axis=-1), "the other values")
