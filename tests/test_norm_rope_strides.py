"""The token strides that hsa_qk_norm_rope's binding takes from its tensors: rows
of a tree ([batch][T][H][d]), of a fused projection, single tokens; and what it
refuses because no one stride describes it."""
import pytest


def stride(*a):
    from hierarchical_sparse_attention_hisa_b200._lib import _token_stride
    return _token_stride("Q", *a)


H, D = 4, 64


def e(*shape):
    import torch
    return torch.empty(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("make,L,heads,want", [
    (lambda: e(10, H, D), 10, H, H * D),
    (lambda: e(10, H, D), 7, H, H * D),                                              # the first tokens of a larger buffer
    (lambda: e(10, 2 * H, D), 10, H, 2 * H * D),                                     # the first heads
    (lambda: e(3, 5, H, D), 15, H, H * D),                                           # a tree's layout
    (lambda: e(3, 5, 2, H, D), 30, H, H * D),
    (lambda: e(3, 1, H, D), 3, H, H * D), (lambda: e(1, 5, H, D), 5, H, H * D),
    (lambda: e(3, 5, (H + 2) * D)[..., :H * D].unflatten(-1, (H, D)), 15, H, (H + 2) * D),  # of a fused projection
    (lambda: e(15, (H + 2) * D)[:, :H * D].unflatten(1, (H, D)), 15, H, (H + 2) * D),
    (lambda: e(H, D), 1, H, H * D), (lambda: e(1, H, D), 1, H, H * D),
    # one head, or a key
    (lambda: e(10, D), 10, 1, D), (lambda: e(10, 1, D), 10, 1, D), (lambda: e(3, 5, D), 15, 1, D),
    (lambda: e(3, 5, 1, D), 15, 1, D), (lambda: e(10, H, D), 10, 1, H * D), (lambda: e(D), 1, 1, D),
    (lambda: e(3, 5, 6 * D)[..., D:2 * D], 15, 1, 6 * D),
])
def test_stride(make, L, heads, want):
    assert stride(make(), L, heads, D) == want


@pytest.mark.parametrize("make,L,heads", [
    (lambda: e(3, 8, H, D)[:, :5], 15, H),          # rows left out after every fifth
    (lambda: e(5, 3, H, D).transpose(0, 1), 15, H),
    (lambda: e(3, 8, D)[:, :5], 15, 1),
    (lambda: e(10, H, D), 11, H), (lambda: e(2, 5, H, D), 11, H), (lambda: e(10, D), 11, 1), (lambda: e(H, D), 2, H),
    (lambda: e(10, H, 2 * D)[..., ::2], 10, H), (lambda: e(10, H, 2 * D)[..., :D], 10, H), (lambda: e(10, H * D), 10, H),
])
def test_refused(make, L, heads):
    with pytest.raises(ValueError):
        stride(make(), L, heads, D)


def test_the_call_refuses_before_anything_else():
    import hierarchical_sparse_attention_hisa_b200 as hsa
    hsa.build()
    Q, K = e(3, 8, H, D)[:, :5], e(3, 5, D)
    with pytest.raises(ValueError):
        hsa.hsa_qk_norm_rope(15, H, D, Q, None, None, None, 1e-6, None, 0, False, None, 0, e(15, H, D), None, 0)
    with pytest.raises(ValueError):
        hsa.hsa_qk_norm_rope(16, H, D, None, K, None, None, 1e-6, None, 0, False, None, 0, None, e(15, D), 0)


@pytest.mark.gpu
def test_tree_rows():
    """[batch][T][H][d] and [batch][T][d], dense and out of a fused projection, as their flattened rows."""
    import torch
    import hierarchical_sparse_attention_hisa_b200 as hsa
    hsa.build()
    batch, T = 6, 5
    g = torch.Generator(device="cuda").manual_seed(2)
    row = torch.randn((batch, T, (H + 2) * D), generator=g, device="cuda").to(torch.bfloat16)
    inv = (10000.0 ** (-torch.arange(0, D, 2, device="cuda").float() / D)).contiguous()
    pos = torch.arange(batch * T, dtype=torch.int32, device="cuda") * 7
    Q, K = row[..., :H * D].unflatten(-1, (H, D)), row[..., H * D:(H + 1) * D]
    want = hsa.qk_norm_rope(Q.reshape(-1, H, D), K.reshape(-1, D), inv_freq=inv, positions=pos)
    for q, k in ((Q, K), (Q.contiguous(), K.contiguous())):
        Qo, Ko = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        hsa.hsa_qk_norm_rope(batch * T, H, D, q, k, None, None, 1e-6, inv, D, False, pos, 0, Qo, Ko)
        assert torch.equal(Qo, want[0]) and torch.equal(Ko, want[1])
