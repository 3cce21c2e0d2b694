"""Drafted trees whose O leaves the range of the attention's fixed reference, or
is not finite.

Large V beside logits that rise along the kept rows: the weights, taken against
the first tile's maximum, and their products with V must not leave the range of
fp32 where the result itself is an ordinary value. Everything is linear in V, and
V is scaled by a power of two, so the library's tolerance (helpers) holds for the
result divided by that power.

NaN and infinity in V rows that every node keeps: softmax(q K^T) V has them in the
same value of every head, whether or not the node is cut into parts. The other
values are within the library's tolerance."""
import numpy as np
import pytest

from helpers import ATOL_MAX, ATOL_MEAN, assert_attn_close, bf16_to_f64, dev, host_bits
from synth import bf16_bits_to_f32, f32_to_bf16_bits
from test_tree import SMALL, Case


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


# one node: a part per tile; 200 nodes of eight tiles: whole ones, cut ones
@pytest.mark.gpu
@pytest.mark.parametrize("ctx,T,H,d", [([1000], 1, 4, 64), ([1000, 990, 980, 970, 960], 40, 12, 64),
                                       ([1000, 990, 980, 970, 960], 40, 70, 128)])
@pytest.mark.parametrize("power", [50, 100, 124])
def test_rising_logits_and_large_values(hsa, ctx, T, H, d, power):
    c = Case(hsa, **dict(SMALL, ctx=ctx, T=T, capacity=1088, m=17, k=1088, H=H, d=d))  # every row is kept
    # logits: N(0, 1), and 55 nats more from cache row 900 on: some 100 weights of 2^79 times the first tile's
    for n in ("Kc", "Kn"):
        x = bf16_bits_to_f32(getattr(c, n)).copy()
        x[..., 0] = 0
        if n == "Kc":
            x[:, 900:, 0] = 55
        setattr(c, n, f32_to_bf16_bits(x))
    x = bf16_bits_to_f32(c.Q).copy()
    x[..., 0] = np.sqrt(d)
    c.Q = f32_to_bf16_bits(x)
    for n in ("Vc", "Vn"):
        setattr(c, n, f32_to_bf16_bits(bf16_bits_to_f32(getattr(c, n)) * np.float32(2.0 ** power)))
    for n in ("Kc", "Kn", "Q", "Vc", "Vn"):
        c.g[n] = dev(getattr(c, n))
    O, idx = c.run()
    O = bf16_to_f64(host_bits(O)) * 2.0 ** -power
    for b in range(c.batch):
        for i in range(0, T, 7):
            rows, ref = c.node(b, i)
            assert np.array_equal(idx[b, i].cpu().numpy(), rows)
            err = np.abs(O[b, i] - ref[0] * 2.0 ** -power)
            assert np.isfinite(O[b, i]).all(), (b, i)
            assert err.max() <= ATOL_MAX and err.mean() <= ATOL_MEAN, (b, i, err.max(), err.mean())


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,T,H,d", [([900], 1, 4, 64), ([950, 800, 700, 650, 600], 40, 4, 64),
                                       ([950, 800, 700, 650, 600], 40, 70, 128)])
def test_nan_and_infinity_in_kept_rows(hsa, ctx, T, H, d):
    c = Case(hsa, **dict(SMALL, ctx=ctx, T=T, capacity=1024, m=16, k=1024, H=H, d=d))  # every cached row is kept
    c.g["Vc"][:, 3, 5] = float("nan")
    c.g["Vc"][:, 130, 7] = float("inf")
    O, idx = c.run()
    assert O[..., 5].isnan().all() and (O[..., 7] == float("inf")).all()
    bits = np.delete(host_bits(O), (5, 7), axis=-1)
    for b in range(c.batch):
        for i in range(0, T, 7):
            rows, ref = c.node(b, i)
            assert np.array_equal(idx[b, i].cpu().numpy(), rows)
            assert_attn_close(bits[b, i][None], np.delete(ref, (5, 7), axis=-1), f"sequence {b} node {i}")
