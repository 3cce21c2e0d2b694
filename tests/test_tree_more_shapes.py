"""Drafted trees, further shapes: long lists that are selected from and not kept
whole, one node over 64 tiles (every tile a part of its own), the work lists'
scores at each width of the trees for d_idx = 64, and real-valued indexer
inputs, where a selection may differ from exact arithmetic's only between
scores closer than the rounding.

Rounding of the scores. A product of two bf16 values is exact in fp32. A sum of
n such products, in whatever order and on whichever unit, makes n additions;
each is off by at most 2^-23 of the magnitudes summed so far (rounding 2^-24,
cutting off, as the matrix unit may, 2^-23), and the unit may cut each product
to the largest one's exponent before it adds (2^-23 once more). So a token's
score is off by at most d_idx * 2^-22 * sum |q k|. A block's score has B
additions per value of the sum and 3 d_idx of the products with its three
parts, or, in the tail, d_idx per token and B of the tokens' scores: at most
(B + 3 d_idx) * 2^-22 * sum |q| sum |k|."""
import numpy as np
import pytest

import oracle
from helpers import assert_attn_close, bf16_to_f64, dev, host_bits
from synth import normal_bf16
from test_tree import Case


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


LONG = dict(B=128, m=64, d_idx=64, capacity=9216)
SHAPES = {
    "k_3000": dict(LONG, k=3000, H=2, d=64, ctx=[9000, 8190, 8600], T=4),
    "k_4097": dict(LONG, k=4097, H=5, d=128, ctx=[9000, 8190], T=5),
    "one_node_k_8000": dict(LONG, k=8000, H=64, d=128, ctx=[9000], T=1),
    "one_node_64_tiles": dict(LONG, k=8192, H=100, d=64, ctx=[9000], T=1),
    "lists_64_t16": dict(B=64, m=200, k=500, d_idx=64, H=4, d=64, ctx=[16000 - 37 * b for b in range(6)], T=16,
                         capacity=16384),
    "lists_64_t24": dict(B=64, m=200, k=500, d_idx=64, H=4, d=64, ctx=[16000 - 41 * b for b in range(4)], T=24,
                         capacity=16384, kind="chain"),
    "lists_64_t32": dict(B=128, m=100, k=700, d_idx=64, H=4, d=64, ctx=[16000, 15999, 15000], T=32, capacity=16384,
                         kind="binary"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", SHAPES)
def test_step_against_oracle(hsa, name):
    import torch
    c = Case(hsa, **SHAPES[name])
    O, idx = c.run()
    c.check(O, idx, {(b, i) for b in range(c.batch) for i in range(b % 3, c.T, 5)} if c.batch * c.T > 20 else None)
    c.check_caches()
    O2, idx2 = c.run()
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(idx, idx2)


def real_case(hsa, **kw):
    """A case whose indexer queries and keys are normal values instead of small integers."""
    c = Case(hsa, **kw)
    c.q, c.kn, c.kc = (normal_bf16(getattr(c, n).shape, 99, t) for n, t in (("q", 1), ("kn", 2), ("kc", 3)))
    for n in ("q", "kn", "kc"):
        c.g[n] = dev(getattr(c, n))
    for b in range(c.batch):
        if c.ctx[b] >= c.B:
            hsa.hsa_block_sums(c.p, int(c.ctx[b]), c.g["kc"][b], c.g["ksum"][b])
    return c


def nodes_of(c, O, idx, step):
    """(query, keys along the path, kept positions) of every step-th node, its attention checked."""
    idx, O = idx.cpu().numpy(), host_bits(O)
    for b in range(c.batch):
        at = int(c.ctx[b])
        for i in range(b % step, c.T, step):
            path = [int(j) for j in c.paths[b, i] if j >= 0]
            seq = lambda cache, new: np.concatenate([cache[b, :at], new[b, path]])  # noqa: E731
            rows = idx[b, i]
            n = int((rows >= 0).sum())
            assert (rows[n:] == -1).all() and (np.diff(rows[:n]) > 0).all()
            back = {at + j: at + s for s, j in enumerate(path)}
            pos = np.array([back[int(r)] if r >= at else int(r) for r in rows[:n]])  # (a drafted row off the path: KeyError)
            ref = oracle.sparse_attn(c.Q[b, i][None], seq(c.Kc, c.Kn), seq(c.Vc, c.Vn), pos[None].astype(np.int32))
            assert_attn_close(O[b, i][None], ref, f"sequence {b} node {i}")
            yield bf16_to_f64(c.q[b, i]), bf16_to_f64(seq(c.kc, c.kn)), pos


def assert_best(score, slack, kept):
    """No score left out is above a kept one by more than both can be off."""
    kept = np.asarray(kept, bool)
    if kept.all() or not kept.any():
        return
    assert (score - slack)[~kept].max() <= (score + slack)[kept].min()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [
    # without lists, and (from 128 MB of kept blocks on) with them at each width; every block is kept
    dict(B=64, m=20, k=200, d_idx=64, ctx=[1200, 700, 1000], T=7, capacity=1280, kind="chain"),
    dict(B=100, m=20, k=333, d_idx=128, ctx=[1900, 1777], T=33, capacity=2000),
    dict(B=64, m=200, k=1000, d_idx=64, ctx=[12000 - 50 * b for b in range(6)], T=16, capacity=12800),
    dict(B=64, m=200, k=1000, d_idx=64, ctx=[12000 - 50 * b for b in range(4)], T=32, capacity=12800),
    dict(B=64, m=200, k=1000, d_idx=128, ctx=[12000, 11000], T=50, capacity=12800, kind="chain"),
    dict(B=128, m=100, k=2048, d_idx=128, ctx=[12000 - 50 * b for b in range(4)], T=16, capacity=12800),
])
def test_real_valued_tokens(hsa, shape):
    c = real_case(hsa, H=4, d=64, **shape)
    O, idx = c.run()
    for q, keys, pos in nodes_of(c, O, idx, 7):
        n = len(keys)
        assert len(pos) == min(c.k, n)
        kept = np.zeros(n, bool)
        kept[pos] = True
        assert_best(keys @ q, c.d_idx * 2.0 ** -22 * (np.abs(keys) @ np.abs(q)), kept)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [
    # every token of the kept blocks is kept, so the rows say which blocks were
    dict(B=16, m=6, k=96, d_idx=64, ctx=[450, 300], T=33, capacity=512, kind="chain"),
    dict(B=64, m=8, k=512, d_idx=128, ctx=[20000, 15000, 9000], T=16, capacity=20480),
    dict(B=32, m=40, k=1280, d_idx=64, ctx=[30000], T=64, capacity=32768, kind="binary"),
    dict(B=128, m=16, k=2048, d_idx=128, ctx=[32000, 31000], T=20, capacity=32768, kind="chain"),
])
def test_real_valued_blocks(hsa, shape):
    c = real_case(hsa, H=4, d=64, **shape)
    O, idx = c.run()
    for q, keys, pos in nodes_of(c, O, idx, 7):
        n, B = len(keys), c.B
        nb = (n - 1) // B + 1
        assert nb > c.m
        blocks = np.unique(pos // B)
        assert len(blocks) == c.m and blocks[0] == 0 and blocks[-1] == nb - 1
        assert len(pos) == (c.m - 1) * B + (n - 1) % B + 1  # whole blocks
        s = (keys @ q)[: (nb - 1) * B].reshape(nb - 1, B).sum(1)
        slack = (B + 3 * c.d_idx) * 2.0 ** -22 * (np.abs(keys) @ np.abs(q))[: (nb - 1) * B].reshape(nb - 1, B).sum(1)
        assert_best(s[1:], slack[1:], np.isin(np.arange(1, nb - 1), blocks))
