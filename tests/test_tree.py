"""Drafted trees: hsa_tree_plan, hsa_tree_step and hsa_tree_commit against the
CPU oracle evaluated along every node's own path, against the decode step, and
their refusals.

Kept rows must match the oracle bit for bit (integer indexer inputs), attention
within the library's tolerance (helpers.assert_attn_close).
"""
import ctypes

import numpy as np
import pytest

import oracle
import synth
from helpers import assert_attn_close, dev, host_bits

TMAX = 64


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


# ------------------------------------------------------------------ trees

def make_parents(kind, batch, T, seed):
    rng = np.random.default_rng(seed)
    i = np.arange(T)
    if kind == "chain":
        p = np.tile(i - 1, (batch, 1))
    elif kind == "star":
        p = np.full((batch, T), -1)
    elif kind == "binary":
        p = np.tile((i - 1) // 2, (batch, 1))
        p[:, 0] = -1
    else:
        p = np.array([[int(rng.integers(max(-1, j - 5), j)) for j in range(T)] for _ in range(batch)])
    return p.reshape(batch, T).astype(np.int32)


def plan_reference(parents, n_nodes, ctx, capacity):
    batch, T = parents.shape
    pos = np.full((batch, T), -1, np.int32)
    paths = np.full((batch, T, T), -1, np.int32)
    for b in range(batch):
        n = T if n_nodes is None else min(max(int(n_nodes[b]), 0), T)
        if ctx[b] < 0 or ctx[b] + n > capacity:
            continue
        for i in range(n):
            chain, j = [], i
            while j >= 0:
                chain.append(j)
                q = int(parents[b, j])
                if q < -1 or q >= j:
                    chain = None
                    break
                j = q
            if chain:
                pos[b, i] = ctx[b] + len(chain) - 1
                paths[b, i, :len(chain)] = chain[::-1]
    return pos, paths


def gpu_plan(hsa, parents, n_nodes, ctx, capacity):
    import torch
    batch, T = parents.shape
    pos = torch.full((batch, T), 99, dtype=torch.int32, device="cuda")
    paths = torch.full((batch, T, T), 99, dtype=torch.int32, device="cuda")
    as_t = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    hsa.hsa_tree_plan(batch, T, capacity, as_t(ctx), as_t(n_nodes), as_t(parents), pos, paths)
    return pos, paths


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chain", "star", "binary", "random"])
@pytest.mark.parametrize("T", [1, 2, 7, 33, 64])
def test_plan(hsa, kind, T):
    ctx = [0, 5, 1000 - T, 1000 - T + 1, -1, 1000, 500, 500, 999]
    n = [T, T, T, T, T, 0, -3, T + 9, 1]
    parents = make_parents(kind, len(ctx), T, T)
    for nn in (n, None):
        pos, paths = gpu_plan(hsa, parents, nn, ctx, 1000)
        want = plan_reference(parents, nn, ctx, 1000)
        assert np.array_equal(pos.cpu().numpy(), want[0])
        assert np.array_equal(paths.cpu().numpy(), want[1])


@pytest.mark.gpu
def test_plan_of_something_that_is_no_tree(hsa):
    # a node of itself, of a later node, below -1, and everything hanging off those
    parents = np.array([[-1, 0, 2, 2, 5, 0, -2, 6, -1, 1 << 30, 8, -(1 << 31)]], np.int32)
    pos, paths = gpu_plan(hsa, parents, None, [10], 100)
    want = plan_reference(parents, None, [10], 100)
    assert want[0][0].tolist() == [10, 11, -1, -1, -1, 11, -1, -1, 10, -1, 11, -1]
    assert np.array_equal(pos.cpu().numpy(), want[0]) and np.array_equal(paths.cpu().numpy(), want[1])


# ------------------------------------------------------------------ one step

class Case:
    """Caches, drafted rows and a plan, on the host (bits) and on the GPU."""

    def __init__(self, hsa, ctx, T, capacity, B, m, k, d_idx, H, d, kind="random", n_nodes=None, seed=1, scale=0.0,
                 zero_q=False):
        import torch
        self.hsa, self.T, self.capacity, self.B, self.m, self.k = hsa, T, capacity, B, m, k
        self.batch = batch = len(ctx)
        self.ctx, self.H, self.d, self.d_idx = np.array(ctx, np.int32), H, d, d_idx
        self.scale = scale
        self.p = hsa.params(B=B, m=m, k=k, d_idx=d_idx, H=H, d=d, scale=scale)
        self.kc = synth.int_bf16((batch, capacity, d_idx), seed, 2)
        self.Kc = synth.normal_bf16((batch, capacity, d), seed, 4)
        self.Vc = synth.normal_bf16((batch, capacity, d), seed, 5)
        self.q = synth.int_bf16((batch, T, d_idx), seed, 30)
        if zero_q:
            self.q[:] = 0
        self.kn = synth.int_bf16((batch, T, d_idx), seed, 31)
        self.Q = synth.normal_bf16((batch, T, H, d), seed, 33)
        self.Kn = synth.normal_bf16((batch, T, d), seed, 34)
        self.Vn = synth.normal_bf16((batch, T, d), seed, 35)
        self.parents = make_parents(kind, batch, T, seed)
        self.n_nodes = n_nodes
        self.pos, self.paths = plan_reference(self.parents, n_nodes, self.ctx, capacity)
        self.g = {n: dev(getattr(self, n)) for n in ("kc", "Kc", "Vc", "q", "kn", "Q", "Kn", "Vn")}
        # block sums of the whole cached blocks; the others hold what must never be read
        self.g["ksum"] = torch.full((batch, capacity // B, d_idx), float("nan"), device="cuda")
        for b in range(batch):
            if self.ctx[b] >= B:
                hsa.hsa_block_sums(self.p, int(self.ctx[b]), self.g["kc"][b], self.g["ksum"][b])
        self.g["ctx"] = torch.from_numpy(self.ctx).cuda()
        self.g["pos"], self.g["paths"] = gpu_plan(hsa, self.parents, n_nodes, self.ctx, capacity)

    def run(self, stream=None, ws=None, O=None, idx=None):
        import torch
        g, hsa = self.g, self.hsa
        if ws is None:  # stale workspace contents must not matter
            ws = torch.full((hsa.hsa_tree_workspace_size(self.p, self.batch, self.T, self.capacity),), 0xA5,
                            dtype=torch.uint8, device="cuda")
        if O is None:
            O = torch.full((self.batch, self.T, self.H, self.d), 5.0, dtype=torch.bfloat16, device="cuda")
        if idx is None:
            idx = torch.full((self.batch, self.T, self.k), 77, dtype=torch.int32, device="cuda")
        hsa.hsa_tree_step(self.p, self.batch, self.T, self.capacity, g["ctx"], g["pos"], g["paths"], g["kc"], g["Kc"],
                          g["Vc"], g["ksum"], g["q"], g["kn"], g["Q"], g["Kn"], g["Vn"], O, idx, ws, stream)
        return O, idx

    def node(self, b, i):
        """The oracle's kept cache rows and fp64 output of node i."""
        c = int(self.ctx[b])
        path = [int(j) for j in self.paths[b, i] if j >= 0]
        seq = lambda cache, new: np.concatenate([cache[b, :c], new[b, path]])  # noqa: E731
        kept = oracle.index(self.q[b, i][None], seq(self.kc, self.kn), self.B, self.m, self.k)
        ref = oracle.sparse_attn(self.Q[b, i][None], seq(self.Kc, self.Kn), seq(self.Vc, self.Vn), kept, self.scale or None)
        rows = kept[0].copy()
        late = rows >= c
        rows[late] = c + np.array(path, np.int32)[rows[late] - c]
        return rows, ref

    def check(self, O, idx, nodes=None):
        idx, O = idx.cpu().numpy(), host_bits(O)
        for b in range(self.batch):
            for i in range(self.T):
                if self.pos[b, i] < 0:
                    assert (idx[b, i] == -1).all() and (O[b, i] == 0).all(), (b, i)
                elif nodes is None or (b, i) in nodes:
                    rows, ref = self.node(b, i)
                    assert np.array_equal(idx[b, i], rows), (b, i)
                    assert_attn_close(O[b, i][None], ref, f"sequence {b} node {i}")

    def check_caches(self):
        """Drafted rows behind the cached ones, everything else as it was."""
        for name, cache, new in (("kc", self.kc, self.kn), ("Kc", self.Kc, self.Kn), ("Vc", self.Vc, self.Vn)):
            want = cache.copy()
            for b, i in np.argwhere(self.pos >= 0):
                want[b, self.ctx[b] + i] = new[b, i]
            assert np.array_equal(host_bits(self.g[name]), want), name
        assert np.array_equal(self.g["ctx"].cpu().numpy(), self.ctx)


SMALL = dict(B=64, m=8, k=256, d_idx=64, H=4, d=64)
STEP_CASES = {
    # ragged lengths from none to the last row, a sequence without room, one without nodes
    "ragged": dict(SMALL, ctx=[1, 63, 500, 1000, 0, 1017, 1018, 640], T=7, capacity=1024,
                   n_nodes=[7, 7, 6, 7, 7, 7, 7, 0]),
    "one_block": dict(B=64, m=2, k=20, d_idx=64, H=4, d=64, ctx=[0, 5, 61, 62, 64], T=3, capacity=64),
    "one_node": dict(SMALL, ctx=[5, 600, 1023], T=1, capacity=1024),
    # 64 drafted tokens in a row complete several small blocks, which then compete as candidates
    "chain_small_blocks": dict(B=16, m=6, k=40, d_idx=128, H=5, d=128, ctx=[200, 7, 0, 447], T=64, capacity=512,
                               kind="chain"),
    "block_of_one": dict(B=1, m=20, k=9, d_idx=64, H=3, d=64, ctx=[100, 30], T=40, capacity=200, kind="binary"),
    "odd_block": dict(B=7, m=3, k=11, d_idx=64, H=2, d=128, ctx=[100, 55, 0, 6, 77], T=64, capacity=203, kind="random"),
    "block_100": dict(B=100, m=5, k=130, d_idx=128, H=16, d=64, ctx=[1950, 999], T=33, capacity=2100),
    # blocks of more than 128 rows: two and eight pieces per block
    "block_200": dict(B=200, m=4, k=300, d_idx=128, H=8, d=128, ctx=[1990, 1799], T=20, capacity=2200),
    "block_1024": dict(B=1024, m=3, k=500, d_idx=64, H=1, d=64, ctx=[5000, 6140], T=12, capacity=7168, kind="chain"),
    "block_256": dict(B=256, m=6, k=512, d_idx=128, H=64, d=128, ctx=[4000, 2815], T=17, capacity=4096),
    "two_blocks": dict(B=32, m=2, k=20, d_idx=64, H=4, d=64, ctx=[500, 31, 32], T=10, capacity=544),
    # every candidate kept: no token scores
    "keeps_all": dict(B=32, m=4, k=128, d_idx=64, H=4, d=64, ctx=[700, 100], T=10, capacity=736),
    "one_kept": dict(B=64, m=4, k=1, d_idx=64, H=4, d=64, ctx=[700, 100], T=6, capacity=768, kind="star"),
    "odd_k": dict(B=64, m=8, k=131, d_idx=64, H=128, d=64, ctx=[900, 300], T=5, capacity=1024),
    "many_heads": dict(B=64, m=8, k=300, d_idx=128, H=100, d=128, ctx=[900], T=9, capacity=1024),
    # 200 rows: one part per query
    "rows_200": dict(SMALL, ctx=[950, 800, 700, 650, 600], T=40, capacity=1024, kind="binary"),
    # 640 and 1280 rows: the selections for many rows
    "rows_640": dict(SMALL, ctx=list(range(955, 855, -10)), T=64, capacity=1024, kind="random"),
    "rows_1280": dict(B=100, m=5, k=130, d_idx=128, H=2, d=64, ctx=list(range(1950, 1930, -1)), T=64, capacity=2100),
    # many rows whose keys do not all start on 16 bytes
    "rows_odd": dict(B=7, m=3, k=11, d_idx=64, H=2, d=128, ctx=list(range(60, 70)), T=64, capacity=203),
    # more than 128 MB of kept blocks: the token scores go through work lists. One row, odd, whole, two and eight
    # pieces of 128 rows per block; small blocks that a path completes
    "lists_1": dict(B=1, m=512, k=300, d_idx=128, H=2, d=64, ctx=list(range(700, 717)), T=64, capacity=800),
    "lists_7": dict(B=7, m=512, k=900, d_idx=128, H=4, d=128, ctx=[4200, 3900, 4201], T=64, capacity=4270),
    "lists_16": dict(B=16, m=400, k=1500, d_idx=128, H=2, d=64, ctx=[7000, 6900], T=50, capacity=7104, kind="chain"),
    "lists_100": dict(B=100, m=80, k=700, d_idx=128, H=16, d=64, ctx=[9950, 9001], T=40, capacity=10100, kind="binary"),
    "lists_64": dict(B=64, m=200, k=2000, d_idx=64, H=4, d=128, ctx=[16000, 15000], T=48, capacity=16384),
    "lists_200": dict(B=200, m=70, k=500, d_idx=128, H=8, d=128, ctx=[17990, 15001], T=32, capacity=18200),
    "lists_256": dict(B=256, m=64, k=2048, d_idx=128, H=64, d=128, ctx=[18000, 17919], T=20, capacity=18176),
    "lists_1024": dict(B=1024, m=16, k=500, d_idx=128, H=1, d=64, ctx=[18420, 17000], T=20, capacity=19456, kind="chain"),
    "wide_rows": dict(B=64, m=300, k=1000, d_idx=64, H=4, d=64, ctx=[30000, 20095], T=6, capacity=32768),
    "scaled": dict(SMALL, ctx=[900], T=6, capacity=1024, scale=0.7),
    # logits hundreds of nats apart: weights that leave the range of a list's first tile
    "hot": dict(B=64, m=16, k=700, d_idx=64, H=20, d=64, ctx=[1900, 1500], T=9, capacity=2048, scale=14.0),
    "hot_wide": dict(B=128, m=8, k=1000, d_idx=128, H=70, d=128, ctx=[1900, 1000], T=40, capacity=2048, scale=8.0),
    # 4 and 64 tiles of kept rows per node
    "long_lists": dict(B=128, m=64, k=8192, d_idx=64, H=3, d=128, ctx=[8190, 9000, 300], T=7, capacity=9216),
    # every score the same: ties go to the lowest position
    "ties": dict(SMALL, ctx=[1000, 700], T=20, capacity=1088, zero_q=True, kind="chain"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", STEP_CASES)
def test_step_against_oracle(hsa, name):
    c = Case(hsa, **STEP_CASES[name])
    O, idx = c.run()
    rows = c.batch * c.T
    some = {(b, i) for b in range(c.batch) for i in range(b % 7, c.T, 11)}
    c.check(O, idx, some if rows > 400 or name.startswith("lists") else None)
    c.check_caches()
    # the same call again, over rows drafted before: the same bits
    O2, idx2 = c.run()
    import torch
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16)) and torch.equal(idx, idx2)
    assert hsa.hsa_device_status(reset=False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["ragged", "block_200", "rows_200", "many_heads", "lists_200"])
def test_rows_that_are_not_kept_do_not_matter(hsa, name):
    """NaN and infinities behind the drafted rows, and in the K and V rows that no node keeps."""
    import torch
    c = Case(hsa, **STEP_CASES[name])
    O, idx = c.run()
    for b in range(c.batch):
        used = torch.zeros(c.capacity, dtype=torch.bool, device="cuda")
        rows = idx[b][idx[b] >= 0].long()
        used[rows] = True
        n = int((c.pos[b] >= 0).sum())
        behind = torch.arange(c.capacity, device="cuda") >= int(c.ctx[b]) + n
        c.g["kc"][b, behind] = float("nan")
        for t, bad in (("Kc", float("nan")), ("Vc", float("inf"))):
            c.g[t][b, ~used] = bad
    O2, idx2 = c.run()
    assert torch.equal(idx, idx2) and torch.equal(O.view(torch.int16), O2.view(torch.int16))


@pytest.mark.gpu
def test_step_128k_batch32(hsa):
    ctx = [131072 - 97 * b for b in range(32)]
    ctx[3], ctx[9] = 131071, 130000
    c = Case(hsa, ctx=ctx, T=16, capacity=131072 + 256, B=128, m=64, k=2048, d_idx=128, H=64, d=128)
    O, idx = c.run()
    c.check(O, idx, nodes={(0, 0), (0, 15), (3, 4), (3, 12), (9, 8), (17, 1), (31, 15)})
    rows = idx.cpu().numpy()
    assert (np.diff(rows, axis=2) > 0).all() and (rows >= 0).all()


@pytest.mark.gpu
def test_step_1m_context(hsa):
    c = Case(hsa, ctx=[(1 << 20) - 3], T=64, capacity=(1 << 20) + 128, B=128, m=64, k=2048, d_idx=128, H=64, d=128,
             kind="binary")
    O, idx = c.run()
    c.check(O, idx, nodes={(0, 0), (0, 31), (0, 63)})


@pytest.mark.gpu
def test_caches_of_more_than_2_31_values(hsa):
    """The last of 2064 sequences in caches of 2.16e9 values each gives what it gives alone; a step and a commit."""
    import torch
    big, cap, T = 2064, 8192, 3
    c = Case(hsa, ctx=[8100], T=T, capacity=cap, B=128, m=8, k=300, d_idx=128, H=8, d=128, kind="chain", seed=3)
    assert big * cap * c.d > 1 << 31
    g1 = dict(c.g)
    g = {}
    for n in ("kc", "Kc", "Vc"):
        g[n] = torch.empty((big, cap, 128), dtype=torch.bfloat16, device="cuda")
        g[n][-1] = g1[n][0]
    g["ksum"] = torch.empty((big, cap // 128, 128), device="cuda")
    g["ksum"][-1] = g1["ksum"][0]
    g["ctx"] = torch.full((big,), -1, dtype=torch.int32, device="cuda")
    g["ctx"][-1] = 8100
    for n in ("q", "kn", "Q", "Kn", "Vn"):
        g[n] = torch.zeros((big, *g1[n].shape[1:]), dtype=torch.bfloat16, device="cuda")
        g[n][-1] = g1[n][0]
    g["pos"] = torch.full((big, T), -1, dtype=torch.int32, device="cuda")
    g["pos"][-1] = g1["pos"][0]
    g["paths"] = torch.full((big, T, T), -1, dtype=torch.int32, device="cuda")
    g["paths"][-1] = g1["paths"][0]
    want_O, want_idx = c.run()
    c.g, c.batch = g, big
    O, idx = c.run()
    assert torch.equal(O[-1].view(torch.int16), want_O[0].view(torch.int16)) and torch.equal(idx[-1], want_idx[0])
    assert (O[:-1] == 0).all() and (idx[:-1] == -1).all()
    acc = torch.full((big,), -1, dtype=torch.int32, device="cuda")
    acc[-1] = T - 1
    for gg, b, a in ((g, big, acc), (g1, 1, acc[-1:].clone())):
        hsa.hsa_tree_commit(c.p, b, T, cap, gg["ctx"], gg["paths"], a, gg["kc"], gg["Kc"], gg["Vc"], gg["ksum"])
    for n in ("kc", "Kc", "Vc"):
        assert torch.equal(g[n][-1].view(torch.int16), g1[n][0].view(torch.int16)), n
    assert int(g["ctx"][-1]) == 8103 and (g["ctx"][:-1] == -1).all()


@pytest.mark.gpu
def test_one_node_is_a_decode_step(hsa):
    import torch
    kw = dict(B=64, m=8, k=256, d_idx=64, H=4, d=64)
    ctx = [1, 63, 500, 1000, 1023, 0]
    c = Case(hsa, ctx=ctx, T=1, capacity=1024, **kw)
    O, idx = c.run()
    g = c.g
    ws = torch.empty(hsa.hsa_decode_workspace_size(c.p, c.batch, 1024), dtype=torch.uint8, device="cuda")
    Od = torch.empty((c.batch, 4, 64), dtype=torch.bfloat16, device="cuda")
    idxd = torch.empty((c.batch, 256), dtype=torch.int32, device="cuda")
    hsa.hsa_decode_step(c.p, c.batch, 1024, g["ctx"], g["kc"], g["Kc"], g["Vc"], g["ksum"], g["q"], g["kn"], g["Q"],
                        g["Kn"], g["Vn"], Od, idxd, ws)
    assert torch.equal(idx[:, 0], idxd)
    assert torch.equal(O[:, 0].view(torch.int16), Od.view(torch.int16))  # the same parts, the same kernels


@pytest.mark.gpu
def test_stale_plan_reaches_nothing_outside(hsa):
    """Positions and paths that do not belong to the lengths: no node of such a sequence takes part, or a node
    reads only rows of its own sequence; nothing is written outside the drafted rows."""
    import torch
    c = Case(hsa, ctx=[500, 600, 700, 900], T=8, capacity=1024, **SMALL)
    g = c.g
    g["pos"][0] = torch.arange(8, dtype=torch.int32, device="cuda")            # positions below the length
    g["pos"][1] += 200                                                         # far behind it
    g["paths"][2] = 1 << 30                                                    # entries that are no nodes
    g["pos"][3, 5:] = 1 << 30
    before = {n: g[n].clone() for n in ("kc", "Kc", "Vc")}
    O, idx = c.run()
    assert (idx[0] == -1).all() and (idx[1] == -1).all() and (idx[3, 5:] == -1).all()
    assert (O[:2] == 0).all() and (O[3, 5:] == 0).all()
    assert (idx[2] < 700 + 8).all()
    for n, was in before.items():
        for b in range(4):
            at = int(c.ctx[b])
            assert torch.equal(g[n][b, :at], was[b, :at]) and torch.equal(g[n][b, at + 8:], was[b, at + 8:]), n
        assert torch.equal(g[n][0], was[0]) and torch.equal(g[n][1], was[1])


@pytest.mark.gpu
def test_step_stays_inside_its_buffers(hsa):
    import torch
    guard, fill = 4096, 0xA5
    for name in ("ragged", "block_200", "odd_k", "rows_200", "lists_7", "lists_200"):
        c = Case(hsa, **STEP_CASES[name])
        want_O, want_idx = c.run()
        sizes = dict(ws=hsa.hsa_tree_workspace_size(c.p, c.batch, c.T, c.capacity), O=want_O.numel() * 2,
                     idx=want_idx.numel() * 4)
        bufs = {n: torch.full((2 * guard + s,), fill, dtype=torch.uint8, device="cuda") for n, s in sizes.items()}
        inner = {n: b[guard:guard + sizes[n]] for n, b in bufs.items()}
        O = inner["O"].view(torch.bfloat16).view(want_O.shape)
        idx = inner["idx"].view(torch.int32).view(want_idx.shape)
        c.run(ws=inner["ws"], O=O, idx=idx)
        assert torch.equal(O.view(torch.int16), want_O.view(torch.int16)) and torch.equal(idx, want_idx), name
        for n, b in bufs.items():
            assert (b[:guard] == fill).all() and (b[guard + sizes[n]:] == fill).all(), (name, n)


@pytest.mark.gpu
def test_step_without_indices_and_on_another_stream(hsa):
    import torch
    c = Case(hsa, **STEP_CASES["rows_200"])
    want_O, _ = c.run()
    g = c.g
    ws = torch.empty(hsa.hsa_tree_workspace_size(c.p, c.batch, c.T, c.capacity), dtype=torch.uint8, device="cuda")
    O = torch.empty_like(want_O)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hsa.hsa_tree_step(c.p, c.batch, c.T, c.capacity, g["ctx"], g["pos"], g["paths"], g["kc"], g["Kc"], g["Vc"],
                      g["ksum"], g["q"], g["kn"], g["Q"], g["Kn"], g["Vn"], O, None, ws, side)
    side.synchronize()
    assert torch.equal(O.view(torch.int16), want_O.view(torch.int16))


@pytest.mark.gpu
def test_two_steps_at_once(hsa):
    """Two calls on two streams, each with its own caches and workspace."""
    import torch
    cases = [Case(hsa, **dict(STEP_CASES[n], seed=s)) for n, s in (("lists_256", 5), ("block_256", 6))]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(c.run())
        torch.cuda.synchronize()
        for (O, idx), (wO, widx) in zip(got, want):
            assert torch.equal(O.view(torch.int16), wO.view(torch.int16)) and torch.equal(idx, widx)


# ------------------------------------------------------------------ commit

def commit_reference(c, accepted):
    """Host caches, sums of newly complete blocks and lengths after accepting `accepted` nodes."""
    kc, Kc, Vc = (host_bits(c.g[n]) for n in ("kc", "Kc", "Vc"))
    ctx = c.ctx.astype(np.int64).copy()
    sums = {}
    for b, a in enumerate(accepted):
        if not (0 <= a < c.T) or c.pos[b, a] < 0:
            continue
        path = [int(j) for j in c.paths[b, a] if j >= 0]
        at = int(ctx[b])
        for cache in (kc, Kc, Vc):
            cache[b, at:at + len(path)] = cache[b, [at + j for j in path]].copy()
        for blk in range(at // c.B, (at + len(path)) // c.B):
            sums[b, blk] = oracle.block_sums(kc[b, blk * c.B:(blk + 1) * c.B], c.B)[0]
        ctx[b] += len(path)
    return kc, Kc, Vc, sums, ctx


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["ragged", "chain_small_blocks", "block_of_one", "odd_block", "block_100", "block_1024",
                                  "rows_200", "one_node"])
@pytest.mark.parametrize("which", ["last", "middle", "none"])
def test_commit(hsa, name, which):
    import torch
    c = Case(hsa, **STEP_CASES[name])
    c.run()
    a = {"last": c.T - 1, "middle": c.T // 2, "none": -1}[which]
    accepted = np.full(c.batch, a, np.int32)
    if c.batch > 1:
        accepted[1] = c.T if which == "last" else -5  # no node: left as it is
    want = commit_reference(c, accepted)
    before = c.g["ksum"].clone()
    hsa.hsa_tree_commit(c.p, c.batch, c.T, c.capacity, c.g["ctx"], c.g["paths"], torch.from_numpy(accepted).cuda(),
                        c.g["kc"], c.g["Kc"], c.g["Vc"], c.g["ksum"])
    for n, w in zip(("kc", "Kc", "Vc"), want):
        assert np.array_equal(host_bits(c.g[n]), w), n
    ks, was = c.g["ksum"].cpu().numpy(), before.cpu().numpy()
    for (b, blk), w in want[3].items():
        assert np.array_equal(ks[b, blk], w), (b, blk)
        was[b, blk] = w
    assert np.array_equal(ks, was, equal_nan=True)
    assert np.array_equal(c.g["ctx"].cpu().numpy(), want[4])


@pytest.mark.gpu
def test_commit_of_paths_that_are_none(hsa):
    """Paths that do not end in the accepted node, run backwards or leave the tree change nothing."""
    import torch
    c = Case(hsa, ctx=[500, 600, 700, 800, 1020], T=4, capacity=1024, kind="chain", **SMALL)
    c.run()
    bad = torch.full((5, 4, 4), -1, dtype=torch.int32, device="cuda")
    bad[0, 3, :2] = torch.tensor([0, 1])            # ends in another node
    bad[1, 3] = torch.tensor([0, 2, 1, 3])          # backwards
    bad[2, 3, :2] = torch.tensor([0, 1 << 30])      # no node
    bad[3, 3] = -1                                  # a node that takes no part
    bad[4, 3] = torch.tensor([0, 1, 2, 3])          # a path, whose rows end with the cache
    before = {n: c.g[n].clone() for n in ("kc", "Kc", "Vc", "ksum")}
    hsa.hsa_tree_commit(c.p, 5, 4, 1024, c.g["ctx"], bad, torch.full((5,), 3, dtype=torch.int32, device="cuda"),
                        c.g["kc"], c.g["Kc"], c.g["Vc"], c.g["ksum"])
    assert c.g["ctx"].tolist() == [500, 600, 700, 800, 1024]
    for n in ("kc", "Kc", "Vc"):
        assert torch.equal(c.g[n], before[n])  # (the chain's rows are in place already)
    assert torch.equal(c.g["ksum"][:4].view(torch.int32), before["ksum"][:4].view(torch.int32))
    assert np.array_equal(c.g["ksum"][4, 15].cpu().numpy(), oracle.block_sums(host_bits(c.g["kc"])[4, 960:], 64)[0])


# ------------------------------------------------------------------ a whole round

def verification_round(hsa, seed, graph):
    """Three rounds of plan, norm + rotation, step and commit, beside the same accepted tokens taken one by one
    with hsa_decode_step from the same projections."""
    import torch
    B, m, k, di, H, d, T, cap, batch = 64, 6, 200, 64, 8, 64, 12, 1024, 3
    p = hsa.params(B=B, m=m, k=k, d_idx=di, H=H, d=d)
    ctx0 = [700, 62, 319]
    kc, Kc, Vc = (dev(synth.int_bf16((batch, cap, di), seed, 2)), dev(synth.normal_bf16((batch, cap, d), seed, 4)),
                  dev(synth.normal_bf16((batch, cap, d), seed, 5)))
    ks = torch.zeros((batch, cap // B, di), device="cuda")
    for b in range(batch):
        hsa.hsa_block_sums(p, ctx0[b], kc[b], ks[b])
    inv = (10000.0 ** (-torch.arange(0, d, 2, device="cuda").float() / d)).contiguous()
    tree = [kc.clone(), Kc.clone(), Vc.clone(), ks.clone(), torch.tensor(ctx0, dtype=torch.int32, device="cuda")]
    seq = [kc, Kc, Vc, ks, tree[4].clone()]
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    parents, positions, paths, accepted = i32(batch, T), i32(batch, T), i32(batch, T, T), i32(batch)
    x = dict(q=bf(batch, T, di), k=bf(batch, T, di), Q=bf(batch * T, H, d), K=bf(batch * T, d), V=bf(batch, T, d))
    Qr, Kr, O, idx = bf(batch * T, H, d), bf(batch * T, d), bf(batch, T, H, d), i32(batch, T, k)
    ws = torch.empty(hsa.hsa_tree_workspace_size(p, batch, T, cap), dtype=torch.uint8, device="cuda")

    def one_round():
        hsa.hsa_tree_plan(batch, T, cap, tree[4], None, parents, positions, paths)
        hsa.hsa_qk_norm_rope(batch * T, H, d, x["Q"], x["K"], None, None, 1e-6, inv, d, False, positions, 0, Qr, Kr)
        hsa.hsa_tree_step(p, batch, T, cap, tree[4], positions, paths, *tree[:4], x["q"], x["k"], Qr, Kr, x["V"], O,
                          idx, ws)
        hsa.hsa_tree_commit(p, batch, T, cap, tree[4], paths, accepted, *tree[:4])

    captured = None
    if graph:
        accepted.fill_(-1)
        parents.fill_(-1)
        for t in x.values():
            t.zero_()
        one_round()  # (nothing accepted: only the drafted rows are touched)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            one_round()
    wsd = torch.empty(hsa.hsa_decode_workspace_size(p, batch, cap), dtype=torch.uint8, device="cuda")
    for r in range(3):
        par = make_parents("random", batch, T, seed + r)
        parents.copy_(torch.from_numpy(par))
        acc = np.array([T - 1, T - 2, -1 if r == 1 else T - 3], np.int32)
        accepted.copy_(torch.from_numpy(acc))
        s = seed + 100 * r
        for n, t, ints in (("q", 30, 1), ("k", 31, 1), ("Q", 33, 0), ("K", 34, 0), ("V", 35, 0)):
            x[n].copy_(dev((synth.int_bf16 if ints else synth.normal_bf16)(tuple(x[n].shape), s, t)))
        lens = seq[4].cpu().numpy().copy()
        captured.replay() if graph else one_round()
        # the same tokens one by one; a sequence that has taken all of its path is held back by its length
        pos, pth = plan_reference(par, None, lens, cap)
        chain = [[int(j) for j in pth[b, acc[b]] if j >= 0] if acc[b] >= 0 else [] for b in range(batch)]
        for step in range(max(len(c) for c in chain)):
            on = [step < len(c) for c in chain]
            at = [c[step] if o else 0 for c, o in zip(chain, on)]
            pick = lambda t: torch.stack([t.view(batch, T, *t.shape[1:] if t.shape[0] == batch * T else t.shape[2:])[b, at[b]]  # noqa: E731
                                          for b in range(batch)])
            keep = seq[4].clone()
            seq[4].copy_(torch.where(torch.tensor(on, device="cuda"), seq[4], cap))  # cap: the step skips it
            Qn, Kn = hsa.qk_norm_rope(pick(x["Q"]), pick(x["K"]), inv_freq=inv, positions=seq[4].clone())
            Od, idxd = bf(batch, H, d), i32(batch, k)
            hsa.hsa_decode_step(p, batch, cap, seq[4], *seq[:4], pick(x["q"]), pick(x["k"]), Qn, Kn, pick(x["V"]), Od,
                                idxd, wsd)
            seq[4].copy_(torch.where(torch.tensor(on, device="cuda"), keep + 1, keep))
            for b in range(batch):
                if not on[b]:
                    continue
                got, want = idx[b, at[b]].cpu().numpy(), idxd[b].cpu().numpy()
                c = int(lens[b])
                back = {c + j: c + s for s, j in enumerate(chain[b])}
                assert [back.get(int(v), int(v)) for v in got] == want.tolist(), (r, step, b)
                assert (O[b, at[b]].float() - Od[b].float()).abs().max() <= 2e-2
        assert torch.equal(tree[4], seq[4])
        for b in range(batch):
            n = int(seq[4][b])
            for u, v in zip(tree[:3], seq[:3]):
                assert torch.equal(u[b, :n].view(torch.int16), v[b, :n].view(torch.int16))
            assert torch.equal(tree[3][b, :n // B], seq[3][b, :n // B])


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_rounds_equal_decode_steps(hsa, graph):
    verification_round(hsa, 71, graph)


# ------------------------------------------------------------------ refusals (CPU)

def vp(x):
    return ctypes.c_void_p(x) if x else None


STEP_PTRS = ["ctx", "pos", "paths", "kc", "Kc", "Vc", "ks", "q", "kn", "Q", "Kn", "Vn", "O", "idx", "ws"]


def call_step(hsa, batch=2, T=4, capacity=1024, params=None, ws_bytes=1 << 40, **over):
    p = hsa.params(**dict(dict(B=64, m=8, k=256, d_idx=64, H=4, d=64), **(params or {})))
    ptr = {n: 0x10000 * (i + 1) for i, n in enumerate(STEP_PTRS)}
    ptr.update(over)
    return hsa.load().hsa_tree_step(ctypes.byref(p), batch, T, capacity, *[vp(ptr[n]) for n in STEP_PTRS], ws_bytes,
                                    None)


@pytest.mark.parametrize("over", [
    dict(batch=-1), dict(T=0), dict(T=TMAX + 1), dict(capacity=0), dict(capacity=1000), dict(capacity=64 * 16385),
    dict(batch=1 << 28), dict(batch=1 << 21, capacity=1024), dict(params=dict(B=0)), dict(params=dict(m=1)),
    dict(params=dict(k=0)), dict(params=dict(d_idx=32)), dict(params=dict(H=129)), dict(params=dict(d=256)),
    dict(params=dict(scale=-1.0)), dict(params=dict(B=96, m=171), capacity=960),
] + [{n: None} for n in STEP_PTRS if n not in ("idx", "ws")]
  + [{n: 0x10008} for n in STEP_PTRS if n not in ("ctx", "pos", "paths", "ws")]
  + [{n: 0x10002} for n in ("ctx", "pos", "paths")])
def test_step_refusals(hsa, over):
    assert call_step(hsa, **over) == 1


def test_step_workspace_refusals(hsa):
    p = hsa.params(B=64, m=8, k=256, d_idx=64, H=4, d=64)
    need = hsa.hsa_tree_workspace_size(p, 2, 4, 1024)
    assert need >= 2 * 4 * (8 * 64 * 4 + 256 * 4)
    assert call_step(hsa, ws=None) == 2 and call_step(hsa, ws=0x10004) == 2
    assert call_step(hsa, ws_bytes=need - 1) == 2
    assert call_step(hsa, batch=0, ws=None) == 0  # nothing to do


def test_workspace_size_refuses_a_missing_answer(hsa):
    p = hsa.params(B=64, m=8, k=256, d_idx=64, H=4, d=64)
    assert hsa.load().hsa_tree_workspace_size(ctypes.byref(p), 2, 4, 1024, None) == 1


@pytest.mark.parametrize("over", [dict(batch=-1), dict(T=0), dict(T=65), dict(capacity=0), dict(capacity=1 << 31),
                                  dict(ctx=None), dict(parents=None), dict(pos=None), dict(paths=None),
                                  dict(n=0x10002), dict(parents=0x10001)])
def test_plan_refusals(hsa, over):
    v = dict(dict(batch=2, T=4, capacity=1024, ctx=0x10000, n=None, parents=0x20000, pos=0x30000, paths=0x40000), **over)
    assert hsa.load().hsa_tree_plan(v["batch"], v["T"], v["capacity"], vp(v["ctx"]), vp(v["n"]), vp(v["parents"]),
                                    vp(v["pos"]), vp(v["paths"]), None) == 1


@pytest.mark.parametrize("over", [dict(batch=-1), dict(T=0), dict(T=65), dict(capacity=1000), dict(d_idx=96),
                                  dict(ctx=None), dict(paths=None), dict(acc=None), dict(kc=None), dict(Kc=0x10008),
                                  dict(Vc=None), dict(ks=0x10004), dict(acc=0x10002)])
def test_commit_refusals(hsa, over):
    v = dict(dict(batch=2, T=4, capacity=1024, d_idx=64, ctx=0x10000, paths=0x20000, acc=0x30000, kc=0x40000,
                  Kc=0x50000, Vc=0x60000, ks=0x70000), **over)
    p = hsa.params(B=64, m=8, k=256, d_idx=v["d_idx"], H=4, d=64)
    assert hsa.load().hsa_tree_commit(ctypes.byref(p), v["batch"], v["T"], v["capacity"],
                                      *[vp(v[n]) for n in ("ctx", "paths", "acc", "kc", "Kc", "Vc", "ks")], None) == 1
