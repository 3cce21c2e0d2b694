"""Cases of the serving operators around the decode step: the per-head norm
with the position rotation that makes queries and keys from the projections,
and the verification of a drafted token tree (plan, step, commit).

``own`` false: the operators in elementary torch operations. ``own`` true:
the library's calls (include/hsa.h) on the same inputs.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
TREE_MAX = 64  # drafted nodes per sequence


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's queries and keys: the smallest call, latency counts
        dict(name="rope_decode_b32", op="rope", L=32, H=64, d=128, rot=128, inter=False, fused=False, scattered=True),
        # the 2K prefill's layer: few heads of 64, adjacent pairs
        dict(name="rope_prefill_2k", op="rope", L=2048, H=4, d=64, rot=64, inter=True, fused=False, scattered=False),
        # the 16K prefill read straight out of a fused projection's rows, half of each head rotated
        dict(name="rope_fused_16k", op="rope", L=16384, H=16, d=128, rot=64, inter=False, fused=True, scattered=False),
        # the 64K prefill: 64 heads, bandwidth counts
        dict(name="rope_prefill_64k", op="rope", L=65536, H=64, d=128, rot=128, inter=False, fused=False, scattered=False),
        # the trees of one serving batch, planned once per drafting round
        dict(name="plan_b32_t16", op="plan", batch=32, T=16, ragged=True),
        # a large batch of the largest trees
        dict(name="plan_b256_t64", op="plan", batch=256, T=64, ragged=True),
        # a small layer with ragged short contexts, some below the selection's thresholds
        dict(name="tree_small_b5_t7", op="tree", batch=5, T=7, ctx=1000, spread=990, capacity=1024, B=64, m=8, k=256,
             d_idx=64, H=4, d=64),
        # one user's short draft over a long context: latency counts
        dict(name="tree_128k_b1_t8", op="tree", batch=1, T=8, ctx=131072, spread=300, capacity=131328, B=128, m=64,
             k=2048, d_idx=128, H=64, d=128),
        # the decode workload's batch with sixteen drafted tokens for each sequence
        dict(name="tree_128k_b32_t16", op="tree", batch=32, T=16, ctx=131072, spread=5000, capacity=131328, B=128,
             m=64, k=2048, d_idx=128, H=64, d=128),
        # the largest tree over the longest context
        dict(name="tree_1m_b1_t64", op="tree", batch=1, T=64, ctx=1048576, spread=200, capacity=1048832, B=128, m=64,
             k=2048, d_idx=128, H=64, d=128),
        # the accepted paths of a serving batch moved into place
        dict(name="commit_b32_t16", op="commit", batch=32, T=16, ctx=16000, spread=15000, capacity=16384, B=128,
             d_idx=128, d=128),
        # large trees in small layers, several blocks completed by one path
        dict(name="commit_b64_t64", op="commit", batch=64, T=64, ctx=4000, spread=3900, capacity=4096, B=64,
             d_idx=64, d=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "rope", "plan", "tree", "tree", "commit"])
    if op == "rope":
        d, H = rng.choice([64, 128]), log(1, 128)
        L = min(log(1, 65536), 65536 * 64 * 128 // (H * d))
        return dict(op=op, L=L, H=H, d=d, rot=16 * rng.randint(1, d // 16), inter=rng.random() < 0.5,
                    fused=rng.random() < 0.5, scattered=rng.random() < 0.5)
    if op == "plan":
        return dict(op=op, batch=log(8, 256), T=rng.randint(2, TREE_MAX), ragged=rng.random() < 0.7)
    if op == "commit":
        B = rng.choice([16, 64, 100, 128, 256])
        capacity = B * log(2, 8192 // B)
        T = rng.randint(1, min(TREE_MAX, capacity // 2))
        ctx = rng.randint(capacity // 2, capacity - T)
        return dict(op=op, batch=log(1, 64), T=T, ctx=ctx, spread=rng.randint(0, ctx), capacity=capacity, B=B,
                    d_idx=rng.choice([64, 128]), d=rng.choice([64, 128]))
    B = rng.choice([32, 64, 128, 256, 100])
    m = rng.randint(2, 8192 // B)
    T = rng.randint(1, TREE_MAX)
    batch = min(log(1, 32), 512 // T)
    capacity = B * (log(1000, 131072) // B + 2)
    ctx = rng.randint(capacity // 2, capacity - T)
    return dict(op=op, batch=batch, T=T, ctx=ctx, spread=rng.randint(0, ctx - 1), capacity=capacity, B=B, m=m,
                k=log(64, 2048), d_idx=rng.choice([64, 128]), H=log(1, 64), d=rng.choice([64, 128]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(g, *shape):
    """Indexer values: integers in [-8, 8], so that every score is exact and selections are comparable."""
    return torch.randint(-8, 9, shape, generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)


def _trees(g, batch, T, ragged):
    """Random parents (-1: a child of the last cached token) and node counts."""
    i = torch.arange(T, device="cuda")
    u = torch.rand((batch, T), generator=g, device="cuda")
    # one node in four hangs anywhere below it, the others off one of the last three nodes
    near = i - 1 - (u * 12).long() % 3
    far = (u * (i + 1)).long() - 1
    v = torch.rand((batch, T), generator=g, device="cuda")
    parents = torch.where(v < 0.25, far, near).clamp(min=-1).minimum(i - 1).to(torch.int32)
    n = torch.full((batch,), T, device="cuda", dtype=torch.int32)
    if ragged:
        n = torch.randint(0, T + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
    return parents.contiguous(), n


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "rope":
        L, H, d, rot = case["L"], case["H"], case["d"], case["rot"]
        if case["fused"]:  # queries, keys and values of a token in one row
            row = _normal(g, L, (H + 2) * d)
            s["Q"], s["K"] = row[:, : H * d].unflatten(1, (H, d)), row[:, H * d: (H + 1) * d]
        else:
            s["Q"], s["K"] = _normal(g, L, H, d), _normal(g, L, d)
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (THETA ** (-2.0 * i / rot)).float()
        s["pos"], s["pos0"] = None, 1000 if L > 1 else 0
        if case["scattered"]:  # decode: every row at its sequence's own length
            s["pos"] = torch.randint(0, 1 << 20, (L,), generator=g, device="cuda", dtype=torch.int32)
        s["Qo"] = torch.empty((L, H, d), device="cuda", dtype=torch.bfloat16)
        s["Ko"] = torch.empty((L, d), device="cuda", dtype=torch.bfloat16)
        return s
    batch, T = case["batch"], case["T"]
    if case["op"] == "plan":
        s["parents"], s["n"] = _trees(g, batch, T, case["ragged"])
        s["capacity"] = 131072
        s["ctx"] = torch.randint(0, 131072 - T, (batch,), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = torch.empty((batch, T), device="cuda", dtype=torch.int32)
        s["paths"] = torch.empty((batch, T, T), device="cuda", dtype=torch.int32)
        return s
    cap, B, di, d = case["capacity"], case["B"], case["d_idx"], case["d"]
    parents, n = _trees(g, batch, T, batch > 1)
    lo = max(0, case["ctx"] - case["spread"])
    s["ctx_len"] = torch.randint(lo, case["ctx"] + 1, (batch,), generator=g, device="cuda",
                                 dtype=torch.int32).clamp(max=cap - T)
    s["positions"], s["paths"] = _plan(parents, n, s["ctx_len"], cap)
    s["k_idx_cache"] = _ints(g, batch, cap, di)
    s["K_cache"], s["V_cache"] = _normal(g, batch, cap, d), _normal(g, batch, cap, d)
    s["ksum"] = s["k_idx_cache"].view(batch, cap // B, B, di).sum(2, dtype=torch.float32)
    if case["op"] == "commit":
        # the deepest node of the first half of a tree is accepted, of every eighth sequence none
        depth = (s["positions"] - s["ctx_len"][:, None]).masked_fill(s["positions"] < 0, -1)
        acc = depth[:, : (T + 1) // 2].argmax(1).to(torch.int32)
        acc = torch.where(s["positions"].gather(1, acc.long()[:, None])[:, 0] < 0, -1, acc)
        s["accepted"] = torch.where(torch.arange(batch, device="cuda") % 8 == 7, -1, acc).to(torch.int32)
        return s
    H = case["H"]
    # the nodes of a tree ask for much the same tokens: three values in four are the sequence's own
    base, fresh = _ints(g, batch, 1, di), _ints(g, batch, T, di)
    s["q_idx"] = torch.where(torch.rand((batch, T, di), generator=g, device="cuda") < 0.75, base, fresh)
    s["k_idx"] = _ints(g, batch, T, di)
    s["Q"], s["K"], s["V"] = _normal(g, batch, T, H, d), _normal(g, batch, T, d), _normal(g, batch, T, d)
    s["O"] = torch.empty((batch, T, H, d), device="cuda", dtype=torch.bfloat16)
    s["indices"] = torch.empty((batch, T, case["k"]), device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------------ plain forms

def _plan(parents, n, ctx, capacity):
    """positions [batch][T] and paths [batch][T][T] (ancestors from the root down, then the node, -1 after)."""
    batch, T = parents.shape
    i = torch.arange(T, device=parents.device)
    # anc[b][i][j]: j is on i's path. The path's closure by repeated squaring of the parent relation.
    up = (parents[:, :, None] == i) | torch.eye(T, dtype=torch.bool, device=parents.device)
    reach = up.float()
    reach = (reach @ reach).clamp(max=1)  # up to 2 levels
    reach = (reach @ reach).clamp(max=1)  # 4
    reach = (reach @ reach).clamp(max=1)  # 8
    reach = (reach @ reach).clamp(max=1)  # 16
    reach = (reach @ reach).clamp(max=1)  # 32
    reach = (reach @ reach).clamp(max=1)  # 64
    anc = reach > 0
    depth = anc.sum(2) - 1
    n = n.clamp(0, T)
    taken = (i < n[:, None]) & (ctx >= 0)[:, None] & (ctx + n <= capacity)[:, None]
    positions = torch.where(taken, ctx[:, None] + depth, -1).to(torch.int32)
    nodes = torch.where(anc, i, T).sort(dim=2).values
    paths = torch.where((nodes < T) & taken[:, :, None], nodes, -1).to(torch.int32)
    return positions, paths


def _rope_rows(x, w, cos, sin, rot, inter):
    """RMS norm over the last axis, times w, then the rotation of its first rot values; fp32, one rounding."""
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., : rot // 2], y[..., rot // 2: rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((r, y[..., rot:]), -1).to(torch.bfloat16)


def _rope(s):
    L = s["L"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(s["pos0"], s["pos0"] + L, device="cuda")
    angle = pos.double()[:, None] * s["inv_freq"].double()  # far positions: 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    return {"Q": _rope_rows(s["Q"], s["qw"], cos[:, None], sin[:, None], s["rot"], s["inter"]),
            "K": _rope_rows(s["K"], s["kw"], cos, sin, s["rot"], s["inter"])}


def _write_rows(cache, slots, taken, rows):
    b = torch.arange(cache.shape[0], device=cache.device)[:, None]
    cache[b, slots] = torch.where(taken[..., None], rows, cache[b, slots])


def _tree(s):
    batch, T, cap, B, m, k, d = (s[n] for n in ("batch", "T", "capacity", "B", "m", "k", "d"))
    dev = s["Q"].device
    ctx, pos, paths = s["ctx_len"].long(), s["positions"].long(), s["paths"].long()
    taken = pos >= 0
    slots = (ctx[:, None] + torch.arange(T, device=dev)).clamp(max=cap - 1)
    for name in ("k_idx", "K", "V"):
        _write_rows(s[name + "_cache"], slots, taken, s[name])
    bi = torch.arange(batch, device=dev)[:, None, None]
    c, q = ctx[:, None, None], s["q_idx"].float()

    def slot(p):  # cache row of position p on each node's own path
        j = (p - c).clamp(0, T - 1)
        return torch.where(p < c, p, c + paths.gather(2, j).clamp(min=0)).clamp(0, cap - 1)

    def token_scores(p):
        return torch.einsum("btnd,btd->btn", s["k_idx_cache"][bi, slot(p)].float(), q)

    # block scores: whole cached blocks from their sums, later ones from their tokens
    f = ctx // B
    nt = (B - 1 + T) // B + 1
    p = f[:, None, None] * B + torch.arange(nt * B, device=dev)
    p = p.expand(batch, T, nt * B)
    tail = torch.where(p <= pos[..., None], token_scores(p), 0.0).view(batch, T, nt, B).sum(3)
    scores = torch.einsum("btd,bnd->btn", q, s["ksum"])
    scores = torch.cat((scores, scores.new_zeros(batch, T, nt)), 2)
    scores = scores.scatter(2, (f[:, None, None] + torch.arange(nt, device=dev)).expand(batch, T, nt), tail)
    blk = torch.arange(scores.shape[2], device=dev)
    nb = (pos // B + 1)[..., None]
    scores = torch.where((blk == 0) | (blk == nb - 1), math.inf, scores).masked_fill(blk >= nb, -math.inf)
    top, which = scores.sort(dim=2, descending=True, stable=True)
    which = torch.where(top[..., :m] > -math.inf, which[..., :m], cap)
    # token scores inside the kept blocks
    p = (which[..., None] * B + torch.arange(B, device=dev)).flatten(2)
    ok = (which[..., None].expand(-1, -1, -1, B).flatten(2) < cap) & (p <= pos[..., None])
    ts = token_scores(p.clamp(max=cap - 1)).masked_fill(~ok, -math.inf)
    # ties to the lowest position: candidates in ascending order, then a stable sort by score
    order = torch.where(ok, p, 1 << 40).argsort(dim=2)
    p, ts = p.gather(2, order), ts.gather(2, order)
    top, at = ts.sort(dim=2, descending=True, stable=True)
    kk = min(k, p.shape[2])
    p = torch.where(top[..., :kk] > -math.inf, p.gather(2, at[..., :kk]), 1 << 40).sort(dim=2).values
    ok = p < 1 << 40
    rows = slot(p.clamp(max=cap - 1))
    idx = torch.full((batch, T, k), -1, device=dev, dtype=torch.int32)
    idx[..., :kk] = torch.where(ok, rows, -1).to(torch.int32)
    # attention over the kept rows
    Kr, Vr = s["K_cache"][bi, rows].float(), s["V_cache"][bi, rows].float()
    x = torch.einsum("bthd,btnd->bthn", s["Q"].float(), Kr) / math.sqrt(d)
    x = x.masked_fill(~ok[:, :, None], -math.inf)
    top = x.amax(3, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - top)
    O = torch.einsum("bthn,btnd->bthd", e, Vr) / e.sum(3, keepdim=True).clamp(min=1e-37)
    return {"O": O.to(torch.bfloat16), "indices": idx, "k_idx_cache": s["k_idx_cache"], "K_cache": s["K_cache"],
            "V_cache": s["V_cache"]}


def _commit(s):
    batch, T, cap, B = (s[n] for n in ("batch", "T", "capacity", "B"))
    ctx = s["ctx_len"].long()
    dev = ctx.device
    acc = s["accepted"].long()
    path = s["paths"].long().gather(1, acc.clamp(min=0)[:, None, None].expand(-1, 1, T))[:, 0]
    path = torch.where(acc[:, None] >= 0, path, -1)
    n = (path >= 0).sum(1)
    taken = path >= 0
    src = (ctx[:, None] + path.clamp(min=0)).clamp(max=cap - 1)
    dst = (ctx[:, None] + torch.arange(T, device=dev)).clamp(max=cap - 1)
    b = torch.arange(batch, device=dev)[:, None]
    for name in ("k_idx_cache", "K_cache", "V_cache"):
        _write_rows(s[name], dst, taken, s[name][b, src])
    # sums of the blocks that the path completes
    f = ctx // B
    nt = (B - 1 + T) // B
    # (entries past the cache's end repeat its last block, with the same values)
    blk = (f[:, None] + torch.arange(nt, device=dev)).clamp(max=cap // B - 1)
    done = (blk >= f[:, None]) & (blk < (ctx + n)[:, None] // B)
    sums = s["k_idx_cache"].view(batch, cap // B, B, -1)[b, blk].float().sum(2)
    s["ksum"][b, blk] = torch.where(done[..., None], sums, s["ksum"][b, blk])
    return {"ctx_len": (ctx + n).to(torch.int32), "k_idx_cache": s["k_idx_cache"], "K_cache": s["K_cache"],
            "V_cache": s["V_cache"], "ksum": s["ksum"]}


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if not own:
        if s["op"] == "plan":
            positions, paths = _plan(s["parents"], s["n"], s["ctx"], s["capacity"])
            return {"positions": positions, "paths": paths}
        return {"rope": _rope, "tree": _tree, "commit": _commit}[s["op"]](s)
    import hierarchical_sparse_attention_hisa_b200 as hsa
    if s["op"] == "rope":
        hsa.hsa_qk_norm_rope(s["L"], s["H"], s["d"], s["Q"], s["K"], s["qw"], s["kw"], EPS, s["inv_freq"], s["rot"],
                             s["inter"], s["pos"], s["pos0"], s["Qo"], s["Ko"])
        return {"Q": s["Qo"], "K": s["Ko"]}
    if s["op"] == "plan":
        hsa.hsa_tree_plan(s["batch"], s["T"], s["capacity"], s["ctx"], s["n"], s["parents"], s["positions"],
                          s["paths"])
        return {"positions": s["positions"], "paths": s["paths"]}
    if s["op"] == "commit":
        p = hsa.params(B=s["B"], d_idx=s["d_idx"], d=s["d"], m=2, k=1, H=1)
        ctx = s["ctx_len"].clone()  # the call advances the lengths; the next pass starts from the same ones
        hsa.hsa_tree_commit(p, s["batch"], s["T"], s["capacity"], ctx, s["paths"], s["accepted"], s["k_idx_cache"],
                            s["K_cache"], s["V_cache"], s["ksum"])
        return {"ctx_len": ctx, "k_idx_cache": s["k_idx_cache"], "K_cache": s["K_cache"], "V_cache": s["V_cache"],
                "ksum": s["ksum"]}
    p = hsa.params(B=s["B"], m=s["m"], k=s["k"], d_idx=s["d_idx"], H=s["H"], d=s["d"])
    if "workspace" not in s:  # a server allocates it once
        s["workspace"] = torch.empty(hsa.hsa_tree_workspace_size(p, s["batch"], s["T"], s["capacity"]),
                                     dtype=torch.uint8, device="cuda")
    hsa.hsa_tree_step(p, s["batch"], s["T"], s["capacity"], s["ctx_len"], s["positions"], s["paths"],
                      s["k_idx_cache"], s["K_cache"], s["V_cache"], s["ksum"], s["q_idx"], s["k_idx"], s["Q"], s["K"],
                      s["V"], s["O"], s["indices"], s["workspace"])
    return {"O": s["O"], "indices": s["indices"], "k_idx_cache": s["k_idx_cache"], "K_cache": s["K_cache"],
            "V_cache": s["V_cache"]}


def work(case):
    op = case["op"]
    if op == "rope":
        elems = case["L"] * (case["H"] + 1) * case["d"]
        # read and written once; square, scale, weight and rotate each value
        return {"bytes": 4.0 * elems + (4.0 * case["L"] if case["scattered"] else 0.0), "flops": 8.0 * elems}
    batch, T = case["batch"], case["T"]
    if op == "plan":
        return {"bytes": batch * (8.0 + 8.0 * T + 4.0 * T * T), "flops": float(batch * T * T)}
    di, d, B = case["d_idx"], case["d"], case["B"]
    row = 2.0 * di + 4.0 * d  # a token in the three caches
    if op == "commit":
        n = max(1, T // 4)  # tokens accepted of a tree of T
        return {"bytes": batch * (2.0 * n * row + 12.0 + 4.0 * T + n / B * (2.0 * B * di + 4.0 * di)),
                "flops": float(batch * n * di)}
    m, k, H = case["m"], case["k"], case["H"]
    ctx = max(1.0, case["ctx"] - case["spread"] / 2)
    nb = ctx / B
    cand = min(ctx, m * B)
    kept = min(k, cand)
    scored = cand if cand > k else 0.0
    blocks = nb if nb > m else 0.0
    per_node = 2.0 * di * (blocks + scored) + 4.0 * H * d * kept
    # a sequence's nodes may all keep the same blocks and rows, so these are counted once
    per_seq = 4.0 * di * blocks + 2.0 * di * scored + 4.0 * d * kept
    per_row = 4.0 * H * d + 2.0 * di + 2.0 * row + 4.0 * k + 4.0 + 4.0 * T
    return {"bytes": batch * (per_seq + T * per_row), "flops": batch * T * per_node}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "plan": _exact_plan, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](s)


def _exact_rope(s):
    L, d, rot = s["L"], s["d"], s["rot"]
    t = s["pos"].double() if s["pos"] is not None else s["pos0"] + torch.arange(L, device="cuda").double()
    out = {}
    for name, w in (("Q", "qw"), ("K", "kw")):
        x = s[name].double().reshape(L, -1, d)
        y = x / (x.square().sum(2, keepdim=True) / d + EPS).sqrt() * s[w].double()
        # each pair as one complex number, turned by its angle
        i = torch.arange(rot // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if s["inter"] else (i, i + rot // 2)
        angle = torch.outer(t, s["inv_freq"].double())[:, None]
        z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(angle), angle)
        y[..., a], y[..., b] = z.real, z.imag
        out[name] = y.reshape(s[name].shape)
    return out


def _exact_plan(s):
    parents, n, ctx = s["parents"].tolist(), s["n"].tolist(), s["ctx"].tolist()
    batch, T = len(parents), len(parents[0])
    positions = [[-1] * T for _ in range(batch)]
    paths = [[[-1] * T for _ in range(T)] for _ in range(batch)]
    for b in range(batch):
        for i in range(n[b]):
            chain, j = [], i
            while j >= 0:
                chain.insert(0, j)
                j = parents[b][j]
            positions[b][i] = ctx[b] + len(chain) - 1
            paths[b][i][: len(chain)] = chain
    return {"positions": torch.tensor(positions, dtype=torch.int32), "paths": torch.tensor(paths, dtype=torch.int32)}


def _exact_tree(s):
    batch, T, B, m, k, d, H = (s[n] for n in ("batch", "T", "B", "m", "k", "d", "H"))
    O = torch.zeros((batch, T, H, d), dtype=torch.float64, device="cuda")
    idx = torch.full((batch, T, k), -1, dtype=torch.int32, device="cuda")
    pos, paths, ctx = s["positions"].tolist(), s["paths"].tolist(), s["ctx_len"].tolist()
    for b in range(batch):
        c = ctx[b]
        for i in range(T):
            if pos[b][i] >= 0:
                for name in ("k_idx", "K", "V"):
                    s[name + "_cache"][b, c + i] = s[name][b, i]
        old = s["k_idx_cache"][b, :c].double() @ s["q_idx"][b].double().T  # [c][T] token scores
        new = s["k_idx"][b].double() @ s["q_idx"][b].double().T
        for i in range(T):
            if pos[b][i] < 0:
                continue
            path = [j for j in paths[b][i] if j >= 0]
            score = torch.cat((old[:, i], new[path, i]))       # along the node's own sequence
            row = torch.cat((torch.arange(c, device="cuda"), c + torch.tensor(path, device="cuda")))
            t = c + len(path) - 1
            nb = t // B + 1
            keep = torch.arange(nb, device="cuda")
            if nb > m:
                sums = score[: (nb - 1) * B].view(nb - 1, B).sum(1)[1:]
                best = torch.sort(-sums, stable=True).indices[: m - 2] + 1
                keep = torch.cat((keep[:1], best.sort().values, keep[-1:]))
            cand = (keep[:, None] * B + torch.arange(B, device="cuda")).flatten()
            cand = cand[cand <= t]
            if len(cand) > k:
                cand = cand[torch.sort(-score[cand], stable=True).indices[:k]].sort().values
            row = row[cand]
            idx[b, i, : len(row)] = row.to(torch.int32)
            w = torch.softmax(s["Q"][b, i].double() @ s["K_cache"][b, row].double().T / math.sqrt(d), 1)
            O[b, i] = w @ s["V_cache"][b, row].double()
    return {"O": O, "indices": idx, "k_idx_cache": s["k_idx_cache"], "K_cache": s["K_cache"], "V_cache": s["V_cache"]}


def _exact_commit(s):
    B, ctx = s["B"], s["ctx_len"].tolist()
    ksum = s["ksum"].double()
    for b, a in enumerate(s["accepted"].tolist()):
        if a < 0:
            continue
        path = [j for j in s["paths"][b, a].tolist() if j >= 0]
        c, n = ctx[b], len(path)
        for name in ("k_idx_cache", "K_cache", "V_cache"):
            s[name][b, c: c + n] = s[name][b, [c + j for j in path]].clone()
        for blk in range(c // B, (c + n) // B):
            ksum[b, blk] = s["k_idx_cache"][b, blk * B: (blk + 1) * B].double().sum(0)
        ctx[b] = c + n
    return {"ctx_len": torch.tensor(ctx, dtype=torch.int32), "k_idx_cache": s["k_idx_cache"],
            "K_cache": s["K_cache"], "V_cache": s["V_cache"], "ksum": ksum}
