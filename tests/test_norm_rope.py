"""hsa_qk_norm_rope against its formula in 64 bits: layouts, strides, partial
and interleaved rotations, far and negative positions, in-place calls; and
the refusals (on the CPU).

Tolerance. The result is rounded once to bf16: half a step, 2^-8 of the value.
Before that, with y the normed row (ymax its largest magnitude), in units of
2^-24: the sum of squares, the reciprocal root and the products with it and the
weight are off by at most 16 relative; the angle, 2^-32 of a turn and its
conversion to fp32, by 2^-22.3 radians (3.2); the fast sine and cosine by 2^-21.2
in [-pi, pi] (7); the coefficients and the rotation round five times (5). All of
it is relative to |a| + |b| <= 2 ymax: 2 ymax * 31.2 * 2^-24 < 4e-6 ymax, and
the rounding's half step is taken of a value that may be off by that much.
"""
import ctypes

import numpy as np
import pytest

EPS = 1e-6


def reference(x, w, inv_freq, pos, rot, inter, eps=EPS):
    """x [L][R][d] float64, pos [L] -> (rotated rows, largest normed magnitude per row)."""
    d = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    out = y.copy()
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    u = (pos[:, None].astype(np.float64) * inv_freq[None].astype(np.float64))[:, None, :]
    # (fp64 keeps the angle to 2^-53 of itself: 2^-22 radians at 2^31)
    out[..., a] = y[..., a] * np.cos(u) - y[..., b] * np.sin(u)
    out[..., b] = y[..., b] * np.cos(u) + y[..., a] * np.sin(u)
    assert out.shape[-1] == d
    return out, np.abs(y).max(-1, keepdims=True)


def check(got, x, w, inv_freq, pos, rot, inter, eps=EPS):
    ref, ymax = reference(x, w, inv_freq, pos, rot, inter, eps)
    slack = 4e-6 * ymax
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= 2.0 ** -8 * (np.abs(ref) + slack) + slack).all(), float((err - 2.0 ** -8 * np.abs(ref)).max())


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def freqs(rot, theta=10000.0):
    return (theta ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("L,H,d,rot,inter", [
    (1, 1, 64, 64, False), (1, 1, 128, 128, True), (1, 128, 128, 128, False), (1, 7, 64, 16, False),
    (33, 64, 128, 128, False), (5, 64, 128, 64, True), (257, 4, 64, 64, True), (1000, 5, 64, 48, False),
    (1000, 16, 128, 96, False), (300, 3, 128, 80, True), (77, 1, 64, 32, False), (129, 128, 64, 0, False),
    (513, 31, 128, 112, False), (4099, 1, 128, 128, False),
    # a token to a group or to a warp, on both sides of the choice
    (2367, 4, 128, 128, False), (2371, 4, 128, 128, True), (2369, 6, 128, 48, False), (2500, 7, 128, 128, False),
    (2401, 11, 64, 64, True), (2403, 12, 64, 32, False), (2405, 13, 64, 64, False),
])
@pytest.mark.parametrize("fused", [False, True])
def test_against_formula(hsa, L, H, d, rot, inter, fused):
    import torch
    g = torch.Generator(device="cuda").manual_seed(L * 131 + H + rot)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if fused:
        row = rnd(L, (H + 2) * d + 8)
        Q, K = row[:, 8:8 + H * d].unflatten(1, (H, d)), row[:, 8 + H * d: 8 + (H + 1) * d]
    else:
        Q, K = rnd(L, H, d), rnd(L, d)
    qw, kw = rnd(d), rnd(d)
    inv = freqs(rot)
    inv_t = torch.from_numpy(inv).cuda() if rot else None
    pos0 = 123457
    Qo, Ko = hsa.qk_norm_rope(Q, K, qw, kw, inv_t, pos0=pos0, eps=EPS, interleaved=inter)
    pos = pos0 + np.arange(L)
    check(f64(Qo), f64(Q), f64(qw), inv, pos, rot, inter)
    check(f64(Ko)[:, None], f64(K)[:, None], f64(kw), inv, pos, rot, inter)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(hsa, inter):
    import torch
    pos = np.array([0, 1, 4095, 131071, (1 << 20) - 1, 1 << 24, (1 << 24) + 1, (1 << 30) + 7, (1 << 31) - 1])
    L, H, d = len(pos), 6, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    Q = torch.randn((L, H, d), generator=g, device="cuda").to(torch.bfloat16)
    inv = freqs(d, theta=1e6)
    Qo, Ko = hsa.qk_norm_rope(Q, None, None, None, torch.from_numpy(inv).cuda(),
                              positions=torch.from_numpy(pos.astype(np.int32)).cuda(), interleaved=inter)
    assert Ko is None
    check(f64(Qo), f64(Q), None, inv, pos, d, inter)


@pytest.mark.gpu
def test_negative_positions_leave_rows_unwritten(hsa):
    import torch
    L, H, d = 40, 9, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    Q = torch.randn((L, H, d), generator=g, device="cuda").to(torch.bfloat16)
    K = torch.randn((L, d), generator=g, device="cuda").to(torch.bfloat16)
    pos = np.arange(L) * 17
    pos[[0, 5, 6, 39]] = [-1, -7, -(1 << 31), -1]
    inv = freqs(d)
    Qo, Ko = torch.full_like(Q, 7.0), torch.full_like(K, 7.0)
    hsa.hsa_qk_norm_rope(L, H, d, Q, K, None, None, EPS, torch.from_numpy(inv).cuda(), d, False,
                         torch.from_numpy(pos.astype(np.int32)).cuda(), 0, Qo, Ko)
    on = pos >= 0
    check(f64(Qo)[on], f64(Q)[on], None, inv, pos[on], d, False)
    check(f64(Ko)[on][:, None], f64(K)[on][:, None], None, inv, pos[on], d, False)
    assert (f64(Qo)[~on] == 7).all() and (f64(Ko)[~on] == 7).all()
    # the module's form hands such rows back as zeros
    Qz, Kz = hsa.qk_norm_rope(Q, K, inv_freq=torch.from_numpy(inv).cuda(),
                              positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    assert (f64(Qz)[~on] == 0).all() and torch.equal(Qz[on], Qo[on]) and torch.equal(Kz[on], Ko[on])


@pytest.mark.gpu
def test_in_place_keys_only_other_stream_and_guards(hsa):
    import torch
    L, H, d, pad = 700, 12, 128, 2048
    g = torch.Generator(device="cuda").manual_seed(5)
    Q = torch.randn((L, H, d), generator=g, device="cuda").to(torch.bfloat16)
    K = torch.randn((L, d), generator=g, device="cuda").to(torch.bfloat16)
    inv = torch.from_numpy(freqs(d)).cuda()
    Qo, Ko = hsa.qk_norm_rope(Q, K, inv_freq=inv)
    buf = torch.full((2 * pad + Q.numel(),), 3.0, dtype=torch.bfloat16, device="cuda")
    Qi, Ki = buf[pad:pad + Q.numel()].view_as(Q), K.clone()
    Qi.copy_(Q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hsa.hsa_qk_norm_rope(L, H, d, Qi, Ki, None, None, EPS, inv, d, False, None, 0, Qi, Ki, side)
    side.synchronize()
    assert torch.equal(Qi, Qo) and torch.equal(Ki, Ko)
    assert (buf[:pad] == 3).all() and (buf[-pad:] == 3).all()
    _, Kk = hsa.qk_norm_rope(None, K, inv_freq=inv)
    assert torch.equal(Kk, Ko)


@pytest.mark.gpu
def test_extreme_rows(hsa):
    """A row of zeros stays zero, large and tiny rows keep their norm, NaN and infinities stay in their row."""
    import torch
    H, d = 4, 64
    Q = torch.ones((3, H, d), device="cuda")
    Q[0, 0] = 0
    Q[0, 1] *= 2.0 ** 60      # squares still finite in fp32
    Q[0, 2] *= 2.0 ** -60     # far below eps
    Q[1, 0, 5] = float("nan")
    Q[1, 1, 5] = float("inf")
    Q = Q.to(torch.bfloat16)
    inv = freqs(d)
    Qo, _ = hsa.qk_norm_rope(Q, None, inv_freq=torch.from_numpy(inv).cuda(), pos0=9)
    got = f64(Qo)
    assert (got[0, 0] == 0).all()
    check(got[[0, 2]], f64(Q)[[0, 2]], None, inv, np.array([9, 11]), d, False)
    check(got[1:2, 2:], f64(Q)[1:2, 2:], None, inv, np.array([10]), d, False)
    assert np.isnan(got[1, 0]).all() and not np.isfinite(got[1, 1]).all()


# ------------------------------------------------------------------ refusals (CPU)

GOOD = dict(L=10, H=4, d=64, Q=0x10000, qs=256, K=0x20000, ks=64, qw=0x30000, kw=0x30000, eps=1e-6, inv=0x40000,
            rot=64, inter=0, pos=None, pos0=0, Qo=0x50000, Ko=0x60000)


def call(hsa, **over):
    v = dict(GOOD, **over)
    ptr = lambda x: ctypes.c_void_p(x) if x else None  # noqa: E731
    return hsa.load().hsa_qk_norm_rope(v["L"], v["H"], v["d"], ptr(v["Q"]), v["qs"], ptr(v["K"]), v["ks"], ptr(v["qw"]),
                                       ptr(v["kw"]), v["eps"], ptr(v["inv"]), v["rot"], v["inter"], ptr(v["pos"]),
                                       v["pos0"], ptr(v["Qo"]), ptr(v["Ko"]), None)


@pytest.mark.parametrize("over", [
    dict(L=-1), dict(L=1 << 31), dict(H=0), dict(H=129), dict(d=96), dict(d=0), dict(rot=-16), dict(rot=80),
    dict(rot=24), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(inter=2), dict(pos0=-1),
    dict(pos0=(1 << 31) - 5), dict(Q=None, K=None), dict(Q=0x10008), dict(K=0x20002), dict(qw=0x30008),
    dict(kw=0x30004), dict(inv=None), dict(inv=0x40002), dict(pos=0x70002), dict(qs=255), dict(qs=248),
    dict(qs=260), dict(ks=56), dict(ks=68), dict(qs=1 << 62), dict(Qo=None), dict(Ko=None), dict(Qo=0x50008),
])
def test_refusals(hsa, over):
    assert call(hsa, **over) == 1  # HSA_ERR_ARG, before anything reaches a device


def test_zero_rows_is_a_no_op(hsa):
    assert call(hsa, L=0, Q=None, K=None) == 0


def test_module_refuses_wrong_tensors(hsa):
    import torch
    with pytest.raises(ValueError):
        hsa.qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        hsa.qk_norm_rope(torch.zeros(2, 3, 64, dtype=torch.bfloat16), None)  # not on the GPU
