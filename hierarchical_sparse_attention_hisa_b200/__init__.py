"""B200-native hierarchical indexed sparse attention (HISA).

Two-stage selection (blocks of B keys scored by their summed representative,
top-m kept with the first and the query's own block forced; then the tokens
of those blocks scored and the top-k kept) followed by exact sparse softmax
attention over the k kept tokens, shared by the H heads of a multi-query
layer. The work runs in libhsa.so (hand-written sm_100a CUDA behind a C ABI,
see include/hsa.h); this package marshals torch tensors into it.

    import hierarchical_sparse_attention_hisa_b200 as hsa
    idx = hsa.index(q_idx, k_idx, B=128, m=64, k=2048)
    O = hsa.sparse_attn(Q, K, V, idx)
"""
from __future__ import annotations

from ._lib import (EXPORTS, HSAError, hsa_block_sums, hsa_decode_step,  # noqa: F401
                   hsa_debug_inject_lost_arrival, hsa_decode_step_noalloc, hsa_device_status,
                   hsa_prefill_host,
                   hsa_prefill_host_workspace_size,
                   hsa_decode_workspace_size, hsa_index, hsa_index_workspace_size, hsa_params,
                   hsa_qk_norm_rope, hsa_select_blocks, hsa_select_tokens, hsa_sparse_attn, hsa_tree_commit,
                   hsa_tree_plan, hsa_tree_step, hsa_tree_workspace_size, kernel_launches, lib_path, load,
                   params, status_string)
from .build import build  # noqa: F401


def _check_bf16(name, t, ndim):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != ndim:
        raise ValueError(f"{name}: expected a contiguous {ndim}-d bf16 CUDA tensor")


class _On:
    """Allocations and fills of a call that runs on `stream` (None: the current one) belong to that stream.

    Made on the current stream instead, a fill would not be ordered with the call's kernels, and a workspace, given
    back when the call returns, could be handed out again while they run.
    """

    def __init__(self, stream, device):
        import torch
        self.ctx = self.caller = None
        if stream is None:
            return
        if not hasattr(stream, "cuda_stream"):  # a raw handle
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream.device != device:
            raise ValueError("the stream is not on the tensors' device")
        self.caller = torch.cuda.current_stream(device)
        self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx:
            self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self.ctx:
            self.ctx.__exit__(*exc)

    def result(self, t):
        """A tensor that the caller will use on its own current stream, too."""
        if self.ctx and t is not None:
            t.record_stream(self.caller)
        return t


def index(q_idx, k_idx, B: int, m: int, k: int, stream=None):
    """indices [Lq][k] int32 for queries at positions Lk-Lq .. Lk-1."""
    import torch
    _check_bf16("q_idx", q_idx, 2)
    _check_bf16("k_idx", k_idx, 2)
    Lq, d_idx = q_idx.shape
    Lk = k_idx.shape[0]
    p = params(B=B, m=m, k=k, d_idx=d_idx)
    with _On(stream, q_idx.device) as on:
        ws = torch.empty(max(hsa_index_workspace_size(p, Lq, Lk), 16), dtype=torch.uint8,
                         device=q_idx.device)
        out = torch.empty((Lq, k), dtype=torch.int32, device=q_idx.device)
        hsa_index(p, Lq, Lk, q_idx, k_idx, out, ws, stream)
    return on.result(out)


def sparse_attn(Q, K, V, indices, scale: float = 0.0, stream=None):
    """O [Lq][H][d] bf16 = softmax attention of Q over the indexed rows of K/V."""
    import torch
    _check_bf16("Q", Q, 3)
    _check_bf16("K", K, 2)
    _check_bf16("V", V, 2)
    Lq, H, d = Q.shape
    p = params(k=indices.shape[1], H=H, d=d, scale=scale)
    with _On(stream, Q.device) as on:
        O = torch.empty_like(Q)
        hsa_sparse_attn(p, Lq, K.shape[0], Q, K, V, indices, O, stream)
    return on.result(O)


def qk_norm_rope(Q, K, q_weight=None, k_weight=None, inv_freq=None, positions=None, pos0: int = 0,
                 eps: float = 1e-6, interleaved: bool = False, stream=None):
    """(Q [L][H][d], K [L][d]) bf16: each head RMS-normed and its first 2 * len(inv_freq) values rotated.

    Q and K may be rows of a wider projection (only a token's own values must be
    contiguous); either may be None. Row i is at positions[i] (int32) or pos0 + i.
    Rows with a negative position come back as zeros. With a stream given, the inputs must be ready on it, and
    its work must be awaited before the results are used elsewhere.
    """
    import torch
    ref = Q if Q is not None else K
    if ref is None:
        raise ValueError("Q and K are both None")
    L, d = ref.shape[0], ref.shape[-1]
    for name, t, ndim in (("Q", Q, 3), ("K", K, 2)):
        if t is not None and (t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != ndim or t.shape[0] != L
                              or t.shape[-1] != d or t.device != ref.device):
            raise ValueError(f"{name}: expected a {ndim}-d bf16 CUDA tensor of the same rows")
    for name, t, shape, dtype in (("q_weight", q_weight, (d,), torch.bfloat16),
                                  ("k_weight", k_weight, (d,), torch.bfloat16),
                                  ("inv_freq", inv_freq, None, torch.float32),
                                  ("positions", positions, (L,), torch.int32)):
        if t is not None and (t.dtype != dtype or t.device != ref.device or not t.is_contiguous() or t.dim() != 1
                              or (shape and tuple(t.shape) != shape)):
            raise ValueError(f"{name}: expected a contiguous 1-d {dtype} tensor on the same device")
    if ref.device.index != torch.cuda.current_device():
        raise ValueError("the tensors are not on the current device")
    H = Q.shape[1] if Q is not None else 1
    rot = 2 * inv_freq.numel() if inv_freq is not None else 0
    new = torch.empty if positions is None else torch.zeros
    with _On(stream, ref.device) as on:
        Qo = new((L, H, d), dtype=torch.bfloat16, device=ref.device) if Q is not None else None
        Ko = new((L, d), dtype=torch.bfloat16, device=ref.device) if K is not None else None
        if L:
            hsa_qk_norm_rope(L, H, d, Q, K, q_weight, k_weight, eps, inv_freq, rot, interleaved, positions, pos0, Qo,
                             Ko, stream)
    return on.result(Qo), on.result(Ko)
