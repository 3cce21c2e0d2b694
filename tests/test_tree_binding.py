"""A missing tensor in a drafted-tree call is the library's own refusal (HSAError
with its status), as in the other calls. On the CPU: nothing reaches a device."""
import pytest

CALLS = {
    "hsa_tree_plan": ("ctx", "n", "parents", "positions", "paths"),
    "hsa_tree_step": ("ctx", "positions", "paths", "kc", "Kc", "Vc", "ks", "q", "kn", "Q", "Kn", "Vn", "O", "idx", "ws"),
    "hsa_tree_commit": ("ctx", "paths", "accepted", "kc", "Kc", "Vc", "ks"),
}
MAY_BE_NONE = {"n", "idx"}


@pytest.mark.parametrize("name,missing", [(c, t) for c, ts in CALLS.items() for t in ts if t not in MAY_BE_NONE])
def test_missing_tensor(name, missing):
    import torch
    import hierarchical_sparse_attention_hisa_b200 as hsa
    hsa.build()
    p = hsa.params(B=64, m=8, k=256, d_idx=64, H=4, d=64)
    batch, T, capacity = 2, 4, 1024
    room = hsa.hsa_tree_workspace_size(p, batch, T, capacity)
    # (any aligned memory: a call with one missing tensor is refused before the others are looked at)
    t = {n: torch.empty(room if n == "ws" else 256, dtype=torch.uint8) for n in CALLS[name]}
    t[missing] = None
    sizes = (batch, T, capacity) if name == "hsa_tree_plan" else (p, batch, T, capacity)
    with pytest.raises(hsa.HSAError) as ex:
        getattr(hsa, name)(*sizes, *[t[n] for n in CALLS[name]], 0)
    assert ex.value.status == (2 if missing == "ws" else 1)  # HSA_ERR_WORKSPACE, HSA_ERR_ARG
