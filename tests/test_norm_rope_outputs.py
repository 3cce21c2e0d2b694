"""hsa_qk_norm_rope writes dense rows: outputs that are not, and calls in place on
rows that are not, are refused before anything is written."""
import pytest

from test_norm_rope import GOOD, call

H, D = 4, 64


@pytest.fixture(scope="module")
def hsa():
    import hierarchical_sparse_attention_hisa_b200 as m
    m.build()
    m.load()
    return m


@pytest.mark.parametrize("over", [dict(Qo=GOOD["Q"], qs=264), dict(Ko=GOOD["K"], ks=72),
                                  dict(L=2, Q=None, Ko=GOOD["K"], ks=128)])
def test_in_place_on_rows_that_are_not_dense(hsa, over):
    assert call(hsa, **over) == 1  # HSA_ERR_ARG


@pytest.mark.parametrize("over", [dict(Qo=GOOD["Q"]), dict(Ko=GOOD["K"]), dict(L=1, Qo=GOOD["Q"], qs=264)])
def test_in_place_on_dense_rows_and_one_row(hsa, over):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are no memory")
    assert call(hsa, **over) != 1  # accepted; then there is no device


def test_outputs_that_are_not_dense(hsa):
    import torch
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16)  # noqa: E731
    row = e(10, (H + 1) * D)
    Q, K = row[:, :H * D].unflatten(1, (H, D)), row[:, H * D:]
    for out in ((Q, e(10, D)), (e(10, H, D), K)):
        with pytest.raises(ValueError):
            hsa.hsa_qk_norm_rope(10, H, D, Q, K, None, None, 1e-6, None, 0, False, None, 0, *out, 0)
