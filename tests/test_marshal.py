"""The compiled marshalling without a GPU: it leaves every call that is not as it should be to the Python."""
import pytest

import dense_gemm_preshuffle_amd as gp


def test_host_tensors_and_wrong_counts_are_left():
    import torch

    m = gp._compiled()
    assert m is not None, "not built"
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    assert m.norm(gp.GP_BF16, x, None, 1.0, 0, None, None, None, 1, None, None, 1e-6, True, None, None, 0, 0) is None
    assert m.norm(gp.GP_BF16, x) is None and m.norm() is None
    assert m.linear(gp.GP_BF16, x, x, None, 0, None, False, None, None, None, 0, 0) is None
    assert m.linear(gp.GP_BF16, None, None, None, 0, None, False, None, None, None, 0, 0) is None
    assert m.linear("a", "b", "c", None, 0, None, False, None, None, None, 0, 0) is None
    assert m.norm_backward(*([None] * 22)) is None and m.linear_backward(*([None] * 15)) is None
    with pytest.raises(TypeError):
        m.bind(1, 2)
