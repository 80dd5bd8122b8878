"""What qk_backward may read of the qk_forward before it, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import build
    build.build()
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def test_a_forward_pass_that_is_refused_leaves_nothing_to_go_back_from(tp):
    import torch
    ctx = tp.QkContext(4, 8, 2, 64, torch.bfloat16, tp.RopeTable(64, device="cpu"), device="cpu")
    ctx._saved = ((), (1 << 44, 768, 512), (1 << 44, 768, 512), (None, None, None, None))  # of an earlier pass
    with pytest.raises(ValueError):
        tp.qk_forward(ctx, torch.zeros(4, 12 * 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="qk_forward"):
        tp.qk_backward(ctx, None, None)
