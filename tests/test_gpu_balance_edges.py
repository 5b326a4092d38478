"""The balance loss's gradient where the header promises a value whatever the inputs hold."""
import numpy as np
import pytest
import torch

from layer_runner import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,E", [(40, 16), (5000, 30), (700, 200)])
@pytest.mark.parametrize("dloss", [1.0, float("inf"), float("nan")])
def test_no_counted_tokens_no_gradient(N, E, dloss):
    """*tokens = 0 writes zeros everywhere, without a token_mask too (a job whose masked batches
    add up to nothing), whatever the logits and dloss hold."""
    m = lib()
    shape = m.make_shape(N, 128, 128, E, 2, 1)
    logits = torch.randn(N, E, device="cuda")
    logits[3], logits[7, 1], logits[9, 2] = float("nan"), float("inf"), -float("inf")
    counts, tokens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E, 1))
    out = torch.full((N, E), -7.0, device="cuda")
    m.moe_balance_loss_backward(shape, logits, counts, tokens, out, balance_coef=1e-2, z_coef=1e-3,
                                dloss=torch.tensor([dloss], device="cuda"))
    assert torch.all(out == 0)
    assert m.moe_get_device_error(True) == 0
