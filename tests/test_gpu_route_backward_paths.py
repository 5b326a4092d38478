"""The router's backward pass on the tensor cores (N E d above the little-work limit of 2^25):
what its tile plans do at the ends of their ranges, and what reaches them from a training step."""
import numpy as np
import pytest
import torch

from layer_runner import lib
from test_gpu_route_backward import call, check, inputs
from training_ref import cuda

pytestmark = pytest.mark.gpu

LITTLE_WORK = 1 << 25


def on_gpu(a):
    return {k: v if v is None else cuda(v) if isinstance(v, np.ndarray) else v.cuda()
            for k, v in a.items()}


# both forms of dx (up to 64 experts, more), bf16 and fp32, before dWr
@pytest.mark.parametrize("N,d,E,K,bf16", [(25703, 1536, 10, 4, True), (16390, 2048, 64, 6, True),
                                          (9001, 1032, 50, 3, False), (12005, 1032, 100, 3, True),
                                          (3001, 2056, 200, 8, False)])
def test_masked_batch_repeated_beside_other_traffic(N, d, E, K, bf16):
    """The whole call as a training step makes it (dx with dx_add, then dWr), over and over while
    another stream keeps the memory busy: the same bits every time, and the weight gradient's are
    those of a call that asks for no dx."""
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, K, 5, 0.05)
    g = on_gpu(a)
    out = call(m, g, E, bf16=bf16, add=True)
    check(a, E, out, bf16=bf16, add=True)
    want = {k: out[k].clone() for k in ("dx", "dw", "db")}
    alone = call(m, g, E, bf16=bf16, dx=False)
    for k in ("dw", "db"):
        assert torch.equal(alone[k], want[k]), k
    src, dst = torch.empty(2, 1 << 26, dtype=torch.uint8, device="cuda").unbind(0)
    side, same = torch.cuda.Stream(), torch.ones((), dtype=torch.bool, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for i in range(200):
        if i % 2 == 0:
            with torch.cuda.stream(side):
                dst.copy_(src)
        for k in want:
            out[k].fill_(-7.0)
        call(m, g, E, bf16=bf16, add=True, out=out)
        for k in want:
            same &= (out[k] == want[k]).all()
    torch.cuda.synchronize()
    assert same.item() and m.moe_get_device_error(True) == 0
