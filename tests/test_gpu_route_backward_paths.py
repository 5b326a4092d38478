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


def pair_gradients(N, d, E, seed):
    """Router weights of a row common to all experts plus 2^-12 of it of their own, and a token's
    gradient v on one expert and -v on another: dx is the small difference of two large products.
    v, the common row and the sum use all 24 bits of fp32."""
    rng, a = inputs(N, d, E, 1, seed)
    common = rng.uniform(1.0, 2.0, (1, d)) * rng.choice([-1.0, 1.0], (1, d))
    a["wr"] = (common * (1.0 + 2.0 ** -12 * rng.standard_normal((E, d)))).astype(np.float32)
    v = (rng.uniform(1.0, 2.0, N) * 2.0 ** rng.integers(-12, 3, N)).astype(np.float32)
    e = np.argsort(rng.random((N, E)), 1)[:, :2]
    a["dlogits"][:] = 0.0
    a["dlogits"][np.arange(N), e[:, 0]] = v
    a["dlogits"][np.arange(N), e[:, 1]] = -v
    return a


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N,d,E", [(1500, 512, 64), (9001, 264, 20), (1700, 520, 40),
                                   (2100, 392, 129), (1300, 264, 100), (700, 1032, 200)])
def test_dx_of_cancelling_products(N, d, E, bf16):
    """dl's entries sum to 0 in a softmax's backward pass, so what all rows of Wr have in common
    drops out of dx, but not the error made in its products. Both terms of an output need 24 bits
    of each factor: six products of bf16 terms, of which at most two steps of 16 experts hold
    something other than 0, so at most 12 truncated additions (2^-23 of at most the terms'
    magnitudes each), with 2^-25 left out: 2^-19 of the magnitudes, beside the output's rounding. A
    factor cut to its first two bf16 terms is off by up to 2^-17 of them."""
    m = lib()
    assert N * d * E > LITTLE_WORK
    a = pair_gradients(N, d, E, E)
    out = call(m, a, E, bf16=bf16, gate=False, dw=False, db=False)
    dl, wr = a["dlogits"].astype(np.float64), a["wr"].astype(np.float64)
    want, size = dl @ wr, np.abs(dl) @ np.abs(wr)
    bound = 2.0 ** -19 * size
    bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -23) * (np.abs(want) + bound)
    err = np.abs(out["dx"].double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / bound).max())
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("N,d,E,bf16", [(4099, 328, 40, True), (1100, 520, 72, True),
                                        (700, 264, 256, True), (4099, 328, 40, False)])
def test_dx_of_far_ranges(N, d, E, bf16):
    """Gradients and weights over 45 binades within a token and within 64 columns, tokens and
    columns of very different size: a factor of a bf16 dx is within 2^-23 of itself or 2^-39 of the
    largest of its token (dl) or its 64 columns (Wr), beside the 2^-17 of the terms that the
    accumulation may lose; results below fp32's normal range may be 0."""
    m = lib()
    rng, a = inputs(N, d, E, 1, 3)
    dl = rng.standard_normal((N, E)) * 2.0 ** -rng.uniform(0, 45, (N, E))
    dl *= 2.0 ** rng.choice([-75.0, 0.0, 80.0], (N, 1))
    wr = rng.standard_normal((E, d)) * 2.0 ** -rng.uniform(0, 45, (E, d))
    wr *= np.repeat(2.0 ** rng.choice([-30.0, 0.0, 30.0], -(-d // 64)), 64)[:d]
    a["dlogits"], a["wr"] = dl.astype(np.float32), wr.astype(np.float32)
    a["dlogits"][5] = 0.0
    out = call(m, a, E, bf16=bf16, gate=False, dw=False, db=False)
    dl, wr = a["dlogits"].astype(np.float64), a["wr"].astype(np.float64)
    want, size = dl @ wr, np.abs(dl) @ np.abs(wr)
    bound = 2.0 ** -17 * size + 2.0 ** -126
    if bf16:
        top = np.maximum.reduceat(np.abs(wr).max(0), np.arange(0, d, 64)).repeat(64)[:d]
        bound += 2.0 ** -38 * (np.abs(dl).max(1, keepdims=True) * np.abs(wr).sum(0)
                               + np.abs(dl).sum(1, keepdims=True) * top)
    bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -23) * (np.abs(want) + bound)
    err = np.abs(out["dx"].double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / bound).max())
    assert torch.all(out["dx"][5] == 0)
    assert m.moe_get_device_error(True) == 0
