"""Refusals of the training entry points, on the CPU: every call below returns before any CUDA
call is reached. Also the references' own pins: the gradients the GPU tests compare with,
against differences of the losses they belong to."""
import ctypes

import numpy as np
import pytest
import torch

from training_ref import balance, balance_grad, gate_grad, swiglu_grads, topk_of

P = 0x100000  # a fake, 16-byte aligned address: never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def m():
    from combine_grouped_gemm_router_b200 import build
    build.build()
    import combine_grouped_gemm_router_b200 as mod
    return mod


def test_balance_loss_refusals(m):
    s = ctypes.byref(m.make_shape(64, 128, 256, 8, 2, 4))
    need = m.moe_balance_workspace_size(m.make_shape(64, 128, 256, 8, 2, 4))
    assert need > 0 and m.moe_balance_workspace_size(m.make_shape(64, 128, 256, 8, 9, 4)) == 0
    f = m._lib.moe_balance_loss
    ok = [s, P, P, None, 1.0, 0.0, P, P, P, P, P, need, None]

    def status(**at):
        args = list(ok)
        for k, v in at.items():
            args[int(k[1:])] = v
        return f(*args)
    for i in (1, 2, 6, 7, 8, 9):
        assert status(**{f"a{i}": None}) == 1, i
    for i in (1, 6, 8):
        assert status(**{f"a{i}": P + 4}) == 4, i      # fp32 arrays: 16 bytes
    for i in (2, 7, 9):
        assert status(**{f"a{i}": P + 2}) == 4, i
    assert status(a10=None) == 3 and status(a11=need - 1) == 3 and status(a10=P + 8) == 4
    for i in (4, 5):
        assert status(**{f"a{i}": NAN}) == 1 and status(**{f"a{i}": INF}) == 1
    assert status(a0=ctypes.byref(m.make_shape(64, 128, 256, 8, 9, 4))) == 1
    assert status(a0=ctypes.byref(m.make_shape(64, 128, 256, 512, 2, 4))) == 2
    assert status(a0=None) == 1


def test_balance_loss_backward_refusals(m):
    s = ctypes.byref(m.make_shape(64, 128, 256, 8, 2, 4))
    f = m._lib.moe_balance_loss_backward
    ok = [s, P, None, P, P, 1.0, 0.0, None, P, None]

    def status(i, v):
        args = list(ok)
        args[i] = v
        return f(*args)
    for i in (1, 3, 4, 8):
        assert status(i, None) == 1, i
    assert status(1, P + 8) == 4 and status(8, P + 4) == 4
    assert status(3, P + 1) == 4 and status(4, P + 2) == 4 and status(7, P + 2) == 4
    assert status(5, NAN) == 1 and status(6, INF) == 1
    empty = ctypes.byref(m.make_shape(0, 128, 256, 8, 2, 4))
    assert f(empty, None, None, None, None, 1.0, 0.0, None, None, None) == 0


def test_route_backward_refusals(m):
    shape = m.make_shape(64, 128, 256, 8, 2, 4)
    s, need = ctypes.byref(shape), m.moe_route_backward_workspace_size(shape)
    assert need > 0 and m.moe_route_backward_workspace_size(m.make_shape(3, 12, 0, 8, 2, 1)) == 0
    f = m._lib.moe_route_backward
    # shape, x, w_router, topk_idx, topk_w, dtopk_w, dlogits, mask, dx_add, dx, dw, dbias, ws, bytes
    Q = P + (1 << 24)
    ok = [s, P, P, P, P, P, P, None, None, Q, P, P, P, need, None]

    def status(*at):
        args = list(ok)
        for i, v in at:
            args[i] = v
        return f(*args)
    assert status((5, None), (6, None)) == 1                 # no gradient at all
    assert status((3, None)) == 1 and status((4, None)) == 1  # gate gradient without the routing
    assert status((1, None)) == 1                            # dw without x
    assert status((2, None)) == 1                            # dx without the weights
    assert status((9, None), (10, None), (11, None)) == 1    # nothing wanted
    for i in (1, 2, 6, 8, 9, 10):
        assert status((i, Q + 4 if i == 9 else P + 4)) == 4, i
    assert status((9, P)) == 1 and status((9, P + 64 * 128 * 2 - 16)) == 1   # dx over x
    for i in (3, 4, 5, 11):
        assert status((i, P + 2)) == 4, i
    assert status((12, None)) == 3 and status((13, need - 1)) == 3 and status((12, P + 8)) == 4
    assert status((0, ctypes.byref(m.make_shape(64, 100, 256, 8, 2, 4)))) == 2   # d % 8
    assert status((0, ctypes.byref(m.make_shape(64, 128, 256, 8, 33, 4)))) == 1
    assert status((0, ctypes.byref(m.make_shape((1 << 30) + 4, 128, 256, 8, 1, 4)))) == 2


def test_checkpoint_refusals(m):
    shape = m.make_shape(64, 128, 256, 8, 2, 4)
    assert m.checkpoint_stride(shape) == 2 * 256 + 16
    assert m.moe_checkpoint_bytes(shape) == m.moe_rows_alloc(shape) * 528
    assert m.checkpoint_stride(m.make_shape(64, 128, 384, 8, 2, 4)) == 768 + 32
    assert m.moe_checkpoint_bytes(m.make_shape(64, 128, 200, 8, 2, 4)) == 0
    assert m.moe_checkpoint_bytes(m.make_shape(64, 128, 0, 8, 2, 4)) == 0
    s = ctypes.byref(shape)
    up, back = m._lib.moe_expert_up_checkpoint, m._lib.moe_swiglu_backward
    for i in range(6):
        args = [P] * 6
        args[i] = None
        assert up(s, *args, None) == 1, i
        args[i] = P + 2
        assert up(s, *args, None) == 4, i
    for i in range(6):
        args = [P] * 6
        args[i] = P + 2
        assert back(s, *args, None) == 4, i
        args[i] = None
        if i < 5:                       # the recomputed h is optional
            assert back(s, *args, None) == 1, i
    assert back(ctypes.byref(m.make_shape(64, 128, 200, 8, 2, 4)), *[P] * 6, None) == 2
    assert up(ctypes.byref(m.make_shape(64, 136, 256, 8, 2, 4)), *[P] * 6, None) == 2
    empty = ctypes.byref(m.make_shape(0, 128, 256, 8, 2, 4))
    assert up(empty, *[None] * 7) == 0 and back(empty, *[None] * 7) == 0


def test_tensors_the_kernels_would_misread_are_refused(m):
    """The binding's own checks: element type, device, layout, size."""
    shape = m.make_shape(8, 128, 128, 8, 2, 1)
    f32, i32 = torch.zeros(64), torch.zeros(64, dtype=torch.int32)
    with pytest.raises(m.MoeError, match="logits is torch.float64"):
        m.moe_balance_loss(shape, f32.double(), i32, f32, i32, f32, i32)
    with pytest.raises(m.MoeError, match="logits is on cpu"):
        m.moe_balance_loss(shape, f32, i32, f32, i32, f32, i32)
    with pytest.raises(m.MoeError, match="counts is torch.int64"):
        m.moe_balance_loss_backward(shape, P, i32.long(), P, P)
    with pytest.raises(m.MoeError, match="dx is torch.bfloat16, not torch.float32"):
        m.moe_route_backward(shape, P, P, torch.zeros(8, 128, dtype=torch.bfloat16), P, dlogits=P)
    with pytest.raises(m.MoeError, match="dh is torch.float16"):
        m.moe_swiglu_backward(shape, P, P, torch.zeros(8, dtype=torch.float16), P, P)
    with pytest.raises(m.MoeError, match="h is torch.bfloat16, not torch.float16"):
        m.moe_expert_up_checkpoint(shape, P, P, P, P, torch.zeros(8, dtype=torch.bfloat16), P)


def test_references_against_differences():
    rng = np.random.default_rng(0)
    N, E, K, h = 9, 7, 3, 1e-5
    logits = rng.standard_normal((N, E))
    idx, _ = topk_of(logits, K)
    mask = (np.arange(N) != 4).astype(np.uint8)
    ref = balance(logits, idx, mask, 0.3, 0.2)
    g, _ = balance_grad(ref, E, 0.3, 0.2, 1.5)
    w = np.take_along_axis(logits, idx.astype(np.int64), 1)
    e = np.exp(w - w.max(1, keepdims=True))
    w, c = e / e.sum(1, keepdims=True), rng.standard_normal((N, K))
    dl, _ = gate_grad(idx, w, c, None, mask, N, E)

    def gates(l):
        t = np.take_along_axis(l, idx.astype(np.int64), 1)
        e = np.exp(t - t.max(1, keepdims=True))
        return ((c * e / e.sum(1, keepdims=True))[mask != 0]).sum()
    for _ in range(3):
        v = rng.standard_normal((N, E))
        up, dn = (1.5 * balance(logits + s * h * v, idx, mask, 0.3, 0.2)["loss"][0] for s in (1, -1))
        assert abs((g * v).sum() - (up - dn) / (2 * h)) < 1e-8
        assert abs((dl * v).sum() - (gates(logits + h * v) - gates(logits - h * v)) / (2 * h)) < 1e-8
    gt, ut, dh = rng.standard_normal((3, 50))
    (dg, du, hh), _ = swiglu_grads(gt, ut, dh)

    def act(g, u):
        return g / (1 + np.exp(-g)) * u
    np.testing.assert_allclose(hh, act(gt, ut), rtol=1e-12)
    np.testing.assert_allclose(dg, dh * (act(gt + h, ut) - act(gt - h, ut)) / (2 * h), atol=1e-9)
    np.testing.assert_allclose(du, dh * (act(gt, ut + h) - act(gt, ut - h)) / (2 * h), atol=1e-9)


def test_raw_workspace_address_is_refused(m):
    """Other arguments may be addresses; a workspace's size has to be known."""
    shape = m.make_shape(8, 128, 128, 8, 2, 1)
    with pytest.raises(m.MoeError, match="moe_balance_loss: ws is a raw address"):
        m.moe_balance_loss(shape, P, P, P, P, P, P, ws=P)
    with pytest.raises(m.MoeError, match="moe_route_backward: ws is a raw address"):
        m.moe_route_backward(shape, P, P, P, P, dlogits=P, ws=P)
