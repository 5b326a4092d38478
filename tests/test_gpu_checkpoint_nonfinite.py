"""The 8-bit checkpoint of pre-activations that overflowed or are NaN: their gradients must not
come back finite, and the finite values beside them keep their codes."""
import numpy as np
import pytest
import torch

from test_gpu_checkpoint import CASES, make, split
from training_ref import f64

pytestmark = pytest.mark.gpu

F16_RANGE = 9   # MOE_ERR_F16_RANGE


def nonfinite_inputs(case, h_bf16):
    """g is +-inf in some columns of one row, u in some of another; a third row is NaN. Column 0 of
    x and of the weights is 0 but for them."""
    m, shape, R, RA, x, (w1, w3), off = make(case, h_bf16)
    x[:, 0] = 0.0
    w1[..., 0] = 0.0
    w3[..., 0] = 0.0
    g = torch.Generator().manual_seed(7)
    hit = torch.rand(2, shape.f, generator=g)
    sign = torch.where(torch.rand(2, shape.f, generator=g) < 0.5, -1.0, 1.0)
    hit[:, 64:96] = 0.0   # a block of nothing else
    big = torch.where(hit < 0.1, sign * 2.0 ** 10, torch.zeros(())).to(torch.bfloat16).cuda()
    w1[..., 0], w3[..., 1] = big[0], big[1]
    w1[..., 1] = 0.0
    x[:, 1] = 0.0
    x[0, 0] = 2.0 ** 120              # times +-2^10: beyond fp32
    x[R - 1, 1] = 2.0 ** 120
    if R > 4:
        x[R // 2, 2] = float("nan")
    return m, shape, R, RA, x, w1, w3, off


@pytest.mark.parametrize("h_bf16", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_nonfinite_pre_activations_stay_nonfinite(orc, case, h_bf16):
    m, shape, R, RA, x, w1, w3, off = nonfinite_inputs(case, h_bf16)
    f, d, E = shape.f, shape.d, shape.E
    hd = torch.bfloat16 if h_bf16 else torch.float16
    h0, h1 = (torch.full((RA, f), 3.0, dtype=hd, device="cuda") for _ in range(2))
    ckpt = torch.full((m.moe_checkpoint_bytes(shape),), 0xAB, dtype=torch.uint8, device="cuda")
    m.moe_expert_up(shape, x, off, w1, w3, h0)
    m.moe_expert_up_checkpoint(shape, x, off, w1, w3, h1, ckpt)
    assert torch.equal(h0.view(torch.int16)[:R], h1.view(torch.int16)[:R])
    assert m.moe_get_device_error(True) == (0 if h_bf16 else F16_RANGE)
    down = m.make_shape(shape.N, f, d, E, 1, 1, h_bf16=True)
    (cg, eg), (cu, eu), pad, tail = split(m, shape, ckpt, R)
    bad = []
    for w, codes, exps in ((w1, cg, eg), (w3, cu, eu)):
        y = torch.zeros(RA, f, dtype=torch.float32, device="cuda")
        m.moe_expert_down(down, x, off, w, y)
        y = y[:R].cpu().numpy()
        bad.append(~np.isfinite(y))
        assert bad[-1].any() and not bad[-1].all()
        want, we = orc.quantize_blocks_e4m3(np.where(bad[-1], np.float32(0.0), y))
        np.testing.assert_array_equal(exps, we)
        np.testing.assert_array_equal(codes[~bad[-1]], want[~bad[-1]])
        assert np.all(codes[bad[-1]] & 0x7F == 0x7F)   # e4m3's NaN
    assert np.all(pad == 0xAB) and np.all(tail == 0xAB)
    m.moe_get_device_error(True)
    dh = torch.full((RA, f), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    outs = [torch.full((RA, f), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    m.moe_swiglu_backward(shape, ckpt, off, dh, outs[0], outs[1], h=outs[2])
    either = bad[0] | bad[1]
    for t, lost in zip(outs, (either, bad[0], either)):
        np.testing.assert_array_equal(np.isfinite(f64(t)[:R]), ~lost)
    assert m.moe_get_device_error(True) == 0
