"""The gate/up GEMM that leaves an 8-bit checkpoint, and the activation's backward pass from it.

The checkpoint must be, bit for bit, the oracle's block code of the fp32 accumulators (which the
down GEMM, run on the same operands, gives as its fp32 y), h the plain gate/up GEMM's h, and the
backward pass the formula's values on the decoded checkpoint."""
import numpy as np
import pytest
import torch

from layer_runner import lib
from training_ref import cuda, f64, swiglu_grads

pytestmark = pytest.mark.gpu

# (name, E, rows per expert, d, f): pair tiles, ragged single tiles with an empty expert, one row,
# widths that end inside the backward pass's column blocks
CASES = [
    ("pair", 2, [1600, 900], 512, 256),
    ("ragged", 5, [1, 37, 0, 300, 129], 256, 384),
    ("one", 3, [0, 1, 0], 128, 128),
    ("wide", 2, [130, 70], 128, 1664),
]


def make(case, h_bf16=False, seed=0):
    m = lib()
    name, E, rows, d, f = case
    R = sum(rows)
    shape = m.make_shape(-(-max(R, E) // E) * E, d, f, E, 1, 1, h_bf16=h_bf16)
    RA = m.moe_rows_alloc(shape)
    g = torch.Generator().manual_seed(seed + sum(map(ord, name)))
    x = torch.randn(RA, d, generator=g) * torch.exp(torch.randn(RA, 1, generator=g))
    x[min(2, R - 1)] = 0.0   # a row of zeros: blocks of exponent 0
    w = [(torch.randn(E, f, d, generator=g) * 0.05).to(torch.bfloat16).cuda() for _ in range(2)]
    off = torch.tensor(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
    return m, shape, R, RA, x.to(torch.bfloat16).cuda(), w, off


def split(m, shape, ckpt, R):
    f, st = shape.f, m.checkpoint_stride(shape)
    rows = ckpt.cpu().numpy().reshape(-1, st)
    g, u = rows[:R, :f], rows[:R, f:2 * f]
    eg, eu = rows[:R, 2 * f:2 * f + f // 32], rows[:R, 2 * f + f // 32:2 * f + f // 16]
    return ((g, eg.astype(np.int32) - 127), (u, eu.astype(np.int32) - 127),
            rows[:R, 2 * f + f // 16:], rows[R:])


@pytest.mark.parametrize("h_bf16", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_checkpoint_is_the_block_code_of_the_accumulators(orc, case, h_bf16):
    m, shape, R, RA, x, (w1, w3), off = make(case, h_bf16)
    f, d, E = shape.f, shape.d, shape.E
    hd = torch.bfloat16 if h_bf16 else torch.float16
    h0, h1 = (torch.full((RA, f), 3.0, dtype=hd, device="cuda") for _ in range(2))
    ckpt = torch.full((m.moe_checkpoint_bytes(shape),), 0xAB, dtype=torch.uint8, device="cuda")
    assert ckpt.numel() == RA * m.checkpoint_stride(shape)
    m.moe_expert_up(shape, x, off, w1, w3, h0)
    m.moe_expert_up_checkpoint(shape, x, off, w1, w3, h1, ckpt)
    assert torch.equal(h0.view(torch.int16), h1.view(torch.int16))
    # the same products from the down GEMM: x [rows][d] as its h (bf16), W1 / W3 as its W2
    down = m.make_shape(shape.N, f, d, E, 1, 1, h_bf16=True)
    (cg, eg), (cu, eu), pad, tail = split(m, shape, ckpt, R)
    for w, codes, exps in ((w1, cg, eg), (w3, cu, eu)):
        y = torch.zeros(RA, f, dtype=torch.float32, device="cuda")
        m.moe_expert_down(down, x, off, w, y)
        want, we = orc.quantize_blocks_e4m3(y[:R].cpu().numpy())
        np.testing.assert_array_equal(exps, we)
        np.testing.assert_array_equal(codes, want)
    assert np.all(pad == 0xAB) and np.all(tail == 0xAB)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("want_h", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_backward_of_a_checkpoint(orc, case, want_h):
    """s is within 2^-20 + |g| 2^-23 relative (the fast exponential 2 ulp and its argument's
    rounding, one addition, the fast division 2 ulp); 1 - s adds s times that, the products
    6 roundings: DS = 2^-18 + |g| 2^-22 of the terms' magnitudes, then one rounding to bf16.
    Past g = -87 e^-|g| leaves fp32's normal range: s is then off by at most its smallest normal,
    2^-126, absolutely (s <= e^-|g| < 2^-126 there, whatever of it is kept), and every result is
    off by that times the factors s is multiplied with (1 + |g| for the two terms of dgate)."""
    m, shape, R, RA, x, (w1, w3), off = make(case)
    f = shape.f
    rng = np.random.default_rng(R)
    h = torch.empty(RA, f, dtype=torch.float16, device="cuda")
    ckpt = torch.full((m.moe_checkpoint_bytes(shape),), 0xAB, dtype=torch.uint8, device="cuda")
    m.moe_expert_up_checkpoint(shape, x, off, w1, w3, h, ckpt)
    check_backward(m, orc, shape, R, RA, ckpt, off, rng, want_h)


def check_backward(m, orc, shape, R, RA, ckpt, off, rng, want_h=True):
    f = shape.f
    dh = torch.from_numpy(rng.standard_normal((RA, f)) * 1e-3).to(torch.bfloat16).cuda()
    outs = [torch.full((RA, f), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    m.moe_swiglu_backward(shape, ckpt, off, dh, outs[0], outs[1], h=outs[2] if want_h else None)
    (cg, eg), (cu, eu), _, _ = split(m, shape, ckpt, R)
    g, u = orc.dequantize_blocks_e4m3(cg, eg), orc.dequantize_blocks_e4m3(cu, eu)
    with np.errstate(over="ignore"):
        want, mag = swiglu_grads(g, u, f64(dh)[:R])
    d64 = np.abs(f64(dh)[:R])
    factors = d64 * np.abs(u) * (1 + np.abs(g)), d64 * np.abs(g), np.abs(g * u)
    for got, v, size, factor in zip(outs[:3 if want_h else 2], want, mag, factors):
        rel = 2.0 ** -18 + np.abs(g) * 2.0 ** -22
        bound = rel * size + 2.0 ** -126 * factor + 1e-38
        bound = bound + 2.0 ** -8 * (np.abs(v) + bound)
        err = np.abs(f64(got)[:R] - v)
        assert np.all(err <= bound), float((err / bound).max())
    for t in outs:   # rows past the last one are left as they were
        assert torch.all(t[R:] == 5.0)
    if not want_h:
        assert torch.all(outs[2] == 5.0)
    # in place of dh
    over = dh.clone()
    m.moe_swiglu_backward(shape, ckpt, off, over, over, outs[1])
    assert torch.equal(over[:R], outs[0][:R]) and torch.equal(over[R:], dh[R:])
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("f", [128, 768, 2048])
def test_backward_of_every_code_and_far_exponents(orc, f):
    """Every finite e4m3 code in both places, exponents over the whole range that keeps the
    results in bf16's, large |g| of both signs (sigmoid at 0 and 1)."""
    m = lib()
    E, R = 2, 261
    shape = m.make_shape(262, 128, f, E, 1, 1)
    RA, st = m.moe_rows_alloc(shape), m.checkpoint_stride(shape)
    rng = np.random.default_rng(f)
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    rows = np.full((RA, st), 0xAB, np.uint8)
    rows[:, :2 * f] = rng.choice(finite, (RA, 2 * f))
    rows[:, 2 * f:2 * f + f // 32] = rng.integers(127 - 20, 127 + 12, (RA, f // 32))
    rows[:, 2 * f + f // 32:2 * f + f // 16] = rng.integers(127 - 40, 127 + 40, (RA, f // 32))
    off = torch.tensor([0, 100, R], dtype=torch.int32, device="cuda")
    check_backward(m, orc, shape, R, RA, cuda(rows.reshape(-1)), off, rng)


def test_no_rows_leaves_everything():
    m = lib()
    shape = m.make_shape(64, 128, 256, 4, 1, 1)
    RA = m.moe_rows_alloc(shape)
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    ckpt = torch.full((m.moe_checkpoint_bytes(shape),), 9, dtype=torch.uint8, device="cuda")
    outs = [torch.full((RA, 256), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    m.moe_swiglu_backward(shape, ckpt, off, *outs)
    assert all(torch.all(t == 5.0) for t in outs)
    empty = m.make_shape(0, 128, 256, 4, 1, 1)
    m.moe_swiglu_backward(empty, None, None, None, None, None)
    m.moe_expert_up_checkpoint(empty, None, None, None, None, None, None)


def test_range_pass_and_graph(orc):
    """Activations beyond fp16's range (h rescaled by the second gate/up pass): the checkpoint and
    h as without it; a captured forward and backward replays over new inputs."""
    m, shape, R, RA, x, (w1, w3), off = make(CASES[1], seed=5)
    f = shape.f
    xb = x * 64
    w1b = w1 * 16
    h0, h1 = (torch.full((RA, f), 3.0, dtype=torch.float16, device="cuda") for _ in range(2))
    ckpt = torch.full((m.moe_checkpoint_bytes(shape),), 0xAB, dtype=torch.uint8, device="cuda")
    m.moe_expert_up(shape, xb, off, w1b, w3, h0)
    m.moe_expert_up_checkpoint(shape, xb, off, w1b, w3, h1, ckpt)
    assert torch.equal(h0.view(torch.int16), h1.view(torch.int16))
    range_word = h1[RA - 1].view(torch.float32)[0].item()
    assert range_word > 65504.0, "the case does not reach the second pass"
    check_backward(m, orc, shape, R, RA, ckpt, off, np.random.default_rng(2))
    dh = torch.randn(RA, f, device="cuda").to(torch.bfloat16)
    want = [torch.zeros(RA, f, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    m.moe_swiglu_backward(shape, ckpt, off, dh, want[0], want[1], h=want[2])
    live, got = torch.zeros_like(xb), [torch.zeros_like(t) for t in want]
    ck2, h2 = torch.zeros_like(ckpt), torch.zeros_like(h1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_expert_up_checkpoint(shape, live, off, w1b, w3, h2, ck2)
        m.moe_swiglu_backward(shape, ck2, off, dh, got[0], got[1], h=got[2])
    live.copy_(xb)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert m.moe_get_device_error(True) == 0
