"""The balance loss with its counts, and its gradient, against the definitions in 64 bits, at the
expert counts where the kernels change form, with masks, -inf logits and empty batches; refusals
of wrong calls are in test_training_host.py.

Tolerances. With X = max |l - max l| of a row, the fast exponential is within 2 ulp + X 2^-24
relative (its argument l * log2(e) is rounded once: X log2(e) half-ulps, times ln 2), the row's
sum adds at most 13 roundings, the division 1 and its reciprocal 2: a probability is within
2 (2^-22 + X 2^-24) + 2^-20 <= PREL = 2^-19 + X 2^-23 relative (both terms rounded up)."""
import numpy as np
import pytest
import torch

from layer_runner import lib
from training_ref import balance, balance_grad, cuda, f64, topk_of

pytestmark = pytest.mark.gpu

# (N, E, K): every lane count of a row (E to 8, 16, 32, 64, 128, 256), with and without E % 4,
# one token, fewer tokens than a warp's rows, one block and many
SHAPES = [(1, 1, 1), (1, 8, 2), (3, 256, 8), (64, 8, 2), (33, 5, 2), (257, 16, 4), (100, 13, 3),
          (1000, 32, 1), (777, 30, 30), (513, 64, 6), (1030, 60, 6), (4099, 128, 8), (300, 96, 7),
          (2051, 160, 6), (6001, 256, 8), (1500, 255, 32), (9000, 7, 3)]


def inputs(N, E, K, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((N, E)) * spread
              - 0.7 * np.log(np.arange(E) + 1.0)).astype(np.float32)
    idx, w = topk_of(logits, K)
    return rng, logits, idx, w


def outputs(E, N=0):
    z = dict(device="cuda")
    return dict(loss=torch.full((4,), -7.0, **z), counts=torch.full((E,), -7, dtype=torch.int32, **z),
                mean=torch.full((E,), -7.0, **z), tokens=torch.full((1,), -7, dtype=torch.int32, **z),
                dlogits=torch.full((N, E), -7.0, **z))


def call(m, shape, logits, idx, o, mask=None, cb=1e-2, cz=1e-3, ws=None, stream=None):
    if ws is None:  # contents do not matter: NaN bytes
        ws = torch.full((m.moe_balance_workspace_size(shape),), 255, dtype=torch.uint8,
                        device="cuda")
    m.moe_balance_loss(shape, logits, idx, o["loss"], o["counts"], o["mean"], o["tokens"],
                       token_mask=mask, balance_coef=cb, z_coef=cz, ws=ws, stream=stream)


def rel_p(logits, keep):
    l = np.asarray(logits, np.float64)[keep]
    if not l.size:
        return 2.0 ** -19
    X = np.where(np.isfinite(l), l.max(1, keepdims=True) - l, 0.0).max()
    return 2.0 ** -19 + X * 2.0 ** -23


def check_loss(o, ref, logits, N):
    np.testing.assert_array_equal(o["counts"].cpu().numpy(), ref["counts"])
    assert o["tokens"].item() == ref["tokens"]
    # the sums: at most N roundings of a thread's fp32 sum and 64 of the warps' (all terms >= 0)
    rel = rel_p(logits, ref["keep"]) + (N + 64) * 2.0 ** -24
    got = f64(o["mean"])
    assert np.all(np.abs(got - ref["prob_mean"]) <= rel * ref["prob_mean"] + 1e-38)
    loss, lse = f64(o["loss"])[:3], ref["lse"][ref["keep"]]
    # lse = m + log s: half an ulp of the sum, 2 ulp of the logarithm, and s's relative error
    dl = 2.0 ** -24 * np.abs(lse) + 2.0 ** -22 * 8 + rel_p(logits, ref["keep"])
    bound = np.array([0.0, rel * ref["loss"][1],
                      (2 * np.abs(lse) * dl + dl ** 2).sum() / max(ref["tokens"], 1)
                      + (N + 66) * 2.0 ** -24 * ref["loss"][2]])
    bound += 2.0 ** -23 * np.abs(ref["loss"])
    bound[0] += 1e-2 * bound[1] + 1e-3 * bound[2]
    assert np.all(np.abs(loss - ref["loss"]) <= bound + 1e-38), (loss, ref["loss"], bound)
    assert o["loss"][3].item() == -7.0


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N,E,K", SHAPES)
def test_loss_and_gradient(N, E, K, masked):
    m = lib()
    rng, logits, idx, _ = inputs(N, E, K, N + E)
    mask = None
    if masked:
        mask = (rng.random(N) < 0.7).astype(np.uint8) * 3
        logits[mask == 0] = np.nan   # a padded row holds anything
        idx[mask == 0] = 1 << 30
    shape = m.make_shape(N, 128, 128, E, K, 1)
    o = outputs(E, N)
    dl, di, dm = cuda(logits), cuda(idx), cuda(mask)
    call(m, shape, dl, di, o, dm)
    ref = balance(logits, idx, mask, 1e-2, 1e-3)
    check_loss(o, ref, logits, N)
    m.moe_balance_loss_backward(shape, dl, o["counts"], o["tokens"], o["dlogits"], token_mask=dm,
                                balance_coef=1e-2, z_coef=1e-3,
                                dloss=torch.tensor([1.75], device="cuda"))
    want, mag = balance_grad(ref, E, 1e-2, 1e-3, 1.75)
    # p twice (in itself and in the inner sum, whose E products add 13 roundings), the terms'
    # own roundings, and lse's 2^-21 absolute error against b
    keep = ref["keep"]
    b = 1.75 * 1e-3 * 2 / max(ref["tokens"], 1)
    bound = (2 * rel_p(logits, keep) + 2.0 ** -19) * mag + ref["p"] * b * 2.0 ** -18
    got = f64(o["dlogits"])
    assert np.all(np.abs(got - want) <= bound + 1e-40)
    assert np.all(got[~keep] == 0.0)
    assert m.moe_get_device_error(True) == 0


def test_gradient_against_differences():
    """Along random directions, the gradient's inner product equals the central difference of
    the 64-bit loss with the counts held (error of the difference: h^2 times a third derivative
    of order 1, and 64-bit cancellation)."""
    m = lib()
    N, E, K = 40, 12, 3
    rng, logits, idx, _ = inputs(N, E, K, 5)
    mask = (np.arange(N) % 5 != 2).astype(np.uint8)
    shape = m.make_shape(N, 128, 128, E, K, 1)
    o = outputs(E, N)
    call(m, shape, cuda(logits), cuda(idx), o, cuda(mask))
    m.moe_balance_loss_backward(shape, cuda(logits), o["counts"], o["tokens"], o["dlogits"],
                                token_mask=cuda(mask), balance_coef=1e-2, z_coef=1e-3)
    got = f64(o["dlogits"])
    for _ in range(4):
        v, h = rng.standard_normal((N, E)), 1e-4
        up, dn = (balance(logits.astype(np.float64) + s * h * v, idx, mask, 1e-2, 1e-3)["loss"][0]
                  for s in (1, -1))
        diff = (up - dn) / (2 * h)
        assert abs((got * v).sum() - diff) <= 1e-5 * np.abs(got * v).sum() + 1e-10


def test_minus_infinity_is_probability_zero():
    m = lib()
    N, E, K = 70, 24, 2
    rng, logits, idx, _ = inputs(N, E, K, 9)
    logits[:, 5] = -np.inf        # an expert switched off
    logits[3, 1:] = -np.inf       # a single expert left
    idx, _ = topk_of(np.where(np.isfinite(logits), logits, -1e30), K)
    shape = m.make_shape(N, 128, 128, E, K, 1)
    o = outputs(E, N)
    call(m, shape, cuda(logits), cuda(idx), o)
    ref = balance(logits, idx, None, 1e-2, 1e-3)
    check_loss(o, ref, logits, N)
    assert o["mean"][5].item() == 0.0
    m.moe_balance_loss_backward(shape, cuda(logits), o["counts"], o["tokens"], o["dlogits"],
                                balance_coef=1e-2, z_coef=1e-3)
    got = f64(o["dlogits"])
    assert np.all(np.isfinite(got)) and np.all(got[:, 5] == 0.0)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("N,E,K,cz", [(42, 8, 2, 0.0), (42, 8, 2, 1e-3), (300, 13, 3, 0.0),
                                      (700, 160, 6, 1e-3), (20011, 64, 6, 0.0),
                                      (9001, 255, 8, 1e-3)])
def test_large_finite_logits(N, E, K, cz):
    """Experts switched off by the type's lowest value (a whole row of it included) and rows far
    from 0. Every difference to a row's maximum is exact in fp32 or so large that its probability
    is 0, so a probability is within PREL of X <= 88, or 2^-126 where it underflows. lse^2 passes
    fp32 in the rows that z_coef = 0 brings: loss[2] is inf there and loss[0] does not see it."""
    m = lib()
    rng, logits, _, _ = inputs(N, E, K, 31)
    logits = np.round(logits * 4) / 4
    kind = np.arange(N) % 7
    lowest, highest = np.finfo(np.float32).min, np.finfo(np.float32).max
    half = rng.random((N, E)) < 0.5
    half[:, 0] = False
    logits[kind == 0] -= 2.0 ** 21
    logits[kind == 1] = np.where(half, 3e9, 3e9 + 512)[kind == 1]
    logits[kind == 2] = np.where(half, lowest, logits)[kind == 2]
    logits[kind == 3] += 3.0 * 2.0 ** 20
    if cz == 0.0:
        logits[kind == 4] = lowest
        logits[kind == 5] = np.where(half, lowest, highest)[kind == 5]
        logits[kind == 6] = np.where(half, -1e30, 1e30)[kind == 6]
    logits = logits.astype(np.float32)
    idx, _ = topk_of(logits, K)
    shape = m.make_shape(N, 128, 128, E, K, 1)
    o = outputs(E, N)
    call(m, shape, cuda(logits), cuda(idx), o, cb=1e-2, cz=cz)
    m.moe_balance_loss_backward(shape, cuda(logits), o["counts"], o["tokens"], o["dlogits"],
                                balance_coef=1e-2, z_coef=cz)
    assert m.moe_get_device_error(True) == 0
    ref = balance(logits, idx, None, 1e-2, cz)
    prel = 2.0 ** -19 + 88 * 2.0 ** -23
    rel = prel + (N + 64) * 2.0 ** -24          # as in check_loss
    mean, loss = f64(o["mean"]), f64(o["loss"])
    assert np.all(np.abs(mean - ref["prob_mean"]) <= rel * ref["prob_mean"] + 2.0 ** -126)
    # lse: 2^-24 of itself from the addition and less than 2^-20 from the logarithm; squared
    want = ref["loss"].copy()
    if cz == 0.0:
        assert loss[2] == np.inf
    else:
        assert abs(loss[2] - want[2]) <= (2.0 ** -18 + rel) * want[2]
    for i in (0, 1):
        assert abs(loss[i] - want[i]) <= (2.0 ** -18 + rel) * abs(want[i])
    a, b = 1e-2 * E / N, cz * 2.0 / N
    inner = (ref["p"] @ ref["share"])[:, None]
    lse = ref["lse"][:, None]
    exact = ref["p"] * (a * (ref["share"] - inner) + b * lse)
    size = ref["p"] * (a * (ref["share"] + inner) + b * np.abs(lse))
    assert np.all(np.abs(f64(o["dlogits"]) - exact) <= size * (3 * prel + 2.0 ** -20)
                  + (a + b * np.abs(lse)) * 2.0 ** -125)


@pytest.mark.parametrize("N", [40, 5000])
def test_nothing_counted(N):
    """Every token masked, or none at all: zeros, and a zero gradient."""
    m = lib()
    E, K = 16, 2
    shape = m.make_shape(N, 128, 128, E, K, 1)
    o = outputs(E, N)
    nan = torch.full((N, E), float("nan"), device="cuda")
    idx = torch.zeros(N, K, dtype=torch.int32, device="cuda")
    mask = torch.zeros(N, dtype=torch.bool, device="cuda")
    call(m, shape, nan, idx, o, mask)
    m.moe_balance_loss_backward(shape, nan, o["counts"], o["tokens"], o["dlogits"],
                                token_mask=mask)
    assert torch.all(o["loss"][:3] == 0) and torch.all(o["counts"] == 0)
    assert torch.all(o["mean"] == 0) and o["tokens"].item() == 0
    assert torch.all(o["dlogits"] == 0)
    empty = m.make_shape(0, 128, 128, E, K, 1)
    o = outputs(E)
    m.moe_balance_loss(empty, None, None, o["loss"], o["counts"], o["mean"], o["tokens"])
    assert torch.all(o["loss"][:3] == 0) and torch.all(o["counts"] == 0)
    assert torch.all(o["mean"] == 0) and o["tokens"].item() == 0
    assert m.moe_get_device_error(True) == 0


def test_bad_values_are_flagged():
    m = lib()
    N, E, K = 90, 8, 2
    _, logits, idx, _ = inputs(N, E, K, 3)
    shape = m.make_shape(N, 128, 128, E, K, 1)
    bad = idx.copy()
    bad[7, 1], bad[50, 0] = E, -1
    o = outputs(E)
    call(m, shape, cuda(logits), cuda(bad), o)
    assert m.moe_get_device_error(True) == 8   # MOE_ERR_DEVICE_BOUNDS
    assert o["counts"].sum().item() == N * K - 2 and np.isfinite(o["loss"][0].item())
    for v in (np.nan, np.inf):
        l = logits.copy()
        l[11, 4] = v
        call(m, shape, cuda(l), cuda(idx), o)
        assert m.moe_get_device_error(True) == 7   # MOE_ERR_NONFINITE
        assert not np.isfinite(o["loss"][0].item())
    # the same expert twice in a token counts twice
    twice = idx.copy()
    twice[:, 1] = twice[:, 0]
    call(m, shape, cuda(logits), cuda(twice), o)
    np.testing.assert_array_equal(o["counts"].cpu().numpy(),
                                  np.bincount(twice.reshape(-1), minlength=E))
    assert m.moe_get_device_error(True) == 0


def test_repeats_streams_and_graphs():
    """The same bits on every run, on another stream, and from a replayed graph over new inputs;
    the gradient may be written over the logits."""
    m = lib()
    N, E, K = 20011, 64, 6
    _, logits, idx, _ = inputs(N, E, K, 21)
    shape = m.make_shape(N, 128, 128, E, K, 1)
    dl, di = cuda(logits), cuda(idx)
    runs = []
    ws = torch.full((m.moe_balance_workspace_size(shape),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o = outputs(E, N)
        call(m, shape, dl, di, o, ws=ws)
        m.moe_balance_loss_backward(shape, dl, o["counts"], o["tokens"], o["dlogits"])
        runs.append(o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = outputs(E, N)
    with torch.cuda.stream(side):
        call(m, shape, dl, di, o, ws=ws, stream=side)
        m.moe_balance_loss_backward(shape, dl, o["counts"], o["tokens"], o["dlogits"])
    side.synchronize()
    runs.append(o)
    live_l, live_i = torch.zeros_like(dl), torch.zeros_like(di)
    o = outputs(E, N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call_ws = ws
        m.moe_balance_loss(shape, live_l, live_i, o["loss"], o["counts"], o["mean"], o["tokens"],
                           balance_coef=1e-2, z_coef=1e-3, ws=call_ws)
        m.moe_balance_loss_backward(shape, live_l, o["counts"], o["tokens"], o["dlogits"])
    live_l.copy_(dl)
    live_i.copy_(di)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    runs.append(o)
    for r in runs[1:]:
        for k in r:
            assert torch.equal(r[k], runs[0][k]), k
    m.moe_balance_loss_backward(shape, live_l, o["counts"], o["tokens"], live_l)
    assert torch.equal(live_l, runs[0]["dlogits"])
