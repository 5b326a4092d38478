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
    drops out of dx, but not the error made in its products. fp32 dx: six products of bf16 terms,
    of which at most two steps of 16 experts hold something other than 0, so at most 12 truncated
    additions (2^-23 of at most the terms' magnitudes each), with 2^-24 left out; bf16 dx: three
    products of fp16 terms, 6 truncated additions, with 3 x 2^-22 left out (of each factor, and
    the product of the small terms). Either is below 2^-19 of the magnitudes, beside the output's
    rounding. A factor cut to its first two bf16 terms is off by up to 2^-17 of them."""
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
    columns of very different size: a factor of a bf16 dx is within 2^-22 of itself or 2^-39 of the
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


# narrow x: one column box (d = 8, 64), two (72, 128), a slice's last one alone (264); with two boxes at
# most, a pair's second CTA has columns past d only, or the odd warps no piece at all
NARROW = [(1 << 20, 8, 5, 2), (70001, 8, 64, 6), (14001, 64, 40, 4), (150007, 72, 4, 1),
          (5003, 128, 64, 6), (17001, 8, 256, 8), (40003, 8, 107, 3), (6001, 64, 100, 8),
          (4501, 72, 130, 5), (2049, 128, 200, 8), (3001, 264, 65, 4)]


@pytest.mark.parametrize("masked", [0.0, 0.2])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,d,E,K", NARROW)
def test_narrow_hidden_states(N, d, E, K, bf16, masked):
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, K, N + d, masked)
    add = masked > 0
    out = call(m, a, E, bf16=bf16, add=add)
    check(a, E, out, bf16=bf16, add=add)
    assert m.moe_get_device_error(True) == 0


# few tokens over very wide x: more column slices than SMs, one short token tile
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,d,E,K", [(1, 140040, 256, 8), (3, 262208, 64, 2), (9, 65544, 129, 4)])
def test_few_tokens_over_wide_hidden_states(N, d, E, K, bf16):
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, K, N)
    out = call(m, a, E, bf16=bf16, add=True)
    check(a, E, out, bf16=bf16, add=True)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("gate,loss", [(True, False), (False, True)])
@pytest.mark.parametrize("want", ["all", "dx", "dw", "db"])
@pytest.mark.parametrize("N,d,E,bf16", [(3001, 520, 24, True), (1501, 264, 100, True),
                                        (1501, 264, 100, False)])
def test_outputs_left_out(N, d, E, bf16, want, gate, loss):
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, 3, 4, 0.1)
    sel = {k: want in ("all", k) for k in ("dx", "dw", "db")}
    out = call(m, a, E, bf16=bf16, gate=gate, loss=loss, **sel)
    check(a, E, out, bf16=bf16, gate=gate, loss=loss)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,d,E", [(3001, 520, 24), (1501, 264, 100)])
def test_wholly_masked_batch(N, d, E, bf16):
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, 2, 1, 0.5)
    a["mask"][:] = 0
    for k in ("w", "dw", "dlogits"):
        a[k][:] = np.nan
    a["x"][:] = float("inf")
    for add in (True, False):
        out = call(m, a, E, bf16=bf16, add=add)
        want = a["add"].to(out["dx"].dtype).cuda() if add else torch.zeros_like(out["dx"])
        assert torch.equal(out["dx"], want)
        assert torch.all(out["dw"] == 0) and torch.all(out["db"] == 0)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,d,E", [(3001, 1032, 12), (1501, 264, 100)])
def test_index_twice_and_out_of_range(N, d, E, bf16):
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, 4, 8)
    a["idx"][:, 2] = a["idx"][:, 0]   # the same expert twice in a token
    check(a, E, call(m, a, E, bf16=bf16), bf16=bf16)
    assert m.moe_get_device_error(True) == 0
    a["idx"][3, 1], a["idx"][N - 1, 3] = E, -1
    check(a, E, call(m, a, E, bf16=bf16), bf16=bf16)
    assert m.moe_get_device_error(True) == 8   # MOE_ERR_DEVICE_BOUNDS


def full_mantissa(rng, *size):
    """fp32 values that use all 24 bits, of both signs, over a few binades."""
    v = rng.uniform(1.0, 2.0, size) * 2.0 ** rng.integers(-4, 5, size)
    return (v * rng.choice([-1.0, 1.0], size)).astype(np.float32)


@pytest.mark.parametrize("N,d,E", [(1500, 512, 64), (9001, 264, 20), (2100, 392, 129),
                                   (1300, 264, 100), (700, 1032, 200)])
def test_every_term_of_a_product_counts(N, d, E):
    """One expert per token: an element of dx is one product, all of it: 6 products of bf16 terms or
    3 of fp16 terms (as many truncated additions, 2^-23 of the result each) and 2^-24 or 3 x 2^-22
    left out, 2^-19 of the value. A factor without its third bf16 term is off by up to 2^-17, a
    product without mid x mid by up to 2^-16. One token per expert: an element of dWr is one product of dl
    (three terms, two additions truncated and one rounded) and an exact bf16: 2^-21; without the
    third term up to 2^-17."""
    m = lib()
    assert N * d * E > LITTLE_WORK
    rng, a = inputs(N, d, E, 1, E)
    a["wr"] = full_mantissa(rng, E, d)
    e, v = rng.integers(0, E, N), full_mantissa(rng, N)
    a["dlogits"][:] = 0.0
    a["dlogits"][np.arange(N), e] = v
    want = v[:, None].astype(np.float64) * a["wr"].astype(np.float64)[e]
    for bf16 in (False, True):
        out = call(m, a, E, bf16=bf16, gate=False, dw=False)
        err = np.abs(out["dx"].double().cpu().numpy() - want)
        bound = (2.0 ** -19 + (2.0 ** -8 if bf16 else 2.0 ** -23)) * np.abs(want)
        assert np.all(err <= bound), float((err / bound).max())
    t, v = rng.permutation(N)[:E], full_mantissa(rng, E)
    a["dlogits"][:] = 0.0
    a["dlogits"][t, np.arange(E)] = v
    out = call(m, a, E, gate=False, dx=False)
    x = a["x"].double().numpy()[t]
    want = v[:, None].astype(np.float64) * x
    err = np.abs(out["dw"].double().cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -21 * np.abs(want)), float((err / np.abs(want)).max())
    assert np.array_equal(out["db"].cpu().numpy(), v)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("N,d,E", [(300_000, 4096, 8), (150_000, 4096, 72)])
def test_long_sums_of_one_sign(N, d, E):
    """All terms positive, so that truncated additions add up. A sum leaves the tensor core after
    128 tokens (24 truncated additions of at most 2^-23 of that sum) and is added in fp32 in at
    most N / 128 rounded steps over all blocks: 24 2^-23 + (N / 128) 2^-24 / 9 parts for what one
    block adds, and 18 for their sum; kept in the tensor core the N / 9 / 16 steps of a block would
    lose half of 2^-24 each."""
    m = lib()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(N, d, device="cuda", dtype=torch.bfloat16).uniform_(0.5, 1.5, generator=g)
    dl = torch.rand(N, E, generator=g, device="cuda") + 0.5
    shape = m.make_shape(N, d, 128, E, 1, 1)
    dw = torch.empty(E, d, device="cuda")
    ws = torch.empty(m.moe_route_backward_workspace_size(shape), dtype=torch.uint8, device="cuda")
    m.moe_route_backward(shape, x, None, None, dw, dlogits=dl, ws=ws)
    want = torch.zeros(E, d, device="cuda", dtype=torch.float64)
    for a in range(0, N, 1 << 15):
        want += dl[a:a + (1 << 15)].double().t() @ x[a:a + (1 << 15)].double()
    bound = 24 * 2.0 ** -23 + (N / 128 / 9 + 1 + 18) * 2.0 ** -24
    err = ((dw.double() - want) / want).abs().max().item()
    assert err <= bound, (err, bound)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,d,E", [(1500, 512, 64), (9001, 264, 20), (1300, 264, 100)])
def test_largest_gradients(N, d, E):
    """dl next to fp32's largest value (it rounds past the largest bf16, so its terms are cut, not
    rounded): one product per output, 2^-19 of it as above and 2^-126 where a term leaves fp32's
    normal range."""
    m = lib()
    assert N * d * E > LITTLE_WORK
    rng, a = inputs(N, d, E, 1, 2)
    big = np.float32(np.finfo(np.float32).max)
    a["dlogits"][:] = 0.0
    e = rng.integers(0, E, N)
    v = np.where(rng.random(N) < 0.5, big, -np.nextafter(big, np.float32(0)))
    v = np.where(rng.random(N) < 0.2, np.float32(3.3895314e38), v).astype(np.float32)  # bf16's largest
    a["dlogits"][np.arange(N), e] = v
    a["wr"] = (full_mantissa(rng, E, d) * 2.0 ** -20).astype(np.float32)
    want = v[:, None].astype(np.float64) * a["wr"].astype(np.float64)[e]
    for bf16 in (False, True):
        out = call(m, a, E, bf16=bf16, gate=False, dw=False, db=False)
        err = np.abs(out["dx"].double().cpu().numpy() - want)
        bound = (2.0 ** -19 + (2.0 ** -8 if bf16 else 2.0 ** -23)) * np.abs(want) + 2.0 ** -126
        assert np.all(err <= bound), float((err / bound).max())
    # dWr: the first E tokens, one expert each, x small
    a["dlogits"][:] = 0.0
    a["dlogits"][np.arange(E), np.arange(E)] = v[:E]
    a["x"] = (a["x"].float() * 2.0 ** -20).to(torch.bfloat16)
    out = call(m, a, E, gate=False, dx=False, db=False)
    want = v[:E, None].astype(np.float64) * a["x"].double().numpy()[:E]
    err = np.abs(out["dw"].double().cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -21 * np.abs(want) + 2.0 ** -126)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N,d,E", [(3001, 520, 24), (1501, 264, 100)])
def test_nonfinite_inputs_show_where_they_enter(N, d, E, value, bf16):
    """A non-finite gradient makes its token's dx and its expert's row of dWr and dbias non-finite, a
    non-finite weight its column of dx, a non-finite hidden state its column of dWr; the rest is
    as without them, within twice an output's own bound (the terms of a value's neighbours are cut
    instead of rounded)."""
    m = lib()
    assert N * d * E > LITTLE_WORK
    _, a = inputs(N, d, E, 2, 6)
    t, e, c = N - 7, E - 2, d - 3
    clean = call(m, a, E, bf16=bf16, gate=False)
    g = {k: torch.from_numpy(a[k]).double().abs() for k in ("dlogits", "wr")}
    size = dict(dx=g["dlogits"] @ g["wr"], dw=g["dlogits"].t() @ a["x"].double().abs(),
                db=g["dlogits"].sum(0))

    def same_but(out, key, lost):
        got, want = out[key].double(), clean[key].double()
        assert not torch.isfinite(got[lost]).any()
        bound = 2.0 ** -16 * size[key].cuda()
        if key == "dx" and bf16:
            bound = bound + 2.0 ** -7 * (want.abs() + bound)
        assert torch.all(((got - want).abs() <= bound)[~lost])

    def nothing(key):
        return torch.zeros_like(clean[key], dtype=torch.bool)
    b = dict(a, dlogits=a["dlogits"].copy())
    b["dlogits"][t, e] = value
    out = call(m, b, E, bf16=bf16, gate=False)
    row, dw, db = nothing("dx"), nothing("dw"), nothing("db")
    row[t], dw[e], db[e] = True, True, True
    same_but(out, "dx", row), same_but(out, "dw", dw), same_but(out, "db", db)
    b = dict(a, wr=a["wr"].copy())
    b["wr"][e, c] = value
    out = call(m, b, E, bf16=bf16, gate=False)
    col = nothing("dx")
    col[:, c] = True
    same_but(out, "dx", col), same_but(out, "dw", nothing("dw"))
    b = dict(a, x=a["x"].clone())
    b["x"][t, c] = value
    out = call(m, b, E, bf16=bf16, gate=False)
    col = nothing("dw")
    col[:, c] = True
    same_but(out, "dw", col), same_but(out, "dx", nothing("dx"))
    assert m.moe_get_device_error(True) == 0
