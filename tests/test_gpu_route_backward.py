"""The router's backward pass against its formula in 64 bits, against differences, and at the
sizes where its tiles end: one token, odd token counts, d and E off the tile sizes, masks,
missing inputs and outputs, fp32 and bf16 dx.

Tolerances. dl is fp32: within DL = (K + 4) 2^-24 of the magnitude of its terms. A product dl * Wr or
dl * x keeps at least 24 bits of the fp32 factors (the fp32 outputs) or 15 (the bf16 dx, whose
own rounding is 2^-8), and a sum of n terms, accumulated in tiles of at most 128 tokens or E
columns with a truncating fp32 adder (2^-23 a step of 16 terms, at most 6 E / 16 or 24 steps)
before they are added in fp32, is within 2^-17 (fp32) or 2^-14 (bf16) of the sum of the terms'
magnitudes."""
import numpy as np
import pytest
import torch

from layer_runner import lib
from training_ref import cuda, f64, gate_grad, topk_of

pytestmark = pytest.mark.gpu


def inputs(N, d, E, K, seed, mask_share=0.0):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((N, E)).astype(np.float32)
    idx, w = topk_of(logits, K)
    a = dict(idx=idx, w=w, dw=rng.standard_normal((N, K)).astype(np.float32) * 0.1,
             dlogits=(rng.standard_normal((N, E)) * 0.01).astype(np.float32),
             x=torch.from_numpy(rng.standard_normal((N, d))).to(torch.bfloat16),
             wr=(rng.standard_normal((E, d)) / d ** 0.5).astype(np.float32),
             add=torch.from_numpy(rng.standard_normal((N, d)) * 0.1).to(torch.bfloat16), mask=None)
    if mask_share:
        keep = rng.random(N) >= mask_share
        a["mask"] = keep.astype(np.uint8)
        # a padded row holds anything
        for k in ("w", "dw", "dlogits"):
            a[k][~keep] = np.nan
        a["idx"][~keep] = -(1 << 31)
        a["x"][torch.from_numpy(~keep)] = float("nan")
    return rng, a


def call(m, a, E, bf16=False, gate=True, loss=True, add=False, dx=True, dw=True, db=True, out=None,
         stream=None):
    N, d = a["x"].shape
    K = a["idx"].shape[1]
    shape = m.make_shape(N, d, 128, E, K, 1, out_bf16=bf16)
    if out is None:
        out = dict(dx=torch.full((N, d), -7.0, dtype=torch.bfloat16 if bf16 else torch.float32,
                                 device="cuda") if dx else None,
                   dw=torch.full((E, d), -7.0, device="cuda") if dw else None,
                   db=torch.full((E,), -7.0, device="cuda") if db else None,
                   ws=torch.full((m.moe_route_backward_workspace_size(shape),), 255,
                                 dtype=torch.uint8, device="cuda"))
    g = {k: cuda(v) if isinstance(v, np.ndarray) else (None if v is None else v.cuda())
         for k, v in a.items()}
    m.moe_route_backward(shape, g["x"], g["wr"], out["dx"], out["dw"], dbias=out["db"],
                         topk_idx=g["idx"] if gate else None, topk_w=g["w"] if gate else None,
                         dtopk_w=g["dw"] if gate else None, dlogits=g["dlogits"] if loss else None,
                         token_mask=g["mask"], dx_add=g["add"] if add else None, ws=out["ws"],
                         stream=stream)
    return out


def check(a, E, out, bf16=False, gate=True, loss=True, add=False):
    N, d = a["x"].shape
    K = a["idx"].shape[1]
    dl, mag = gate_grad(a["idx"], a["w"], a["dw"] if gate else None,
                        a["dlogits"] if loss else None, a["mask"], N, E)
    keep = np.ones(N, bool) if a["mask"] is None else a["mask"] != 0
    x = np.where(keep[:, None], f64(a["x"]), 0.0)
    wr, rel = a["wr"].astype(np.float64), (K + 4) * 2.0 ** -24
    if out["dx"] is not None:
        want, size = dl @ wr, mag @ np.abs(wr)
        bound = (rel + 2.0 ** (-14 if bf16 else -17)) * size
        if add:
            want = want + f64(a["add"])
        bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -23) * (np.abs(want) + bound) + 1e-37
        err = np.abs(f64(out["dx"]) - want)
        assert np.all(err <= bound), float((err / bound).max())
    if out["dw"] is not None:
        want, size = dl.T @ x, mag.T @ np.abs(x)
        err, bound = np.abs(f64(out["dw"]) - want), (rel + 2.0 ** -17) * size + 1e-37
        assert np.all(err <= bound), float((err / bound).max())
    if out["db"] is not None:
        err = np.abs(f64(out["db"]) - dl.sum(0))
        bound = (rel + 2.0 ** -17) * mag.sum(0) + 1e-37
        assert np.all(err <= bound), float((err / bound).max())


# (N, d, E, K): one token, one expert, token counts around 64 and 128, d off 64 and 128 (d % 8
# is what is asked), E off 64, the largest E, K = 32
SHAPES = [(1, 8, 1, 1), (1, 128, 256, 8), (2, 24, 3, 2), (63, 136, 8, 2), (64, 128, 8, 2),
          (65, 64, 64, 6), (127, 120, 65, 4), (128, 256, 128, 8), (129, 264, 96, 32),
          (300, 72, 17, 5), (513, 512, 200, 8), (1111, 1000, 64, 6), (2049, 384, 130, 3),
          (700, 2048, 256, 8), (4097, 128, 40, 2),
          # the tensor-core path on narrow and ragged x, on E just past 64 and 128
          (260, 8, 3, 2), (1000, 24, 100, 4), (258, 40, 65, 1), (385, 200, 129, 3),
          (2000, 328, 64, 1), (515, 1032, 33, 32),
          # beyond the little-work path: E to 64, 128, 256, ragged in every direction
          (9001, 152, 50, 3), (5003, 264, 64, 6), (4099, 1000, 20, 2), (3001, 328, 100, 4),
          (2100, 392, 129, 5), (1500, 776, 65, 8), (1100, 1064, 193, 8), (1300, 512, 256, 4)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("N,d,E,K", SHAPES)
def test_against_the_formula(N, d, E, K, masked, bf16):
    m = lib()
    _, a = inputs(N, d, E, K, N + d + E, masked)
    add = (N + d) % 16 < 8
    out = call(m, a, E, bf16=bf16, add=add)
    check(a, E, out, bf16=bf16, add=add)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("gate,loss", [(True, False), (False, True)])
@pytest.mark.parametrize("want", ["all", "dx", "dw", "db"])
def test_inputs_and_outputs_left_out(gate, loss, want):
    m = lib()
    _, a = inputs(333, 200, 24, 3, 4, 0.1)
    sel = {k: want in ("all", k) for k in ("dx", "dw", "db")}
    out = call(m, a, 24, gate=gate, loss=loss, **sel)
    check(a, 24, out, gate=gate, loss=loss)
    assert m.moe_get_device_error(True) == 0


def test_every_token_masked():
    m = lib()
    for N in (5, 700):
        _, a = inputs(N, 136, 9, 2, 1, 0.5)
        a["mask"][:] = 0
        for k in ("w", "dw", "dlogits"):
            a[k][:] = np.nan
        a["x"][:] = float("inf")
        out = call(m, a, 9, add=True)
        assert torch.equal(out["dx"], a["add"].float().cuda())
        assert torch.all(out["dw"] == 0) and torch.all(out["db"] == 0)
        out = call(m, a, 9)
        assert torch.all(out["dx"] == 0)
    assert m.moe_get_device_error(True) == 0


def test_empty_batch_writes_zero_weight_gradients():
    m = lib()
    shape = m.make_shape(0, 128, 128, 8, 2, 1)
    dw, db = torch.full((8, 128), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    m.moe_route_backward(shape, None, None, None, dw, dbias=db)
    assert torch.all(dw == 0) and torch.all(db == 0)


def test_index_twice_and_out_of_range():
    m = lib()
    _, a = inputs(150, 128, 12, 4, 8)
    a["idx"][:, 2] = a["idx"][:, 0]   # the same expert twice in a token
    out = call(m, a, 12)
    check(a, 12, out)
    assert m.moe_get_device_error(True) == 0
    a["idx"][3, 1], a["idx"][149, 3] = 12, -1
    out = call(m, a, 12)
    check(a, 12, out)
    assert m.moe_get_device_error(True) == 8   # MOE_ERR_DEVICE_BOUNDS


def test_gate_gradient_against_differences():
    """The router as a function of its weights: loss = sum of c * gate weights + sum of g * logits;
    its gradients along random directions of x, Wr and the bias against central differences in
    64 bits (third derivatives of order 1 times h^2, against the products' magnitudes)."""
    m = lib()
    N, d, E, K = 37, 48, 10, 3
    rng, a = inputs(N, d, E, K, 12)
    x, wr, b = f64(a["x"]), a["wr"].astype(np.float64), rng.standard_normal(E) * 0.1

    def loss(x, wr, b):
        logits = x @ wr.T + b
        top = np.take_along_axis(logits, a["idx"].astype(np.int64), 1)
        e = np.exp(top - top.max(1, keepdims=True))
        return (a["dw"] * (e / e.sum(1, keepdims=True))).sum() + (a["dlogits"] * logits).sum()

    top = np.take_along_axis(x @ wr.T + b, a["idx"].astype(np.int64), 1)
    e = np.exp(top - top.max(1, keepdims=True))
    a["w"] = (e / e.sum(1, keepdims=True)).astype(np.float32)
    out = call(m, a, E)
    dx, dw, db = f64(out["dx"]), f64(out["dw"]), f64(out["db"])
    h = 1e-5
    for _ in range(4):
        vx, vw, vb = (rng.standard_normal(v.shape) for v in (x, wr, b))
        for got, v, at in ((dx, vx, 0), (dw, vw, 1), (db, vb, 2)):
            step = [(x, wr, b)[i] + (h * v if i == at else 0.0) for i in range(3)]
            back = [(x, wr, b)[i] - (h * v if i == at else 0.0) for i in range(3)]
            diff = (loss(*step) - loss(*back)) / (2 * h)
            assert abs((got * v).sum() - diff) <= 2e-5 * np.abs(got * v).sum() + 1e-9


@pytest.mark.parametrize("E,bf16", [(64, True), (200, False), (64, False), (200, True)])
def test_repeats_streams_and_graphs(E, bf16):
    """The same bits on every run, on another stream, from a graph's replay over new inputs, and
    with a bf16 dx written over dx_add."""
    m = lib()
    N, d, K = 3001, 520, 4
    _, a = inputs(N, d, E, K, 77, 0.05)
    first = call(m, a, E, bf16=bf16, add=True)
    check(a, E, first, bf16=bf16, add=True)
    runs = [call(m, a, E, bf16=bf16, add=True) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        runs.append(call(m, a, E, bf16=bf16, add=True))
    side.synchronize()
    g = {k: cuda(v) if isinstance(v, np.ndarray) else v.cuda() for k, v in a.items()}
    live = {k: torch.zeros_like(v) for k, v in g.items()}
    shape = m.make_shape(N, d, 128, E, K, 1, out_bf16=bf16)
    out = {k: torch.full_like(v, 1) for k, v in first.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_route_backward(shape, live["x"], live["wr"], out["dx"], out["dw"], dbias=out["db"],
                             topk_idx=live["idx"], topk_w=live["w"], dtopk_w=live["dw"],
                             dlogits=live["dlogits"], token_mask=live["mask"], dx_add=live["add"],
                             ws=out["ws"])
    for k in g:
        live[k].copy_(g[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    runs.append(out)
    for r in runs:
        for k in ("dx", "dw", "db"):
            assert torch.equal(r[k], first[k]), k
    if bf16:
        over = g["add"].clone()
        m.moe_route_backward(shape, g["x"], g["wr"], over, out["dw"], dbias=out["db"],
                             topk_idx=g["idx"], topk_w=g["w"], dtopk_w=g["dw"],
                             dlogits=g["dlogits"], token_mask=g["mask"], dx_add=over, ws=out["ws"])
        assert torch.equal(over, first["dx"])
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("N,d,E,K", [(25703, 1536, 10, 4), (16390, 2048, 64, 6),
                                     (12005, 1032, 100, 3)])
def test_masked_rows_beside_other_traffic(N, d, E, K):
    """Copies of x that land late and out of order (another stream keeps the memory busy) change
    no bit of the weight gradient of a masked batch."""
    m = lib()
    _, a = inputs(N, d, E, K, 5, 0.05)
    g = {k: v if v is None else cuda(v) if isinstance(v, np.ndarray) else v.cuda()
         for k, v in a.items()}
    out = call(m, g, E, bf16=True, dx=False)
    check(a, E, dict(out, dx=None))
    want = {k: out[k].clone() for k in ("dw", "db")}
    src, dst = torch.empty(2, 1 << 26, dtype=torch.uint8, device="cuda").unbind(0)
    side, same = torch.cuda.Stream(), torch.ones((), dtype=torch.bool, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for i in range(400):
        if i % 2 == 0:
            with torch.cuda.stream(side):
                dst.copy_(src)
        call(m, g, E, bf16=True, dx=False, out=out)
        for k in want:
            same &= (out[k] == want[k]).all()
    torch.cuda.synchronize()
    assert same.item() and m.moe_get_device_error(True) == 0


def test_dx_over_x_is_refused():
    m = lib()
    shape = m.make_shape(300, 64, 128, 8, 2, 1, out_bf16=True)
    x = torch.zeros(300, 64, dtype=torch.bfloat16, device="cuda")
    wr = torch.zeros(8, 64, device="cuda")
    dl = torch.zeros(300, 8, device="cuda")
    ws = torch.empty(m.moe_route_backward_workspace_size(shape), dtype=torch.uint8, device="cuda")
    with pytest.raises(m.MoeError, match="INVALID_ARG"):
        m.moe_route_backward(shape, x, wr, x, torch.zeros_like(wr), dlogits=dl, ws=ws)
    m.moe_route_backward(shape, x, wr, x, None, dlogits=dl, ws=ws)   # x is not read then


FIRST_CALL = """
import torch, combine_grouped_gemm_router_b200 as m
N, d, E, K = 700, 256, {E}, 2
sh = m.make_shape(N, d, 128, E, K, 1)
z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
x, wr, dl = torch.ones(N, d, device="cuda", dtype=torch.bfloat16), z(E, d), torch.ones(N, E, device="cuda")
idx, counts, tok = z(N, K, dtype=torch.int32), z(E, dtype=torch.int32), z(1, dtype=torch.int32)
dx, dw, db, loss, mean = z(N, d), z(E, d), z(E), z(3), z(E)
ws = torch.empty(m.moe_route_backward_workspace_size(sh) + m.moe_balance_workspace_size(sh),
                 dtype=torch.uint8, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    m.moe_balance_loss(sh, dl, idx, loss, counts, mean, tok, ws=ws)
    m.moe_route_backward(sh, x, wr, dx, dw, dbias=db, dlogits=dl, ws=ws)
g.replay()
torch.cuda.synchronize()
assert torch.all(dw == N) and torch.all(db == N) and tok.item() == N and counts[0].item() == N * K
print("ok")
"""


@pytest.mark.parametrize("E", [16, 200])
def test_first_call_of_a_process_may_be_captured(E):
    """The one-time setup of the kernels (shared-memory limits, resident pairs) does not need an
    eager call before a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(E=E)], cwd=root, timeout=120,
                       capture_output=True, text=True)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-800:]
