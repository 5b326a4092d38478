"""One training step of the layer's router and activation as a user runs it: route -> balance loss ->
dispatch -> gate/up GEMM with the 8-bit checkpoint -> down -> combine, and back: the gradient of the
combine's weights and rows (torch), the activation's backward pass from the checkpoint, the balance
loss's gradient, the router's backward pass. Compared with torch.autograd in 64 bits over the same
selection, the layer's expert outputs taken as the GPU made them.

The router's gradients carry the roundings of dl and of the products (2^-15 of the sum of the
terms' magnitudes, see test_gpu_route_backward.py) and of the fp32 y, dtopk_w and gate weights
(2^-15 as well: sums of at most 512 terms), and the fp32 logits', which are off by
DL = d 2^-24 sum |x| |Wr| at most: a probability or a gate weight by 2 DL relative, their products
by 4 DL. The activation's gradients are
those of the 8-bit values: e4m3 is within 2^-4 of a value in its block's range (2^-10 of the
block's scale below it), so g and u are off by at most that, and the gradients by that times the
derivatives' bounds."""
import numpy as np
import pytest
import torch

from layer_runner import lib
from moe_workloads import Workload, make_layer_inputs
from training_ref import f64

pytestmark = pytest.mark.gpu

CASES = [
    Workload("step_small", N=96, d=256, f=256, E=8, K=2, W=4, s=0.6),
    Workload("step_drop", N=700, d=384, f=256, E=20, K=3, W=1, cf=1.1, s=0.8),
    Workload("step_wide", N=1040, d=512, f=128, E=72, K=6, W=8),
]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("w", CASES, ids=lambda w: w.name)
def test_step(w, captured):
    m = lib()
    dev = torch.device("cuda")
    inp = make_layer_inputs(w, seed=11)
    N, d, f, E, K = w.N, w.d, w.f, w.E, w.K
    shape = m.make_shape(N, d, f, E, K, w.W, w.cf)
    RA = m.moe_rows_alloc(shape)
    x, wr, w1, w3 = (inp[k].to(dev) for k in ("x", "w_router", "w1", "w3"))
    bias = None if inp["bias"] is None else inp["bias"].to(dev)
    w2 = m.w2_for(shape, inp["w2"].to(dev))
    g = torch.Generator(device=dev).manual_seed(4)
    dout = torch.randn(N, d, generator=g, device=dev) / N
    mask = (torch.rand(N, generator=g, device=dev) < 0.9).to(torch.uint8)
    dout[mask == 0] = 0.0   # a padded token's output reaches no loss
    cb, cz = 2e-2, 1e-3

    def new(*size, dtype=torch.float32):
        return torch.zeros(*size, dtype=dtype, device=dev)
    i32, bf = torch.int32, torch.bfloat16
    logits, topk_idx, topk_w = new(N, E), new(N, K, dtype=i32), new(N, K)
    counts, kept, offsets = new(E, dtype=i32), new(E, dtype=i32), new(E + 1, dtype=i32)
    row_of, assign = new(N * K, dtype=i32), new(RA, dtype=i32)
    xs, h, y = new(RA, d, dtype=bf), new(RA, f, dtype=torch.float16), new(RA, d)
    ckpt = new(m.moe_checkpoint_bytes(shape), dtype=torch.uint8)
    out = new(N, d)
    loss, loss_counts, mean, tokens = new(3), new(E, dtype=i32), new(E), new(1, dtype=i32)
    dh, dgate, dup, h2 = (new(RA, f, dtype=bf) for _ in range(4))
    dlogits, dtopk_w = new(N, E), new(N, K)
    dx, dwr, dbias = new(N, d), new(E, d), new(E)
    ws = new(m.moe_workspace_size(shape), dtype=torch.uint8)
    ws_b = new(m.moe_balance_workspace_size(shape), dtype=torch.uint8)
    ws_r = new(m.moe_route_backward_workspace_size(shape), dtype=torch.uint8)

    def step():
        m.moe_route(shape, x, wr, bias, topk_idx, topk_w, logits, ws)
        m.moe_balance_loss(shape, logits, topk_idx, loss, loss_counts, mean, tokens,
                           token_mask=mask, balance_coef=cb, z_coef=cz, ws=ws_b)
        m.moe_dispatch(shape, x, topk_idx, counts, kept, offsets, row_of, assign, xs, ws=ws)
        m.moe_expert_up_checkpoint(shape, xs, offsets, w1, w3, h, ckpt)
        m.moe_expert_down(shape, h, offsets, w2, y)
        m.moe_combine(shape, y, row_of, topk_w, out)
        # back through the combine: dropped slots have no row and no gradient
        row = row_of.clamp(min=0).long().view(N, K)
        live = (row_of >= 0).view(N, K)
        ys = y[row]                                                     # [N][K][d]
        torch.mul((ys * dout[:, None]).sum(2), live, out=dtopk_w)
        dy = torch.zeros(RA + 1, d, device=dev)
        dy[torch.where(live, row, RA).flatten()] = (topk_w[..., None] * dout[:, None]).flatten(0, 1)
        # dh = dy W2 of each row's expert (a library GEMM; here by expert, over every row)
        for e in range(E):
            mine = (torch.arange(RA, device=dev) >= offsets[e]) & (torch.arange(RA, device=dev)
                                                                  < offsets[e + 1])
            dh.copy_(torch.where(mine[:, None], (dy[:RA] @ w2[e].float()).to(bf), dh))
        m.moe_swiglu_backward(shape, ckpt, offsets, dh, dgate, dup, h=h2)
        m.moe_balance_loss_backward(shape, logits, loss_counts, tokens, dlogits, token_mask=mask,
                                    balance_coef=cb, z_coef=cz)
        m.moe_route_backward(shape, x, wr, dx, dwr, dbias=dbias, topk_idx=topk_idx, topk_w=topk_w,
                             dtopk_w=dtopk_w, dlogits=dlogits, token_mask=mask, ws=ws_r)

    step()
    if captured:
        eager = [t.clone() for t in (out, loss, dgate, dup, h2, dx, dwr, dbias)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (out, loss, dgate, dup, h2, dx, dwr, dbias, dh, ckpt, y):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        R = int(offsets[E].item())
        for a, b in zip((out, loss, dgate[:R], dup[:R], h2[:R], dx, dwr, dbias),
                        (*eager[:2], *(t[:R] for t in eager[2:5]), *eager[5:])):
            assert torch.equal(a, b)
        return
    torch.cuda.synchronize()
    assert m.moe_get_device_error(True) == 0
    R = int(offsets[E].item())

    # ---- the router, by autograd in 64 bits
    X, WR = x.double().requires_grad_(), wr.double().requires_grad_()
    B = (torch.zeros(E, device=dev, dtype=torch.float64) if bias is None
         else bias.double()).clone().requires_grad_()
    L = X @ WR.t() + B
    P = torch.softmax(L, 1)
    keep = mask.double()
    M = keep.sum()
    idx = topk_idx.long()
    hits = torch.zeros(E, device=dev, dtype=torch.float64).index_add_(
        0, idx.flatten(), keep.repeat_interleave(K))
    bal = E * (hits / (M * K) * (P * keep[:, None]).sum(0) / M).sum()
    z = (torch.logsumexp(L, 1).square() * keep).sum() / M
    gates = torch.softmax(L.gather(1, idx), 1)
    live = (row_of >= 0).view(N, K)
    routed = (gates[..., None] * y[row_of.clamp(min=0).long().view(N, K)].double()
              * live[..., None]).sum(1)
    total = cb * bal + cz * z + (routed * dout.double()).sum()
    total.backward()
    assert torch.equal(loss_counts.double(), hits) and tokens.item() == M.item()
    want = torch.stack([cb * bal + cz * z, bal, z]).detach()
    # fp32 sums of N terms, and the logits' DL
    DL = float(d * 2.0 ** -24 * (X.detach().abs() @ WR.detach().abs().t()).max())
    np.testing.assert_allclose(f64(loss), f64(want), rtol=2.0 ** -17 + 4 * DL)
    # the magnitudes the gradients are sums of: |dl| against |Wr| and |x|, dl's own terms included
    adl = (cb * E / M * P * (hits / (M * K) + (P * hits / (M * K)).sum(1, keepdim=True))
           + cz * 2 / M * torch.logsumexp(L, 1).abs()[:, None] * P).detach() * keep[:, None]
    dw = (y[row_of.clamp(min=0).long().view(N, K)].double() * dout.double()[:, None]).abs().sum(2)
    gate_mag = gates.detach() * (dw + (gates.detach() * dw).sum(1, keepdim=True)) * live
    adl = adl.scatter_add(1, idx, gate_mag * keep[:, None])
    for got, ref, mag in ((dx, X.grad, adl @ WR.detach().abs()),
                          (dwr, WR.grad, adl.t() @ X.detach().abs()), (dbias, B.grad, adl.sum(0))):
        bound = (2.0 ** -14 + 4 * DL) * mag + 1e-30
        err = (got.double() - ref).abs()
        assert torch.all(err <= bound), float((err / bound).max())

    # ---- the activation: g and u from the GEMM's operands, the gradients of the exact values
    exact = torch.zeros(R, f, device=dev, dtype=torch.float64)
    gx, ux = exact.clone(), exact.clone()
    bounds = offsets.tolist()
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        gx[a:b], ux[a:b] = xs[a:b].double() @ w1[e].double().t(), xs[a:b].double() @ w3[e].double().t()
    G, U = gx.clone().requires_grad_(), ux.clone().requires_grad_()
    (torch.nn.functional.silu(G) * U * dh[:R].double()).sum().backward()

    def off(v):  # a code's distance from the value it stands for
        top = v.abs().view(R, -1, 32).amax(2).repeat_interleave(32, 1)
        return v.abs() * 2.0 ** -4 + top * 2.0 ** -17 + 1e-5
    # |d/dg silu'| <= 0.5, silu' <= 1.1, |silu(a) - silu(b)| <= 1.1 |a - b|
    D = dh[:R].double().abs()
    for got, ref, b in ((dgate, G.grad, D * (off(ux) * 1.1 + (ux.abs() + off(ux)) * 0.5 * off(gx))),
                        (dup, U.grad, D * 1.1 * off(gx)),
                        (h2, torch.nn.functional.silu(gx) * ux,
                         1.1 * off(gx) * (ux.abs() + off(ux)) + (gx.abs() + off(gx)) * off(ux))):
        bound = b * 1.01 + 2.0 ** -8 * ref.abs() + 1e-30
        err = (got[:R].double() - ref).abs()
        assert torch.all(err <= bound), float((err / bound).max())
