"""The training operators where element offsets pass 32 bits (more than 2^32 bytes and 2^31
elements), and two calls at once on two streams. References are 64-bit torch operations on the GPU, chunk by
chunk; the tolerances are those of the operators' own tests (test_gpu_balance.py,
test_gpu_route_backward.py, test_gpu_checkpoint.py)."""
import numpy as np
import pytest
import torch

from layer_runner import lib
from test_gpu_route_backward import call, check, inputs
from training_ref import f64, swiglu_grads

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_balance_over_many_tokens():
    m = lib()
    N, E, K = 8_500_001, 256, 2     # 2.18e9 logits
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.empty(N, E, device="cuda").normal_(0.0, 1.5, generator=g)
    idx = torch.randint(0, E, (N, K), generator=g, device="cuda", dtype=torch.int32)
    mask = (torch.rand(N, generator=g, device="cuda") < 0.9).to(torch.uint8)
    shape = m.make_shape(N, 128, 128, E, K, 1)
    loss, mean = torch.zeros(3, device="cuda"), torch.zeros(E, device="cuda")
    counts, tok = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E, 1))
    ws = torch.empty(m.moe_balance_workspace_size(shape), dtype=torch.uint8, device="cuda")
    m.moe_balance_loss(shape, logits, idx, loss, counts, mean, tok, token_mask=mask,
                       balance_coef=0.5, z_coef=0.25, ws=ws)
    M = int(mask.sum())
    hits = torch.bincount(idx[mask.bool()].flatten(), minlength=E)
    p_sum, z_sum = torch.zeros(E, device="cuda", dtype=torch.float64), 0.0
    for a in range(0, N, 1 << 20):
        l = logits[a:a + (1 << 20)][mask[a:a + (1 << 20)].bool()].double()
        p_sum += torch.softmax(l, 1).sum(0)
        z_sum += float(torch.logsumexp(l, 1).square().sum())
    bal = E * float((hits / (M * K)).double() @ p_sum) / M
    want = np.array([0.5 * bal + 0.25 * z_sum / M, bal, z_sum / M])
    assert tok.item() == M and torch.equal(counts.long(), hits)
    # a thread adds about N / 9472 rows: (900 + 64) 2^-24, and PREL with X below 20
    rel = 2.0 ** -19 + 20 * 2.0 ** -23 + 964 * 2.0 ** -24
    assert np.all(np.abs(f64(loss) - want) <= rel * np.abs(want))
    assert torch.all((mean.double() - p_sum / M).abs() <= rel * p_sum / M)
    dl = torch.empty_like(logits)
    m.moe_balance_loss_backward(shape, logits, counts, tok, dl, token_mask=mask, balance_coef=0.5,
                                z_coef=0.25)
    share = (hits / (M * K)).double()
    for a in (0, N // 2, N - 1000):
        l, keep = logits[a:a + 1000].double(), mask[a:a + 1000].double()[:, None]
        p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)[:, None]
        inner = (p * share).sum(1, keepdim=True)
        ref = p * (0.5 * E / M * (share - inner) + 0.5 / M * lse) * keep
        mag = p * (0.5 * E / M * (share + inner) + 0.5 / M * lse.abs())
        bound = (2 * (2.0 ** -19 + 20 * 2.0 ** -23) + 2.0 ** -19) * mag + p * 0.5 / M * 2.0 ** -18
        assert torch.all((dl[a:a + 1000].double() - ref).abs() <= bound + 1e-40)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("E,bf16", [(8, True), (72, False)])
def test_route_backward_over_many_tokens(E, bf16):
    m = lib()
    N, d = 600_011, 4096            # 2.46e9 hidden values
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(N, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    dl = torch.randn(N, E, generator=g, device="cuda")
    wr = torch.randn(E, d, generator=g, device="cuda") / 64
    shape = m.make_shape(N, d, 128, E, 1, 1, out_bf16=bf16)
    dx = torch.empty(N, d, device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    dw, db = torch.empty(E, d, device="cuda"), torch.empty(E, device="cuda")
    ws = torch.empty(m.moe_route_backward_workspace_size(shape), dtype=torch.uint8, device="cuda")
    m.moe_route_backward(shape, x, wr, dx, dw, dbias=db, dlogits=dl, ws=ws)
    ref, mag = (torch.zeros(E, d, device="cuda", dtype=torch.float64) for _ in range(2))
    for a in range(0, N, 1 << 15):
        xs, ds = x[a:a + (1 << 15)].double(), dl[a:a + (1 << 15)].double()
        ref += ds.t() @ xs
        mag += ds.abs().t() @ xs.abs()
    assert torch.all((dw.double() - ref).abs() <= 2.0 ** -17 * mag)
    assert torch.all((db.double() - dl.double().sum(0)).abs() <= 2.0 ** -17 * dl.double().abs().sum(0))
    for a in (0, N // 2, N - 300):
        want = dl[a:a + 300].double() @ wr.double()
        size = dl[a:a + 300].double().abs() @ wr.double().abs()
        bound = 2.0 ** (-14 if bf16 else -17) * size
        bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -23) * (want.abs() + bound)
        assert torch.all((dx[a:a + 300].double() - want).abs() <= bound)
    assert m.moe_get_device_error(True) == 0


def test_activation_backward_over_many_rows(orc):
    m = lib()
    R, f = 1_420_003, 1536          # 2.18e9 values of each array
    shape = m.make_shape(R, 128, f, 1, 1, 1)
    RA, st = m.moe_rows_alloc(shape), m.checkpoint_stride(shape)
    g = torch.Generator(device="cuda").manual_seed(3)
    ckpt = torch.randint(0, 120, (RA, st), generator=g, device="cuda", dtype=torch.uint8)
    dh = torch.empty(RA, f, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    outs = [torch.full((RA, f), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    ckpt[:, 2 * f:] = ckpt[:, 2 * f:] % 16 + 110   # exponents -17 .. -2
    m.moe_swiglu_backward(shape, ckpt.flatten(), off, dh, outs[0], outs[1], h=outs[2])
    for a in (0, R // 2, R - 40):
        rows = ckpt[a:a + 40].cpu().numpy()
        u = orc.dequantize_blocks_e4m3(rows[:, f:2 * f], rows[:, 2 * f + f // 32:2 * f + f // 16]
                                       .astype(np.int32) - 127)
        v = orc.dequantize_blocks_e4m3(rows[:, :f], rows[:, 2 * f:2 * f + f // 32]
                                       .astype(np.int32) - 127)
        want, mag = swiglu_grads(v, u, f64(dh[a:a + 40]))
        for t, w, size in zip(outs, want, mag):
            rel = 2.0 ** -18 + np.abs(v) * 2.0 ** -22
            bound = rel * size + 2.0 ** -8 * (np.abs(w) + rel * size) + 1e-38
            assert np.all(np.abs(f64(t[a:a + 40]) - w) <= bound)
    for t in outs:
        assert torch.all(t[R:] == 7.0)
    assert m.moe_get_device_error(True) == 0


@pytest.mark.parametrize("E", [24, 200])
def test_two_calls_at_once(E):
    """Two streams, a workspace and outputs each: both as alone."""
    m = lib()
    cases = [inputs(3001 + 700 * i, 520, E, 4, 50 + i, 0.05)[1] for i in range(2)]
    alone = [call(m, a, E, add=True) for a in cases]
    for a, o in zip(cases, alone):
        check(a, E, o, add=True)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for a, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(call(m, a, E, add=True))
        torch.cuda.synchronize()
        for o, w in zip(got, alone):
            assert all(torch.equal(o[k], w[k]) for k in ("dx", "dw", "db"))
    assert m.moe_get_device_error(True) == 0
