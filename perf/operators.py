"""Cases of the layer's training operators: the balance loss with its per-expert counts and its
gradient, the router's backward pass, the gate/up GEMM that leaves an 8-bit checkpoint, and the
activation's backward pass that reads it.

``run`` computes a case either in plain torch operations (``own`` false) or by the calls a user of
the package makes (``own`` true). Sizes are those of the repository's workloads (the 64-token layer,
the 4-layer stack, the 128-expert layer, the Mixtral-shaped layer, the 256-expert decode layer), odd
ones beside them, and long batches.
"""
import math

import torch

own = False

BALANCE_COEF, Z_COEF = 1e-2, 1e-3


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the 64-token layer: one short step, where launches count
        dict(name="balance_tiny", op="balance", N=64, E=8, K=2, mask=0.0),
        # a packed batch of many sequences over 256 experts, some of it padding
        dict(name="balance_pack", op="balance", N=131072, E=256, K=8, mask=0.07),
        # one layer of the 4-layer stack
        dict(name="balance_grad_stack", op="balance_grad", N=32768, E=64, K=6, mask=0.0),
        # an odd token count, an expert count that is no power of two, padding
        dict(name="balance_grad_odd", op="balance_grad", N=30011, E=160, K=6, mask=0.2),
        # the 64-token layer's router
        dict(name="route_grad_tiny", op="route_grad", N=64, d=128, E=8, K=2, bf16=True, add=False,
             loss=True, mask=0.0),
        # the 128-expert layer's router, gradients of the gate weights alone
        dict(name="route_grad_e128", op="route_grad", N=8192, d=2048, E=128, K=8, bf16=True,
             add=False, loss=False, mask=0.0),
        # one layer of the stack: both gradients, the residual's gradient added, padding
        dict(name="route_grad_stack", op="route_grad", N=32768, d=4096, E=64, K=6, bf16=True,
             add=True, loss=True, mask=0.05),
        # the widest router (256 experts, d of the decode layer), an odd batch, fp32 dx
        dict(name="route_grad_e256", op="route_grad", N=4001, d=7168, E=256, K=8, bf16=False,
             add=False, loss=True, mask=0.0),
        # the experts of the 128-expert layer: forward with the checkpoint, then the activation's
        # backward pass from it
        dict(name="experts_e128", op="experts", N=8192, K=8, d=2048, f=768, E=128),
        # the experts of the Mixtral-shaped layer
        dict(name="experts_mixtral", op="experts", N=4096, K=2, d=4096, f=14336, E=8),
        # the activation's backward pass alone: a few rows over many experts
        dict(name="act_grad_few", op="act_grad", N=16, K=8, f=2048, E=256),
        # ... and one layer of the stack
        dict(name="act_grad_stack", op="act_grad", N=32768, K=6, f=1536, E=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "balance_grad", "route_grad", "experts", "act_grad"])
    E = _log_int(rng, 4, 256)
    K = rng.randint(1, min(8, E))
    mask = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op in ("balance", "balance_grad"):
        return dict(op=op, N=_log_int(rng, 32, 131072), E=E, K=K, mask=mask)
    if op == "route_grad":
        d = 8 * _log_int(rng, 16, 896)
        N = _log_int(rng, 32, min(32768, (1 << 27) // d))
        return dict(op=op, N=N, d=d, E=E, K=K, bf16=rng.random() < 0.6, add=rng.random() < 0.4,
                    loss=rng.random() < 0.7, mask=mask)
    if op == "experts":
        d, f = 128 * _log_int(rng, 2, 32), 128 * _log_int(rng, 2, 48)
        E = min(E, max(1, (1 << 28) // (d * f)))
        K = min(K, E)
        return dict(op=op, N=_log_int(rng, 32, max(64, min(8192, (1 << 37) // (d * f * K)))), K=K,
                    d=d, f=f, E=E)
    f = 128 * _log_int(rng, 1, 112)
    return dict(op=op, N=_log_int(rng, 16, min(32768, (1 << 28) // (f * K))), K=K, f=f, E=E)


# ---------------------------------------------------------------- inputs

def _offsets(N, K, E, g):
    """Rows per expert of a skewed routing of N * K assignments, as the dispatch leaves them:
    exclusive scan [E + 1] and the counts (host)."""
    p = torch.softmax(0.35 * torch.randn(E, generator=g, device="cuda"), 0)
    e = torch.multinomial(p, N * K, replacement=True, generator=g)
    counts = torch.bincount(e, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0).to(torch.int32)
    return off, counts


def _routing(N, E, K, g):
    """Logits with a Zipf-like skew, the K largest of each token and the softmax over them."""
    bias = -0.3 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    logits = torch.randn(N, E, generator=g, device="cuda") + bias
    top, idx = logits.topk(K, dim=1)
    return logits, idx.to(torch.int32), torch.softmax(top, 1)


def _mask(N, share, g):
    if share <= 0.0:
        return None
    return (torch.rand(N, generator=g, device="cuda") >= share).to(torch.uint8)


def _quantize(v):
    """[R][f] fp32 -> (e4m3 codes of v * 2^-j, j) per block of 32 columns: j is the smallest power
    with max|block| * 2^-j <= 448 (0 for a zero block)."""
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    m, e = torch.frexp(amax)                      # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    j = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    j = torch.where(amax > 0, j, torch.zeros_like(j))
    inv = ((127 - j) << 23).view(torch.float32)   # 2^-j
    return (b * inv[:, :, None]).to(torch.float8_e4m3fn), j


def _dequantize(codes, j):
    return (codes.float() * ((j + 127) << 23).view(torch.float32)[:, :, None]).flatten(1)


def _stride(f):
    return 2 * f + (f // 16 + 15) // 16 * 16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case)
    if op in ("balance", "balance_grad", "route_grad"):
        N, E, K = case["N"], case["E"], case["K"]
        s["logits"], s["idx"], s["w"] = _routing(N, E, K, g)
        s["mask"] = _mask(N, case["mask"], g)
    if op == "balance_grad":
        keep = torch.ones(N, dtype=torch.bool, device="cuda") if s["mask"] is None \
            else s["mask"].bool()
        s["counts"] = torch.bincount(s["idx"][keep].flatten(), minlength=E).to(torch.int32)
        s["tokens"] = keep.sum().to(torch.int32).reshape(1)
        s["dloss"] = 0.5 + torch.rand(1, generator=g, device="cuda")
    if op == "route_grad":
        d = case["d"]
        s["x"] = torch.randn(N, d, generator=g, device="cuda").to(torch.bfloat16)
        s["wr"] = torch.randn(E, d, generator=g, device="cuda") / d ** 0.5
        s["dw"] = torch.randn(N, K, generator=g, device="cuda") / N
        s["dlogits"] = (1e-1 / N) * torch.softmax(s["logits"], 1) * \
            torch.randn(N, E, generator=g, device="cuda") if case["loss"] else None
        s["add"] = (torch.randn(N, d, generator=g, device="cuda") / N).to(torch.bfloat16) \
            if case["add"] else None
    if op in ("experts", "act_grad"):
        N, K, E, f = case["N"], case["K"], case["E"], case["f"]
        R = N * K
        s["R"], rows = R, R + 128
        s["off"], counts = _offsets(N, K, E, g)
        s["dh"] = (1e-3 * torch.randn(rows, f, generator=g, device="cuda")).to(torch.bfloat16)
    if op == "experts":
        d = case["d"]
        s["cap"] = int(counts.max())
        s["x"] = torch.randn(rows, d, generator=g, device="cuda").to(torch.bfloat16)
        for n in ("w1", "w3"):
            s[n] = torch.empty(E, f, d, device="cuda", dtype=torch.bfloat16).normal_(
                0.0, 0.02, generator=g)
    if op == "act_grad":
        s["ckpt"] = torch.zeros(rows, _stride(f), dtype=torch.uint8, device="cuda")
        # pre-activations of unit scale with rows and columns of other sizes, as trained ones have
        for at in range(0, R, 1 << 16):
            n = min(1 << 16, R - at)
            out = s["ckpt"][at:at + n]
            for i in range(2):
                v = torch.randn(n, f, generator=g, device="cuda")
                v *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
                v *= torch.exp(0.3 * torch.randn(1, f, generator=g, device="cuda"))
                codes, j = _quantize(v)
                out[:, i * f:(i + 1) * f] = codes.view(torch.uint8).view(n, f)
                out[:, 2 * f + i * (f // 32):2 * f + (i + 1) * (f // 32)] = (j + 127).to(torch.uint8)
    s["out"] = _buffers(s)
    return s


def _buffers(s):
    """What the calls write, and their workspace and shape: allocated once by the user's program."""
    op = s["op"]
    if not own:
        return None
    import combine_grouped_gemm_router_b200 as moe

    def new(*size, dtype=torch.float32):
        return torch.empty(*size, dtype=dtype, device="cuda")

    N, E, K = s["N"], s["E"], s["K"]
    bf = torch.bfloat16
    o = {"moe": moe}
    if op in ("balance", "balance_grad"):
        o["shape"] = sh = moe.make_shape(N, 128, 128, E, K, 1)
        o["dlogits"] = new(N, E) if op == "balance_grad" else None
        o["loss"], o["counts"], o["mean"] = new(3), new(E, dtype=torch.int32), new(E)
        o["tokens"] = new(1, dtype=torch.int32)
        o["ws"] = new(moe.moe_balance_workspace_size(sh), dtype=torch.uint8)
    elif op == "route_grad":
        o["shape"] = sh = moe.make_shape(N, s["d"], 128, E, K, 1, out_bf16=s["bf16"])
        o["dx"] = new(N, s["d"], dtype=bf if s["bf16"] else torch.float32)
        o["dwr"], o["dbias"] = new(E, s["d"]), new(E)
        o["ws"] = new(moe.moe_route_backward_workspace_size(sh), dtype=torch.uint8)
    else:
        o["shape"] = sh = moe.make_shape(N, s.get("d", 128), s["f"], E, K, 1)
        rows = moe.moe_rows_alloc(sh)
        for n in ("dgate", "dup", "h2"):
            o[n] = new(rows, s["f"], dtype=bf)
        if op == "experts":
            o["h"] = new(rows, s["f"], dtype=torch.float16)
            o["ckpt"] = new(moe.moe_checkpoint_bytes(sh), dtype=torch.uint8)
    return o


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    o, op = s["out"], s["op"]
    moe, sh = o["moe"], o["shape"]
    if op == "balance":
        moe.moe_balance_loss(sh, s["logits"], s["idx"], o["loss"], o["counts"], o["mean"],
                             o["tokens"], token_mask=s["mask"], balance_coef=BALANCE_COEF,
                             z_coef=Z_COEF, ws=o["ws"])
        return [o["loss"], o["counts"], o["mean"], o["tokens"]]
    if op == "balance_grad":
        moe.moe_balance_loss_backward(sh, s["logits"], s["counts"], s["tokens"], o["dlogits"],
                                      token_mask=s["mask"], balance_coef=BALANCE_COEF,
                                      z_coef=Z_COEF, dloss=s["dloss"])
        return [o["dlogits"]]
    if op == "route_grad":
        moe.moe_route_backward(sh, s["x"], s["wr"], o["dx"], o["dwr"], dbias=o["dbias"],
                               topk_idx=s["idx"], topk_w=s["w"], dtopk_w=s["dw"],
                               dlogits=s["dlogits"], token_mask=s["mask"], dx_add=s["add"],
                               ws=o["ws"])
        return [o["dx"], o["dwr"], o["dbias"]]
    R = s["R"]
    ckpt = s.get("ckpt")
    if op == "experts":
        ckpt = o["ckpt"]
        moe.moe_expert_up_checkpoint(sh, s["x"], s["off"], s["w1"], s["w3"], o["h"], ckpt)
    moe.moe_swiglu_backward(sh, ckpt, s["off"], s["dh"], o["dgate"], o["dup"], h=o["h2"])
    grads = [o["dgate"][:R], o["dup"][:R], o["h2"][:R]]
    return grads if op == "act_grad" else [o["h"][:R]] + grads


def _plain_balance(s):
    l, K, E = s["logits"], s["K"], s["E"]
    keep = torch.ones(l.shape[0], device="cuda") if s["mask"] is None else s["mask"].float()
    m = keep.sum()
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total)).flatten()
    mean = (e / total * keep[:, None]).sum(0) / m
    hits = torch.zeros(E, device="cuda", dtype=torch.int64).index_add_(
        0, s["idx"].flatten().long(), keep.long().repeat_interleave(K))
    balance = E * (hits.float() / (m * K) * mean).sum()
    z = (lse * lse * keep).sum() / m
    return [torch.stack([BALANCE_COEF * balance + Z_COEF * z, balance, z]), hits.to(torch.int32),
            mean, m.to(torch.int32).reshape(1)]


def _plain_balance_grad(s):
    l, K, E = s["logits"], s["K"], s["E"]
    m = s["tokens"].float()
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - top)
    total = e.sum(1, keepdim=True)
    p = e / total
    lse = top + torch.log(total)
    share = s["counts"].float() / (m * K)
    inner = (share * p).sum(1, keepdim=True)
    dl = s["dloss"] * p * (BALANCE_COEF * E / m * (share - inner) + 2 * Z_COEF / m * lse)
    return [dl if s["mask"] is None else torch.where(s["mask"].bool()[:, None], dl, 0.0)]


def _plain_route_grad(s):
    w, dw = s["w"], s["dw"]
    gate = w * (dw - (w * dw).sum(1, keepdim=True))
    dl = torch.zeros(s["N"], s["E"], device="cuda") if s["dlogits"] is None \
        else s["dlogits"].clone()
    dl.scatter_add_(1, s["idx"].long(), gate)
    x = s["x"].float()
    if s["mask"] is not None:
        keep = s["mask"].bool()[:, None]
        dl, x = torch.where(keep, dl, 0.0), torch.where(keep, x, 0.0)
    dx = dl @ s["wr"]
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return [dx.to(torch.bfloat16) if s["bf16"] else dx, dl.t() @ x, dl.sum(0)]


def _swiglu_grads(g, u, dh):
    sig = torch.sigmoid(g)
    out = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig, g * sig * u
    return [v.to(torch.bfloat16) for v in out]


def _plain_act_grad(s):
    R, f, c = s["R"], s["f"], s["ckpt"]
    v = []
    for i in range(2):  # gate, up
        codes = c[:R, i * f:(i + 1) * f].view(torch.float8_e4m3fn).unflatten(1, (-1, 32))
        j = c[:R, 2 * f + i * (f // 32):2 * f + (i + 1) * (f // 32)].int() - 127
        v.append(_dequantize(codes, j))
    return _swiglu_grads(v[0], v[1], s["dh"][:R].float())


def _plain_experts(s):
    E, R, cap, off = s["E"], s["R"], s["cap"], s["off"].long()
    slot = off[:-1, None] + torch.arange(cap, device="cuda")          # [E][cap] rows, padded
    xp = s["x"][slot.clamp(max=R - 1)].float()
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), off.diff(), output_size=R)
    at = expert * cap + torch.arange(R, device="cuda") - off[expert]  # row -> its padded place
    g = torch.bmm(xp, s["w1"].float().transpose(1, 2)).flatten(0, 1)[at]
    u = torch.bmm(xp, s["w3"].float().transpose(1, 2)).flatten(0, 1)[at]
    h = (g * torch.sigmoid(g) * u).to(torch.float16)
    return [h] + _swiglu_grads(_dequantize(*_quantize(g)), _dequantize(*_quantize(u)),
                               s["dh"][:R].float())


_PLAIN = {"balance": _plain_balance, "balance_grad": _plain_balance_grad,
          "route_grad": _plain_route_grad, "experts": _plain_experts, "act_grad": _plain_act_grad}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    N, E, K, op = case["N"], case["E"], case["K"], case["op"]
    if op == "balance":
        return {"bytes": 4 * N * E + 4 * N * K + (N if case["mask"] else 0) + 8 * E,
                "flops": 8 * N * E}
    if op == "balance_grad":
        return {"bytes": 8 * N * E + (N if case["mask"] else 0) + 4 * E, "flops": 10 * N * E}
    if op == "route_grad":
        d = case["d"]
        return {"bytes": (2 + (2 if case["bf16"] else 4) + (2 if case["add"] else 0)) * N * d
                + 8 * E * d + 12 * N * K + (4 * N * E if case["loss"] else 0) + 4 * E
                + (N if case["mask"] else 0), "flops": 4 * N * E * d}
    R, f = N * K, case["f"]
    codes = 2 * R * f + 2 * R * (f // 32)
    if op == "act_grad":
        return {"bytes": codes + 8 * R * f, "flops": 20 * R * f}
    d = case["d"]
    # x, both weights and dh in, h and the three outputs of the backward pass out; the checkpoint
    # is written by the one call and read by the other
    return {"bytes": 2 * R * d + 4 * E * f * d + 2 * codes + 10 * R * f, "flops": 4 * R * f * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def _round_e4m3(v):
    """Values [R][f] in 64 bits -> what their block codes stand for."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    j = torch.ceil(torch.log2(amax / 448.0))
    j = torch.where(amax > 448.0 * torch.exp2(j), j + 1, j)           # log2 next to a border
    j = torch.where(amax <= 448.0 * torch.exp2(j - 1), j - 1, j).clamp(-126, 127)
    j = torch.where(amax > 0, j, 0.0)
    a = b / torch.exp2(j)
    step = torch.exp2(torch.frexp(a.abs()).exponent.clamp(min=-5).double() - 4)
    return (torch.round(a / step) * step * torch.exp2(j)).reshape(v.shape)


def _exact_swiglu(g, u, dh):
    half = 0.5 * torch.tanh(0.5 * g)
    sig = 0.5 + half
    silu = g * sig
    return [dh * u * (sig + silu * (0.5 - half)), dh * silu, silu * u]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    E, K = case["E"], case["K"]
    if op in ("balance", "balance_grad"):
        keep = torch.ones(case["N"], dtype=torch.bool, device="cuda") if s["mask"] is None \
            else s["mask"] != 0
        l, m = s["logits"].double(), int(keep.sum())
        logp = torch.log_softmax(l, 1)
        lse = torch.logsumexp(l, 1)
        hits = torch.stack([((s["idx"] == e) & keep[:, None]).sum() for e in range(E)])
        share = hits.double() / (m * K)
        if op == "balance":
            mean = torch.exp(logp[keep]).sum(0) / m
            balance, z = E * torch.dot(share, mean), lse[keep].square().sum() / m
            return [torch.stack([BALANCE_COEF * balance + Z_COEF * z, balance, z]), None, mean, None]
        # d/dl of cb E sum_e f_e P_e + cz mean lse^2 through dp_e/dl_i = p_e (1[e = i] - p_i)
        p = torch.exp(logp)
        dl = BALANCE_COEF * E / m * (p * share - p * (p @ share)[:, None])
        dl += Z_COEF * (2.0 / m) * lse[:, None] * p
        return [dl * keep[:, None] * s["dloss"].double()]
    if op == "route_grad":
        w, dw = s["w"].double(), s["dw"].double()
        dl = torch.zeros(case["N"], E, dtype=torch.float64, device="cuda")
        rows = torch.arange(case["N"], device="cuda")
        for k in range(K):  # the softmax's Jacobian, one column after another
            for i in range(K):
                dl[rows, s["idx"][:, i].long()] += dw[:, k] * w[:, k] * ((1.0 if i == k else 0.0)
                                                                         - w[:, i])
        if s["dlogits"] is not None:
            dl += s["dlogits"].double()
        if s["mask"] is not None:
            dl[s["mask"] == 0] = 0.0
        dx = dl @ s["wr"].double()
        if s["add"] is not None:
            dx += s["add"].double()
        return [dx, dl.t() @ s["x"].double(), dl.sum(0)]
    R, f = s["R"], case["f"]
    dh = s["dh"][:R].double()
    if op == "act_grad":
        c = s["ckpt"][:R]
        table = torch.tensor([_e4m3(b) for b in range(256)], dtype=torch.float64, device="cuda")
        v = [table[c[:, i * f:(i + 1) * f].int()]
             * torch.exp2(c[:, 2 * f + i * f // 32:2 * f + (i + 1) * f // 32].double() - 127)
             .repeat_interleave(32, 1) for i in range(2)]
        return _exact_swiglu(v[0], v[1], dh)
    out = [torch.empty(R, f, dtype=torch.float64, device="cuda") for _ in range(4)]
    bounds = s["off"].tolist()
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        x = s["x"][a:b].double()
        g, u = x @ s["w1"][e].double().t(), x @ s["w3"][e].double().t()
        rows = [_exact_swiglu(g, u, dh[a:b])[2]]
        rows += _exact_swiglu(_round_e4m3(g), _round_e4m3(u), dh[a:b])
        for o, r in zip(out, rows):
            o[a:b] = r
    return out


def _e4m3(b):
    """The value of an e4m3 code: sign, 4 exponent bits with bias 7, 3 mantissa bits."""
    sign, e, m = -1.0 if b & 128 else 1.0, b >> 3 & 15, b & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9))
