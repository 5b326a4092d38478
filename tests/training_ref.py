"""The training operators' definitions in 64 bits (numpy), and random inputs for them."""
from __future__ import annotations

import numpy as np
import torch


def softmax64(logits):
    """(p, lse) of each row, 64 bits; -inf logits have probability 0."""
    l = np.asarray(logits, np.float64)
    m = l.max(1, keepdims=True)
    e = np.exp(l - m)
    s = e.sum(1, keepdims=True)
    return e / s, (m + np.log(s))[:, 0]


def balance(logits, topk_idx, mask, cb, cz, counts=None, tokens=None):
    """dict: loss [3], counts, prob_mean, tokens, share (f_e), p, lse, keep. counts / tokens given:
    held fixed (what the gradient differentiates)."""
    N, E = logits.shape
    K = topk_idx.shape[1]
    keep = np.ones(N, bool) if mask is None else np.asarray(mask) != 0
    p = np.zeros((N, E))
    lse = np.zeros(N)
    p[keep], lse[keep] = softmax64(np.asarray(logits)[keep])
    idx = np.asarray(topk_idx)[keep].reshape(-1)
    own = np.bincount(idx[(idx >= 0) & (idx < E)], minlength=E)
    counts = own if counts is None else counts
    M = int(keep.sum()) if tokens is None else tokens
    if M == 0:
        z = np.zeros(3)
        return dict(loss=z, counts=counts, prob_mean=np.zeros(E), tokens=0, share=np.zeros(E),
                    p=p, lse=lse, keep=keep)
    share, mean = counts / (M * K), p.sum(0) / M
    bal, zz = E * float(share @ mean), float((lse ** 2).sum() / M)
    return dict(loss=np.array([cb * bal + cz * zz, bal, zz]), counts=counts, prob_mean=mean,
                tokens=M, share=share, p=p, lse=lse, keep=keep)


def balance_grad(ref, E, cb, cz, dloss):
    """Gradient of ref's loss[0] and the magnitude of the terms it is the sum of."""
    p, M = ref["p"], max(ref["tokens"], 1)
    on = ref["keep"][:, None] * (1.0 if ref["tokens"] else 0.0)
    inner = p @ ref["share"]
    a, b = dloss * cb * E / M, dloss * cz * 2.0 / M
    g = p * (a * (ref["share"][None] - inner[:, None]) + b * ref["lse"][:, None])
    mag = p * (abs(a) * (ref["share"][None] + inner[:, None]) + abs(b * ref["lse"])[:, None])
    return g * on, mag * on


def gate_grad(topk_idx, topk_w, dtopk_w, dlogits, mask, N, E):
    """dl [N][E] and the magnitude of its terms, 64 bits."""
    dl = np.zeros((N, E))
    mag = np.zeros((N, E))
    keep = np.ones(N, bool) if mask is None else np.asarray(mask) != 0
    if dlogits is not None:
        dl[keep] += np.asarray(dlogits, np.float64)[keep]
        mag[keep] += np.abs(dl[keep])
    if dtopk_w is not None:
        idx = np.asarray(topk_idx)
        ok = (idx >= 0) & (idx < E) & keep[:, None]
        w = np.where(ok, np.asarray(topk_w, np.float64), 0.0)
        dw = np.where(ok, np.asarray(dtopk_w, np.float64), 0.0)
        s, sm = (w * dw).sum(1, keepdims=True), np.abs(w * dw).sum(1, keepdims=True)
        t, k = np.nonzero(ok)
        np.add.at(dl, (t, idx[t, k]), (w * (dw - s))[t, k])
        np.add.at(mag, (t, idx[t, k]), (w * (np.abs(dw) + sm))[t, k])
    return dl, mag


def swiglu_grads(g, u, dh):
    """(dgate, dup, h) and the magnitudes of their terms."""
    s = 1.0 / (1.0 + np.exp(-g))
    silu = g * s
    mag = (np.abs(dh * u) * s * (1.0 + np.abs(g)), np.abs(dh * silu), np.abs(silu * u))
    return (dh * u * s * (1.0 + g * (1.0 - s)), dh * silu, silu * u), mag


def topk_of(logits, K):
    """The K largest of each row (ties to the lower index) and the softmax over them."""
    order = np.argsort(-np.asarray(logits, np.float64), 1, kind="stable")[:, :K]
    w, _ = softmax64(np.take_along_axis(np.asarray(logits), order, 1))
    return order.astype(np.int32), w.astype(np.float32)


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()
