"""64-bit definitions of the mixture-of-experts operators and rigorous error
bounds for their tests (no kernel arithmetic here)."""
import math

import torch

import oracle


def route(logits, top_k, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1,
          renormalize=True, scale=1.0):
    """(indices, weights, keys) of the header's definition, token by token."""
    T, E = logits.shape
    idx = torch.zeros((T, top_k), dtype=torch.int32)
    wts = torch.zeros((T, top_k), dtype=torch.float64)
    L = logits.detach().cpu().double().tolist()
    B = bias.detach().cpu().double().tolist() if bias is not None else None
    gs = E // n_groups
    for t in range(T):
        l = L[t]
        if score == "sigmoid":
            s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in l]
        else:
            clean = [v for v in l if v == v]
            m = max(clean) if clean else -math.inf
            ex = [0.0 if m == -math.inf or v != v else (1.0 if v == m else math.exp(v - m)) for v in l]
            z = math.fsum(ex)
            s = [v / z if z > 0 else 0.0 for v in ex]
        sel = s if B is None else [a + b for a, b in zip(s, B)]
        sel = [v if l[i] == l[i] else math.nan for i, v in enumerate(sel)]
        key = [(v if B is None else sel[i]) if v == v else math.nan for i, v in enumerate(l)]
        live = set(range(E))
        if n_groups > 1:
            gsc = []
            for g in range(n_groups):
                mem = sorted((v for v in sel[g * gs:(g + 1) * gs]), key=lambda v: (v != v, -v if v == v else 0))
                gsc.append(sum(mem[:group_top]))
            order = sorted(range(n_groups), key=lambda g: (gsc[g] != gsc[g], -gsc[g] if gsc[g] == gsc[g] else 0, g))
            keep = set(order[:topk_groups])
            live = {e for e in range(E) if e // gs in keep}
        chosen = sorted(live, key=lambda e: (key[e] != key[e], -key[e] if key[e] == key[e] else 0, e))[:top_k]
        w = [s[e] for e in chosen]
        if renormalize:
            if score == "softmax":  # relative to the largest chosen logit
                lc = [l[e] for e in chosen]
                m = max([v for v in lc if v == v], default=-math.inf)
                w = [0.0 if m == -math.inf or v != v else (1.0 if v == m else math.exp(v - m)) for v in lc]
            z = math.fsum(w)
            w = [v / z if z > 0 else 0.0 for v in w]
        if any(v != v for v in l):
            w = [math.nan] * top_k
        idx[t] = torch.tensor(chosen, dtype=torch.int32)
        wts[t] = torch.tensor(w, dtype=torch.float64) * scale
    return idx, wts


def act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def dense(packed, rows, mode, gs):
    """[E, rows, cols] float64 of a stacked packed weight on the CPU: the exact
    s q + b or X * element, not rounded to the dtype."""
    wq, s, b = packed
    E, R, words = wq.shape
    w64 = wq.to(torch.int64) & 0xFFFFFFFF
    q = torch.stack([(w64 >> (4 * i)) & 15 for i in range(8)], -1).reshape(E, R, words * 8)
    if mode == "affine":
        return s.double().repeat_interleave(gs, -1) * q.double() + b.double().repeat_interleave(gs, -1)
    val = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)[q]
    if mode == "mxfp4":
        x = torch.where(s == 255, math.nan, torch.pow(torch.tensor(2.0, dtype=torch.float64), s.double() - 127))
    else:
        x = s.view(torch.float8_e4m3fn).double()
    return x.repeat_interleave(gs, -1) * val


def quantize(w, gs, mode):
    """Stacked weight [E, rows, cols] packed by the oracle."""
    E, R, C = w.shape
    wq, s, b = oracle.quantize(w.reshape(E * R, C), gs, 4, mode)
    return (wq.reshape(E, R, -1), s.reshape(E, R, -1), None if b is None else b.reshape(E, R, -1))


def experts(x, indices, weights, gate, up, down, mode, gs, activation, few_rows):
    """(y, bound): the layer in float64 and a bound of |kernel - y| per output.

    The bound adds up, at their largest, the roundings the header names.
    few_rows: activations as integers, off by at most half a unit where their
    largest of 32 is at least 2^13 units, that is 2^-14 of it.  Otherwise: h, and
    each affine weight, rounded to the dtype (half a step, eps/2, relative; twice
    for a weight: the product s q is not rounded, s q + b once, and half a step
    more covers the cancellation-free case of b + s q near a power of two).
    fp32 sums of n terms: n 2^-24 of the sum of magnitudes.  The activations'
    slopes are below 1.13 (silu 1.1), their fp32 evaluation within 2^-20.
    """
    half = torch.finfo(x.dtype).eps / 2
    X = x.double()
    dev = X.device
    T, K = X.shape
    E, I = gate[0].shape[:2]
    N = down[0].shape[1]
    y = torch.zeros(T, N, dtype=torch.float64, device=dev)
    bound = torch.zeros(T, N, dtype=torch.float64, device=dev)

    def in_err(v):
        if not few_rows:
            return torch.zeros_like(v)
        m = v.abs().reshape(v.shape[0], -1, 32).amax(-1, keepdim=True)
        return (m * 2.0 ** -14).expand(-1, -1, 32).reshape(v.shape)

    wr = 2 * half if (mode == "affine" and not few_rows) else 0.0
    for e in range(E):
        t, j = (indices == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        Wg, Wu, Wd = (dense(tuple(None if p is None else p[e:e + 1] for p in w), None, mode, gs)[0].to(dev)
                      for w in (gate, up, down))
        x_, w = X[t], weights[t, j].double()[:, None]
        g, u = x_ @ Wg.T, x_ @ Wu.T
        rel = wr + K * 2.0 ** -24
        dg = in_err(x_) @ Wg.abs().T + rel * (x_.abs() @ Wg.abs().T)
        du = in_err(x_) @ Wu.abs().T + rel * (x_.abs() @ Wu.abs().T)
        a = act(g, activation)
        da = 1.13 * dg + 2.0 ** -20 * a.abs()
        h = a * u
        dh = da * (u.abs() + du) + a.abs() * du + 2.0 ** -23 * h.abs()
        if not few_rows:
            dh = dh + half * (h.abs() + dh) + torch.finfo(x.dtype).tiny
        dh = dh + in_err(h.abs() + dh)
        part = dh @ Wd.abs().T + (wr + I * 2.0 ** -24) * ((h.abs() + dh) @ Wd.abs().T)
        y.index_add_(0, t, w * (h @ Wd.T))
        bound.index_add_(0, t, w.abs() * (part + 2.0 ** -22 * (h.abs() @ Wd.abs().T)))
    return y, bound + half * (y.abs() + bound) + torch.finfo(x.dtype).tiny
