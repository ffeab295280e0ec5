"""Workloads of the mixture-of-experts operators: routing tokens to experts and
the experts' gated products on 4-bit weights.

With ``own`` false, ``run`` computes an operator in its plain form, elementary
torch operations in 32 bits (64 for the keys that experts are chosen by);
with ``own`` true it makes the library's call on the same inputs.  ``exact``
evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

# E2M1 values of the codes 0..15 (sign in bit 3).
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = E2M1 + [-v for v in E2M1]
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _route(name, **kw):
    c = dict(op="route", name=name, T=1, E=8, k=2, dtype="bf16", score="softmax", bias=False, n_groups=1,
             topk_groups=1, group_top=1, renormalize=True, scale=1.0)
    c.update(kw)
    return c


def _experts(name, **kw):
    c = dict(op="experts", name=name, T=1, E=8, k=2, K=4096, I=14336, dtype="bf16", mode="mxfp4",
             group_size=32, act="silu", skew=0.0, dropped=0.0)
    c.update(kw)
    return c


def listed():
    return [
        # one generated token, few experts: the smallest call there is
        _route("route_1_of_8"),
        # a decode batch over many experts
        _route("route_64x64", T=64, E=64, k=8, dtype="f32"),
        # a long prompt: sigmoid scores, a balance bias, 4 of 8 groups of experts
        _route("route_16384x256_groups", T=16384, E=256, k=8, dtype="f32", score="sigmoid", bias=True,
               n_groups=8, topk_groups=4, group_top=2, scale=2.5),
        # a ragged prompt, an odd number of experts, weights not renormalised
        _route("route_3001x60", T=3001, E=60, k=6, dtype="f16", renormalize=False, scale=1.5),
        # one token through two of eight large experts
        _experts("experts_1x2of8_mxfp4"),
        # one token through eight of 64 small experts
        _experts("experts_1x8of64_nvfp4", E=64, k=8, K=2048, I=1024, mode="nvfp4", group_size=16),
        # a few sequences decoding together
        _experts("experts_5x4of16_affine", T=5, E=16, k=4, K=2048, I=2048, dtype="f16", mode="affine",
                 group_size=64),
        # a decode batch that touches nearly every expert with a few rows each
        _experts("experts_32x8of64_mxfp4", T=32, E=64, k=8, K=2048, I=1024),
        # odd sizes, padded slots (index -1), the tanh form of gelu
        _experts("experts_77x3of10_odd", T=77, E=10, k=3, K=1088, I=704, dtype="f16", mode="nvfp4",
                 group_size=16, act="gelu_tanh", dropped=0.1),
        # 512 tokens over eight large experts of uneven popularity
        _experts("experts_512x2of8_mxfp4", T=512, skew=1.2),
        # a prompt over many small experts
        _experts("experts_4096x8of64_affine", T=4096, E=64, k=8, K=2048, I=1024, mode="affine", group_size=64,
                 skew=0.5),
        # a prompt over eight large experts
        _experts("experts_2048x2of8_nvfp4", T=2048, mode="nvfp4", group_size=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        E = rng.randint(2, 256)
        n_groups = rng.choice([1, 1, 2, 4, 8])
        E = max(n_groups * 2, E // n_groups * n_groups)
        topk_groups = rng.randint(1, n_groups)
        return dict(op="route", T=_log_int(rng, 1, 16384), E=E,
                    k=rng.randint(1, min(16, E // n_groups * topk_groups)),
                    dtype=rng.choice(["bf16", "f16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, n_groups=n_groups, topk_groups=topk_groups,
                    group_top=rng.choice([1, 2]), renormalize=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.5, 2.5]))
    while True:
        mode, gs = rng.choice([("mxfp4", 32), ("nvfp4", 16), ("affine", 32), ("affine", 64), ("affine", 128)])
        step = max(64, gs)
        E = _log_int(rng, 1, 64)
        c = dict(op="experts", T=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(8, E)),
                 K=step * max(1, _log_int(rng, 256, 4096) // step), I=step * max(1, _log_int(rng, 128, 14336) // step),
                 dtype=rng.choice(["bf16", "f16"]), mode=mode, group_size=gs,
                 act=rng.choice(["silu", "gelu_tanh"]), skew=rng.choice([0.0, 0.5, 1.2]),
                 dropped=rng.choice([0.0, 0.0, 0.1]))
        if E * c["K"] * c["I"] <= 8 * 4096 * 14336 and c["T"] * c["k"] * c["K"] * c["I"] <= 4096 * 4096 * 14336:
            return c


# ---------------------------------------------------------------- inputs

def _pack(codes):
    """4-bit codes [rows, cols] (uint8) -> int32 words, least significant code first."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous().view(torch.int32)


def _quantize(w, mode, gs, dtype):
    """A float32 weight [rows, cols] -> packed codes, scales, biases."""
    rows, cols = w.shape
    g = w.view(rows, cols // gs, gs)
    if mode == "affine":
        lo, hi = g.amin(-1), g.amax(-1)
        s, b = ((hi - lo) / 15).to(dtype), lo.to(dtype)
        sf = s.float().clamp_min(1e-30)
        q = ((g - b.float().unsqueeze(-1)) / sf.unsqueeze(-1)).round().clamp(0, 15).to(torch.uint8)
        return _pack(q.view(rows, cols)), s, b
    amax = g.abs().amax(-1)
    if mode == "mxfp4":
        byte = (torch.frexp(amax).exponent - 3 + 127).clamp(1, 254).to(torch.uint8)
        x = _e8m0(byte)
    else:
        x8 = (amax / 6).to(torch.float8_e4m3fn)
        byte, x = x8.view(torch.uint8), x8.float()
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    v = g / x.clamp_min(1e-30).unsqueeze(-1)
    q = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return _pack(q.view(rows, cols)), byte, None


def _stack(gen, E, rows, cols, std, mode, gs, dtype):
    """E quantized experts of N(0, std^2) weights, stacked on the leading axis."""
    parts = []
    for _ in range(E):
        w = torch.randn((rows, cols), generator=gen, device="cuda") * std
        parts.append(_quantize(w, mode, gs, dtype))
    return tuple(torch.stack([p[i] for p in parts]) if parts[0][i] is not None else None for i in range(3))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, E, k = case["T"], case["E"], case["k"]
    st = dict(case)
    if case["op"] == "route":
        st["logits"] = (torch.randn((T, E), generator=gen, device="cuda") * 1.5).to(dt)
        st["b"] = torch.randn((E,), generator=gen, device="cuda") * 0.1 if case["bias"] else None
        return st
    K, I, mode, gs = case["K"], case["I"], case["mode"], case["group_size"]
    st["x"] = torch.randn((T, K), generator=gen, device="cuda").to(dt)
    st["gate"] = _stack(gen, E, I, K, K ** -0.5, mode, gs, dt)
    st["up"] = _stack(gen, E, I, K, K ** -0.5, mode, gs, dt)
    st["down"] = _stack(gen, E, K, I, I ** -0.5, mode, gs, dt)
    # Experts as a router gives them: distinct per token, popularity ~ rank^-skew, random slots dropped.
    order = torch.randperm(E, generator=gen, device="cuda")
    pop = -case["skew"] * torch.log(1.0 + order.float())
    u = torch.rand((T, E), generator=gen, device="cuda").clamp_min(1e-6)
    val, idx = torch.topk(pop - torch.log(-torch.log(u)), k, dim=-1)
    drop = torch.rand((T, k), generator=gen, device="cuda") < case["dropped"]
    st["indices"] = torch.where(drop, -1, idx).to(torch.int32)
    st["weights"] = torch.softmax(val, -1)
    if own:
        from quantized_matmul_03_b200 import binding as qb
        n = qb.qmm_moe_experts_workspace_size(T, K, k, E, I, K, dt)
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms

def _e8m0(byte):
    return (byte.to(torch.int32) << 23).view(torch.float32)  # 2^(byte - 127), byte >= 1


def _dense(packed, e, mode, gs):
    """Expert e of a stack as a float32 matrix."""
    wq, s, b = packed
    by = wq[e].view(torch.uint8)
    codes = torch.stack([by & 15, by >> 4], -1).view(by.shape[0], -1)
    if mode == "affine":
        q = codes.float().view(codes.shape[0], -1, gs)
        w = s[e].float().unsqueeze(-1) * q + b[e].float().unsqueeze(-1)
    else:
        table = torch.tensor(E2M1, device=wq.device)
        x = _e8m0(s[e]) if mode == "mxfp4" else s[e].view(torch.float8_e4m3fn).float()
        w = x.unsqueeze(-1) * table[codes.int()].view(codes.shape[0], -1, gs)
    return w.view(codes.shape[0], -1)


def _plain_route(st):
    lg, T, E, k = st["logits"], st["T"], st["E"], st["k"]
    l = lg.double()
    if st["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    key = l if st["b"] is None else s + st["b"].double()
    G = st["n_groups"]
    if G > 1:
        gk = (s if st["b"] is None else key).view(T, G, E // G)
        top = torch.sort(gk, dim=-1, descending=True)[0][..., :st["group_top"]].sum(-1)
        keep = torch.sort(top, dim=-1, descending=True, stable=True)[1][:, :st["topk_groups"]]
        live = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        key = torch.where(live.unsqueeze(-1), key.view(T, G, E // G), -math.inf).view(T, E)
    idx = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(s, 1, idx)
    if st["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return {"indices": idx.to(torch.int32), "weights": (w * st["scale"]).float()}


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _plain_experts(st):
    x, T, k, E = st["x"], st["T"], st["k"], st["E"]
    flat = st["indices"].view(-1).long()
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(flat, stable=True)[1]
    counts = torch.bincount(flat, minlength=E + 1).tolist()
    w = st["weights"].view(-1, 1)
    out = torch.zeros((T * k, x.shape[1]), device=x.device)
    at = 0
    for e in range(E):
        rows = order[at:at + counts[e]]
        at += counts[e]
        if rows.numel() == 0:
            continue
        xe = x[rows // k].float()
        g = xe @ _dense(st["gate"], e, st["mode"], st["group_size"]).T
        u = xe @ _dense(st["up"], e, st["mode"], st["group_size"]).T
        h = _act(g, st["act"]) * u
        out[rows] = w[rows] * (h @ _dense(st["down"], e, st["mode"], st["group_size"]).T)
    return out.view(T, k, -1).sum(1).to(x.dtype)


def run(state):
    st = state
    if not own:
        return _plain_route(st) if st["op"] == "route" else _plain_experts(st)
    from quantized_matmul_03_b200 import binding as qb
    if st["op"] == "route":
        idx, w = qb.qmm_moe_route(st["logits"], st["k"], score=st["score"], bias=st["b"], n_groups=st["n_groups"],
                                  topk_groups=st["topk_groups"], group_top=st["group_top"],
                                  renormalize=st["renormalize"], scale=st["scale"])
        return {"indices": idx, "weights": w}
    return qb.qmm_moe_experts(st["x"], st["indices"], st["weights"], st["gate"], st["up"], st["down"],
                              group_size=st["group_size"], bits=4, mode=st["mode"], activation=st["act"],
                              workspace=st["workspace"])


# ---------------------------------------------------------------- accounting

def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * E * es + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    K, I, gs = case["K"], case["I"], case["group_size"]
    touched = E * (1 - (1 - k / E) ** T)  # experts that T tokens reach when all are equally popular
    per_group = 4 if case["mode"] == "affine" else 1
    weights = touched * 3 * K * I * (0.5 + per_group / gs)
    return {"bytes": int(weights) + 4 * T * K + 8 * T * k, "flops": 6 * T * k * K * I}


# ---------------------------------------------------------------- 64 bits

def _exact_route(st):
    l = st["logits"].cpu().double()
    if st["score"] == "softmax":
        s = torch.exp(l - torch.logsumexp(l, -1, keepdim=True))
    else:
        s = torch.sigmoid(l)
    k, G, E = st["k"], st["n_groups"], st["E"]
    sel = s + st["b"].cpu().double() if st["b"] is not None else s
    key = sel if st["b"] is not None else l
    if G > 1:
        best = torch.topk(sel.view(-1, G, E // G), st["group_top"], -1)[0].sum(-1)
        rank = torch.argsort(torch.argsort(-best, dim=-1, stable=True), dim=-1)
        key = key.masked_fill((rank >= st["topk_groups"]).repeat_interleave(E // G, 1), -math.inf)
    idx = torch.argsort(-key, dim=-1, stable=True)[:, :k]
    w = s.gather(1, idx)
    if st["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return {"indices": idx.to(torch.int32), "weights": w * st["scale"]}


def _exact_matrix(packed, e, mode, gs):
    wq, s, b = packed
    words = wq[e].to(torch.int64) & 0xFFFFFFFF
    codes = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], -1).view(words.shape[0], -1)
    if mode == "affine":
        scale = s[e].double().repeat_interleave(gs, 1)
        return scale * codes.double() + b[e].double().repeat_interleave(gs, 1)
    if mode == "mxfp4":
        values = [2.0 ** (i - 127) for i in range(256)]
    else:  # E4M3: bias 7, subnormals below 2^-6
        values = [(-1 if i & 128 else 1) * ((i & 7) / 8 * 2.0 ** -6 if (i >> 3) & 15 == 0 else
                                            (1 + (i & 7) / 8) * 2.0 ** (((i >> 3) & 15) - 7)) for i in range(256)]
    t = torch.tensor(values, dtype=torch.float64, device=wq.device)
    v = torch.tensor(E2M1, dtype=torch.float64, device=wq.device)
    return t[s[e].long()].repeat_interleave(gs, 1) * v[codes]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st)
    x, idx, w = st["x"].double(), st["indices"], st["weights"].double()
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        for j in range(case["k"]):
            t = torch.nonzero(idx[:, j] == e).view(-1)
            if t.numel() == 0:
                continue
            if j == 0 or "e" not in st or st["e"] != e:
                st["e"] = e
                st["m"] = [_exact_matrix(st[n], e, case["mode"], case["group_size"]) for n in ("gate", "up", "down")]
            wg, wu, wd = st["m"]
            a = x[t] @ wg.T
            a = a * torch.sigmoid(a) if case["act"] == "silu" else \
                torch.nn.functional.gelu(a, approximate="tanh")
            y.index_add_(0, t, w[t, j, None] * ((a * (x[t] @ wu.T)) @ wd.T))
    return y
