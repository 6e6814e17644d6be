"""Measured calls of the few-token operators on 4-bit weights: a decoding step's linear layers.

Three operators, in the order a decoding step uses them:

  gemv   y = W T x for a few tokens: 4-bit weights with group scales (MXFP4, NVFP4, INT4) against 16-bit
         activations that get their blockwise transform on the way
  route  the router of a mixture-of-experts layer: softmax over the experts, the top ones and their weights
  moe    the whole mixture-of-experts layer on 4-bit experts (router, gate and up, SiLU, down, weighted sum),
         and its form for routing that the caller brings along (some slots dropped)

``run`` computes them in plain torch operations, or through the package where ``own`` is true.
"""
import math

import torch

own = False

LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the smallest call: a narrow projection of one token, where only latency counts
        dict(name="gemv int4 g16 256x256 n1", op="gemv", fmt="int4", G=16, n=1, d_out=256, d_in=256, T="none",
             f32=False),
        # one token through a square attention projection, transforms per block (the headline layer's sizes)
        dict(name="gemv mxfp4 4096x4096 n1", op="gemv", fmt="mxfp4", G=32, n=1, d_out=4096, d_in=4096, T="block",
             f32=False),
        # a down projection (the NVFP4 workload's sizes) for three sequences at once
        dict(name="gemv nvfp4 4096x14336 n3", op="gemv", fmt="nvfp4", G=16, n=3, d_out=4096, d_in=14336, T="block",
             f32=False),
        # an odd number of output rows, one Hadamard matrix shared by all blocks, a small decoding batch
        dict(name="gemv int4 g32 8197x5120 n8", op="gemv", fmt="int4", G=32, n=8, d_out=8197, d_in=5120, T="shared",
             f32=False),
        # an output head: many rows, fp32 logits, no transform
        dict(name="gemv mxfp4 65537x4096 n1 f32", op="gemv", fmt="mxfp4", G=32, n=1, d_out=65537, d_in=4096,
             T="none", f32=True),
        # the widest layer of the per-layer benchmark under a decoding batch of 16
        dict(name="gemv mxfp4 57344x8192 n16", op="gemv", fmt="mxfp4", G=32, n=16, d_out=57344, d_in=8192,
             T="block", f32=False),
        # routing one token among many experts
        dict(name="route 1x4096 e64 k8", op="route", n=1, d=4096, E=64, k=8, f32=False, renorm=True),
        # routing a batch: odd token count, fp32 router weights, plain softmax weights
        dict(name="route 129x8192 e256 k8 f32", op="route", n=129, d=8192, E=256, k=8, f32=True, renorm=False),
        # the smallest layer
        dict(name="moe int4 n1 e8 k2 256x128", op="moe", fmt="int4", G=32, n=1, E=8, k=2, d=256, f=128, T="block",
             renorm=True, drop=False),
        # one token through many narrow experts
        dict(name="moe mxfp4 n1 e64 k8 2048x1024", op="moe", fmt="mxfp4", G=32, n=1, E=64, k=8, d=2048, f=1024,
             T="block", renorm=True, drop=False),
        # three tokens through few wide experts
        dict(name="moe nvfp4 n3 e8 k2 4096x14336", op="moe", fmt="nvfp4", G=16, n=3, E=8, k=2, d=4096, f=14336,
             T="block", renorm=True, drop=False),
        # a decoding batch whose routing is given, a tenth of its slots dropped by a capacity limit
        dict(name="moe mxfp4 n32 e64 k4 4096x1536", op="moe", fmt="mxfp4", G=32, n=32, E=64, k=4, d=4096, f=1536,
             T="block", renorm=True, drop=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _format(rng):
    return rng.choice((("mxfp4", 32), ("nvfp4", 16), ("int4", 16), ("int4", 32)))


def draw(rng):
    op = rng.choice(("gemv", "gemv", "route", "moe", "moe"))
    if op == "route":
        E = _log(rng, 2, 256)
        return dict(op=op, n=_log(rng, 1, 129), d=8 * _log(rng, 8, 1024), E=E, k=rng.randint(1, min(8, E)),
                    f32=rng.random() < 0.5, renorm=rng.random() < 0.5)
    fmt, G = _format(rng)
    T = rng.choice(("block", "shared", "none"))
    if op == "gemv":
        while True:
            c = dict(op=op, fmt=fmt, G=G, n=_log(rng, 1, 16), d_out=_log(rng, 32, 65537),
                     d_in=G * _log(rng, 64 / G, 14336 / G), T=T, f32=rng.random() < 0.3)
            if c["d_out"] * c["d_in"] <= 57344 * 8192:
                return c
    while True:
        E = _log(rng, 2, 128)
        c = dict(op=op, fmt=fmt, G=G, n=_log(rng, 1, 32), E=E, k=rng.randint(1, min(8, E)),
                 d=G * _log(rng, 128 / G, 4096 / G), f=G * _log(rng, 64 / G, 14336 / G), T=T,
                 renorm=rng.random() < 0.5, drop=rng.random() < 0.3)
        experts, slots = c["E"] * c["d"] * c["f"], c["n"] * c["k"] * c["d"] * c["f"]
        if experts <= 64 * 4096 * 1536 and slots <= 128 * 4096 * 1536:
            return c


# ---------------------------------------------------------------- inputs

def _quantised(w, fmt, G):
    """AbsMax round-to-nearest of fp32 w [..., K]: (codes u8 [..., K/2], scales [..., K/G], tensor scale)."""
    g = w.reshape(*w.shape[:-1], w.shape[-1] // G, G)
    amax = g.abs().amax(-1)
    ts = None
    if fmt == "int4":
        scales = (amax / 7).clamp_min(1e-30)
        q = (g / scales[..., None]).round().clamp(-7, 7).to(torch.int32) & 15
    else:
        if fmt == "mxfp4":
            e = torch.ceil(torch.log2((amax / 6).clamp_min(2.0 ** -120)))
            scales, value = (e + 127).to(torch.uint8), torch.exp2(e)
        else:
            ts = amax.amax().reshape(1) / 2688
            s = (amax / (6 * ts)).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
            scales, value = s.view(torch.uint8), s.float() * ts
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
        v = g / value[..., None]
        q = torch.bucketize(v.abs(), edges, out_int32=True) | ((v < 0).to(torch.int32) << 3)
    q = q.reshape(*w.shape[:-1], w.shape[-1] // 2, 2)
    return (q[..., 0] | (q[..., 1] << 4)).to(torch.uint8), scales.contiguous(), ts


def _weights(gen, E, rows, K, fmt, G):
    """E quantised matrices [rows][K], some rows larger than others; made a slab at a time."""
    codes = torch.empty((E, rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, rows, K // G), dtype=torch.float32 if fmt == "int4" else torch.uint8, device="cuda")
    ts = torch.empty(E, device="cuda") if fmt == "nvfp4" else None
    step = rows if fmt == "nvfp4" else max(1, (1 << 27) // K)
    for e in range(E):
        for r in range(0, rows, step):
            m = min(step, rows - r)
            w = torch.randn((m, K), generator=gen, device="cuda")
            w *= torch.exp(0.5 * torch.randn((m, 1), generator=gen, device="cuda")) * K ** -0.5
            codes[e, r:r + m], scales[e, r:r + m], t = _quantised(w, fmt, G)
            if t is not None:
                ts[e] = t[0]
    return codes, scales, ts


def _tokens(gen, n, d):
    """bf16 activations with a spread of channel sizes and a few outlier channels."""
    x = torch.randn((n, d), generator=gen, device="cuda") * torch.exp(torch.randn(d, generator=gen, device="cuda"))
    hot = torch.randperm(d, generator=gen, device="cuda")[: max(1, d // 200)]
    x[:, hot] *= 30
    return x.to(torch.bfloat16)


def _transforms(gen, kind, d, G):
    if kind == "none":
        return None
    if kind == "shared":
        i = torch.arange(G)
        ones = sum(((i[:, None] & i[None, :]) >> b) & 1 for b in range(5))
        return ((1 - 2 * (ones & 1)).float() / G ** 0.5).cuda()
    return torch.eye(G, device="cuda") + 0.1 * torch.randn((d // G, G, G), generator=gen, device="cuda")


def _router(gen, E, d):
    return torch.randn((E, d), generator=gen, device="cuda") * (2.0 / d ** 0.5)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "gemv":
        s["x"] = _tokens(gen, c["n"], c["d_in"])
        s["T"] = _transforms(gen, c["T"], c["d_in"], c["G"])
        codes, scales, s["ts"] = _weights(gen, 1, c["d_out"], c["d_in"], c["fmt"], c["G"])
        s["codes"], s["scales"] = codes[0], scales[0]
    elif c["op"] == "route":
        s["x"] = torch.randn((c["n"], c["d"]), generator=gen, device="cuda").to(torch.bfloat16)
        r = _router(gen, c["E"], c["d"])
        s["router"] = r if c["f32"] else r.to(torch.bfloat16)
    else:
        s["x"] = torch.randn((c["n"], c["d"]), generator=gen, device="cuda").to(torch.bfloat16)
        s["router"] = _router(gen, c["E"], c["d"]).to(torch.bfloat16)
        s["T_in"] = _transforms(gen, c["T"], c["d"], c["G"])
        s["T_out"] = _transforms(gen, c["T"], c["f"], c["G"])
        s["w_in"] = _weights(gen, c["E"], 2 * c["f"], c["d"], c["fmt"], c["G"])
        s["w_out"] = _weights(gen, c["E"], c["d"], c["f"], c["fmt"], c["G"])
        if c["drop"]:
            p = torch.softmax(s["x"].float() @ s["router"].float().T, -1)
            w, ids = torch.topk(p, c["k"])
            lost = torch.rand(ids.shape, generator=gen, device="cuda") < 0.1
            s["ids"] = torch.where(lost, -1, ids).to(torch.int32)
            s["weights"] = (w / w.sum(-1, keepdim=True)).contiguous()
    return s


# ---------------------------------------------------------------- plain forms

def _values(codes, scales, ts, G, fmt):
    """fp32 values of codes [..., K/2] under scales [..., K/G] and tensor scales [...] (or none)."""
    if fmt == "int4":
        table = torch.arange(16, device="cuda").float()
        table = torch.where(table > 7, table - 16, table)
        s = scales
    else:
        half = torch.tensor(LUT, device="cuda")
        table = torch.cat((half, -half))
        s = torch.exp2(scales.float() - 127) if fmt == "mxfp4" else scales.view(torch.float8_e4m3fn).float()
    if ts is not None:
        s = s * ts[..., None, None] if codes.dim() == 3 else s * ts
    byte = torch.arange(256, device="cuda")
    pairs = torch.stack((table[byte & 15], table[byte >> 4]), -1)
    v = pairs[codes.int()].reshape(*codes.shape[:-1], -1, G)
    return (v * s[..., None]).flatten(-2)


def _transformed(x, T, G):
    """fp32 blockwise T x of x [n][d]."""
    x = x.float()
    if T is None:
        return x
    b = x.reshape(x.shape[0], -1, G)
    return (torch.einsum("brc,nbc->nbr", T, b) if T.dim() == 3 else b @ T.T).flatten(-2)


def _routed(x, router, k, renorm):
    logits = x.double() @ router.double().T
    order = torch.sort(logits, dim=-1, descending=True, stable=True)   # ties keep the lower index first
    p = torch.softmax(logits, -1).gather(-1, order.indices[:, :k])
    if renorm:
        p = p / p.sum(-1, keepdim=True)
    return order.indices[:, :k].to(torch.int32), p.float()


def _experts(x, ids, weights, T_in, w_in, T_out, w_out, G, fmt):
    n, k = ids.shape
    e = ids.clamp_min(0).flatten().long()
    pick = lambda w: (w[0][e], w[1][e], None if w[2] is None else w[2][e])
    y = _transformed(x, T_in, G).repeat_interleave(k, 0)
    gate, up = torch.bmm(_values(*pick(w_in), G, fmt), y[..., None])[..., 0].chunk(2, -1)
    h = gate / (1 + torch.exp(-gate)) * up
    o = torch.bmm(_values(*pick(w_out), G, fmt), _transformed(h, T_out, G)[..., None])[..., 0]
    w = torch.where(ids < 0, 0.0, weights).flatten()
    return (o * w[:, None]).reshape(n, k, -1).sum(1)


def run(state):
    c, s = state["case"], state
    if c["op"] == "gemv":
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        if own:
            import blockwise_adaptive_transforms_b200 as W
            return W.wush_gemv(s["x"], s["T"], s["codes"], s["scales"], s["ts"], c["G"], c["fmt"], out_dtype=dtype)
        return (_transformed(s["x"], s["T"], c["G"])
                @ _values(s["codes"], s["scales"], s["ts"], c["G"], c["fmt"]).T).to(dtype)
    if c["op"] == "route":
        if own:
            import blockwise_adaptive_transforms_b200 as W
            return W.wush_moe_route(s["x"], s["router"], c["k"], renormalise=c["renorm"])
        return _routed(s["x"], s["router"], c["k"], c["renorm"])
    if c["drop"]:
        if own:
            import blockwise_adaptive_transforms_b200 as W
            return W.wush_moe_experts(s["x"], s["ids"], s["weights"], s["T_in"], s["w_in"], s["T_out"], s["w_out"],
                                      c["G"], c["fmt"])
        return _experts(s["x"], s["ids"], s["weights"], s["T_in"], s["w_in"], s["T_out"], s["w_out"], c["G"],
                        c["fmt"]).to(torch.bfloat16)
    if own:
        import blockwise_adaptive_transforms_b200 as W
        return W.wush_moe_layer(s["x"], s["router"], c["k"], s["T_in"], s["w_in"], s["T_out"], s["w_out"], c["G"],
                                c["fmt"], renormalise=c["renorm"])
    ids, weights = _routed(s["x"], s["router"], c["k"], c["renorm"])
    y = _experts(s["x"], ids, weights, s["T_in"], s["w_in"], s["T_out"], s["w_out"], c["G"], c["fmt"])
    return y.to(torch.bfloat16), ids, weights


# ---------------------------------------------------------------- the definition in 64 bits

def _decode64(codes, scales, ts, G, fmt):
    """Values of one matrix's rows, from the formats' definitions."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int64)
    if fmt == "int4":
        v = ((q ^ 8) - 8).double()
    else:
        e, m = (q >> 1) & 3, q & 1
        mag = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * 2.0 ** (e.double() - 1))
        v = torch.where(q >= 8, -mag, mag)
    if fmt == "int4":
        s = scales.double()
    elif fmt == "mxfp4":
        s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), scales.double() - 127)
    else:
        b = scales.to(torch.int64)
        e, m = (b >> 3) & 15, (b & 7).double()
        s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7)) * ts.double()
    return v * s.repeat_interleave(G, -1)


def _times64(y, codes, scales, ts, G, fmt):
    """y [n][K] against one matrix, a slab of rows at a time."""
    step = max(1, (1 << 26) // y.shape[-1])
    return torch.cat([y @ _decode64(codes[r:r + step], scales[r:r + step], ts, G, fmt).T
                      for r in range(0, codes.shape[0], step)], -1)


def _blocks64(x, T, G):
    x = x.double()
    if T is None:
        return x
    out = torch.empty_like(x)
    T = T.double()
    for b in range(x.shape[1] // G):
        out[:, b * G:(b + 1) * G] = x[:, b * G:(b + 1) * G] @ (T if T.dim() == 2 else T[b]).T
    return out


def _route64(x, router, k, renorm):
    logits = (x.double()[:, None, :] * router.double()).sum(-1) if x.shape[0] * router.numel() < 1 << 27 else \
        x.double() @ router.double().T
    rows, ids = logits.tolist(), []
    for row in rows:
        ids.append(sorted(range(len(row)), key=lambda i: (-row[i], i))[:k])
    ids = torch.tensor(ids, device="cuda")
    top = logits.gather(-1, ids)
    high = logits.max(-1, keepdim=True).values
    e = torch.exp(top - high)
    return ids.to(torch.int32), e / (e.sum(-1, keepdim=True) if renorm else
                                     torch.exp(logits - high).sum(-1, keepdim=True))


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "gemv":
        return _times64(_blocks64(s["x"], s["T"], c["G"]), s["codes"], s["scales"], s["ts"], c["G"], c["fmt"])
    if c["op"] == "route":
        return _route64(s["x"], s["router"], c["k"], c["renorm"])
    ids, weights = (s["ids"], s["weights"].double()) if c["drop"] else \
        _route64(s["x"], s["router"], c["k"], c["renorm"])
    y = _blocks64(s["x"], s["T_in"], c["G"])
    out = torch.zeros_like(y)
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        t, j = (ids == e).nonzero(as_tuple=True)
        mat = lambda w: (w[0][e], w[1][e], None if w[2] is None else w[2][e], c["G"], c["fmt"])
        gu = _times64(y[t], *mat(s["w_in"]))
        gate, up = gu[:, :c["f"]], gu[:, c["f"]:]
        h = gate * torch.sigmoid(gate) * up
        out.index_add_(0, t, _times64(_blocks64(h, s["T_out"], c["G"]), *mat(s["w_out"])) * weights[t, j][:, None])
    return out if c["drop"] else (out, ids, weights)


# ---------------------------------------------------------------- what a pass cannot do without

def _matrix_bytes(rows, K, fmt, G):
    return rows * (K // 2 + K // G * (4 if fmt == "int4" else 1)) + (4 if fmt == "nvfp4" else 0)


def _T_bytes(kind, d, G):
    return {"none": 0, "shared": G * G * 4, "block": d * G * 4}[kind]


def work(case):
    c = dict(case)
    n = c["n"]
    if c["op"] == "gemv":
        b = _matrix_bytes(c["d_out"], c["d_in"], c["fmt"], c["G"]) + _T_bytes(c["T"], c["d_in"], c["G"])
        b += n * (2 * c["d_in"] + c["d_out"] * (4 if c["f32"] else 2))
        f = 2 * n * c["d_in"] * c["d_out"] + (0 if c["T"] == "none" else 2 * n * c["d_in"] * c["G"])
        return {"bytes": b, "flops": f}
    k, E, d = c["k"], c["E"], c["d"]
    route = {"bytes": 2 * n * d + E * d * (4 if c.get("f32") else 2) + 8 * n * k, "flops": 2 * n * E * d}
    if c["op"] == "route":
        return route
    f = c["f"]
    # experts that at least one token is expected to choose: only their weights are read
    slots = 0.9 if c["drop"] else 1.0
    active = E * (1 - (1 - slots * k / E) ** n)
    b = active * (_matrix_bytes(2 * f, d, c["fmt"], c["G"]) + _matrix_bytes(d, f, c["fmt"], c["G"]))
    b += _T_bytes(c["T"], d, c["G"]) + _T_bytes(c["T"], f, c["G"]) + 4 * n * d + 8 * n * k
    fl = slots * n * k * 6 * d * f
    if c["T"] != "none":
        fl += 2 * n * d * c["G"] + slots * n * k * 2 * f * c["G"]
    if not c["drop"]:
        b, fl = b + 2 * E * d, fl + route["flops"]
    return {"bytes": b, "flops": fl}
