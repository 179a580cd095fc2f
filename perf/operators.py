"""Timed cases of the 16-bit MoE operators: rows sorted by expert and back with
their gradients, the grouped product with bias, activation, gate operand and
residual, its activation gradient and its two product gradients.

`prepare` makes what a program holds before the call, `run` makes one pass: the
plain form in elementary torch operations (32 bits, rounded once), or with
`own` set the library's calls.  `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SQRT_HALF = math.sqrt(0.5)
TANH_C = math.sqrt(2.0 / math.pi)

# the experts' product of a Mixtral-shaped layer at 4096 tokens: no case costs more
MOST_FLOPS = 2 * 8192 * 4096 * 14336
MOST_WEIGHTS = 8 * 4096 * 14336


def listed():
    return [
        # rows to the experts and back in one decoding step of a Mixtral-shaped layer
        dict(name="dispatch-decode", kind="dispatch", dtype="fp16", T=16, H=4096, E=8, k=2, S=0, zipf=0.0,
             renorm=True, drop=0.0),
        # the same layer reading a prompt of 4096 tokens
        dict(name="dispatch-prefill", kind="dispatch", dtype="bf16", T=4096, H=4096, E=8, k=2, S=0, zipf=0.0,
             renorm=True, drop=0.0),
        # backward pass of the dispatch of a DeepSeekMoE-shaped layer: skewed routing, two shared experts
        dict(name="dispatch-grad-shared", kind="dispatch_grad", dtype="bf16", T=8192, H=2048, E=64, k=6, S=2,
             zipf=1.2, renorm=False, drop=0.0),
        # the same in 32 bits at odd sizes, with pairs dropped (some tokens lose every expert)
        dict(name="dispatch-grad-dropped", kind="dispatch_grad", dtype="fp32", T=777, H=1003, E=5, k=2, S=0,
             zipf=0.0, renorm=True, drop=0.15),
        # one token through a dense output projection with bias and residual
        dict(name="linear-token", kind="linear", dtype="bf16", R=1, E=1, N=4096, K=14336, zipf=0.0, bias=True,
             act="none", mul=False, res=True, out="same", keep=False),
        # the gate product of every expert in one decoding step of 16 tokens, top 2 of 8
        dict(name="experts-decode", kind="linear", dtype="fp16", R=32, E=8, N=14336, K=4096, zipf=0.0, bias=False,
             act="silu", mul=True, res=False, out="same", keep=False),
        # the same product for a prompt of 4096 tokens, keeping what the backward pass needs
        dict(name="experts-prefill", kind="linear", dtype="bf16", R=8192, E=8, N=14336, K=4096, zipf=0.0,
             bias=False, act="silu", mul=True, res=False, out="same", keep=True),
        # the router's own product: 64 logits in 32 bits for each of 4096 tokens
        dict(name="gate-logits", kind="linear", dtype="fp16", R=4096, E=1, N=64, K=2048, zipf=0.0, bias=False,
             act="none", mul=False, res=False, out="fp32", keep=False),
        # gradients of the down product of eight experts, 2048 tokens, weight gradients in 32 bits
        dict(name="experts-grad", kind="linear_grad", dtype="bf16", R=4096, E=8, N=4096, K=14336, zipf=0.0,
             out="fp32"),
        # gradients of many small experts under skewed routing (some have no row)
        dict(name="experts-grad-ragged", kind="linear_grad", dtype="fp16", R=2048, E=66, N=1408, K=2048, zipf=1.2,
             out="same"),
        # gradient through the activation and the gate operand of a Mixtral-shaped layer
        dict(name="act-grad-gated", kind="act_grad", dtype="bf16", R=8192, E=8, N=14336, zipf=0.0, bias=False,
             act="silu", mul=True),
        # through a GELU with bias gradients, odd sizes
        dict(name="act-grad-bias", kind="act_grad", dtype="fp16", R=1031, E=6, N=1403, zipf=0.0, bias=True,
             act="gelu", mul=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; two in three are multiples of 8 where they can be."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 16 and rng.random() < 0.67:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["dispatch", "dispatch_grad", "linear", "linear", "linear_grad", "act_grad"])
    zipf = rng.choice([0.0, 0.0, 1.2])
    if kind in ("dispatch", "dispatch_grad"):
        E = rng.choice([2, 5, 8, 16, 64, 160])
        k = rng.randint(1, min(E, 8))
        S = rng.choice([0, 0, 1, 2])
        H = _spread(rng, 64, 8192)
        T = _spread(rng, 1, max(16, min(16384, (1 << 27) // (H * (k + S)))))
        return dict(kind=kind, dtype=rng.choice(["fp16", "bf16", "fp32"]), T=T, H=H, E=E, k=k, S=S, zipf=zipf,
                    renorm=rng.random() < 0.5, drop=rng.choice([0.0, 0.0, 0.1]))
    dtype = rng.choice(["fp16", "bf16"])
    E = rng.choice([1, 1, 3, 8, 16, 64])
    N = _spread(rng, 16, 16384)
    if kind == "act_grad":
        return dict(kind=kind, dtype=dtype, R=_spread(rng, 1, min(16384, (1 << 26) // N)), E=E, N=N, zipf=zipf,
                    bias=rng.random() < 0.5, act=rng.choice(["relu", "silu", "gelu", "gelu_tanh"]),
                    mul=rng.random() < 0.5)
    K = _spread(rng, 16, max(32, min(16384, MOST_WEIGHTS // (N * E))))
    R = _spread(rng, 1, max(2, min(16384, MOST_FLOPS // (8 * N * K))))
    case = dict(kind=kind, dtype=dtype, R=R, E=E, N=N, K=K, zipf=zipf, out=rng.choice(["same", "fp32"]))
    if kind == "linear":
        case.update(bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                    mul=rng.random() < 0.3, res=rng.random() < 0.5, keep=rng.random() < 0.3)
    return case


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


def _logits(gen, T, E, zipf):
    """Router logits N(0, 1), with the log of a shuffled Zipf distribution added where the routing is skewed."""
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if zipf:
        p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -zipf
        p = p[torch.randperm(E, generator=gen, device="cuda")]
        logits = logits + torch.log(p / p.sum())
    return logits


def _routing(gen, c):
    """Routing tables: logits, picked experts, slot weights and each pair's row in expert order (-1: dropped)."""
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits = _logits(gen, T, E, c["zipf"])
    top, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(logits, 1).gather(1, ids)
    if c["renorm"]:
        w = torch.softmax(top, 1)
    shared = torch.arange(E, E + S, device="cuda").expand(T, S)
    expert = torch.cat([ids, shared], 1).reshape(-1)
    slot_w = torch.cat([w, torch.ones((T, S), device="cuda")], 1).reshape(-1).contiguous()
    P = T * (k + S)
    dropped = int(c["drop"] * P)
    kept = torch.ones(P, dtype=torch.bool, device="cuda")
    kept[torch.randperm(P, generator=gen, device="cuda")[:dropped]] = False
    order = torch.argsort(torch.where(kept, expert, E + S), stable=True)
    pos = torch.empty(P, dtype=torch.int64, device="cuda")
    pos[order] = torch.arange(P, device="cuda")
    rows = P - dropped
    pos = torch.where(kept, pos, -1).to(torch.int32)
    return dict(logits=logits, ids=ids.to(torch.int32), slot_w=slot_w, pos=pos, rows=rows)


def _offsets(gen, c):
    """Rows of each expert: every row picks one (skewed where the case says so), as a device table and host bounds."""
    pick = _logits(gen, c["R"], c["E"], c["zipf"]).argmax(1)
    counts = torch.bincount(pick, minlength=c["E"])
    offsets = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, offsets.tolist()


def prepare(case, seed):
    c, gen = case, _gen(seed)
    dt = DTYPES[c["dtype"]]
    s = dict(case=c)
    if c["kind"] in ("dispatch", "dispatch_grad"):
        s.update(_routing(gen, c))
        T, H, R = c["T"], c["H"], s["rows"]
        s["y"] = _normal(gen, (R, H), 1.0, dt)
        if c["kind"] == "dispatch":
            s["x"] = _normal(gen, (T, H), 1.0, dt)
        else:
            s["dout"] = _normal(gen, (T, H), 0.1, dt)
            s["dxs"] = _normal(gen, (R, H), 0.1, dt)
        return s
    R, E, N = c["R"], c["E"], c["N"]
    if E > 1:
        s["offsets"], s["bounds"] = _offsets(gen, c)
    else:
        s["offsets"], s["bounds"] = None, [0, R]
    if c["kind"] == "act_grad":
        s["dy"] = _normal(gen, (R, N), 0.1, dt)
        s["pre"] = _normal(gen, (R, N), 1.3, dt)
        s["mul"] = _normal(gen, (R, N), 1.3, dt) if c["mul"] else None
        return s
    K = c["K"]
    s["x"] = _normal(gen, (R, K), 1.0, dt)
    s["w"] = torch.empty((E, N, K), dtype=dt, device="cuda")
    for e in range(E):
        s["w"][e] = _normal(gen, (N, K), 0.02, dt)
    if c["kind"] == "linear_grad":
        s["dy"] = _normal(gen, (R, N), 0.1, dt)
        return s
    s["bias"] = _normal(gen, (E, N), 0.1, dt) if c["bias"] else None
    s["mul"] = _normal(gen, (R, N), 1.0, dt) if c["mul"] else None
    s["res"] = _normal(gen, (R, N), 1.0, dt) if c["res"] else None
    return s


def _out_dtype(c):
    return torch.float32 if c["out"] == "fp32" else DTYPES[c["dtype"]]


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import extreme_quantized_moe_amd as m

    c = s["case"]
    if c["kind"] == "dispatch":
        slots = c["k"] + c["S"]
        xs = m.moe_permute(s["x"], s["pos"], slots, num_rows=s["rows"])
        return dict(xs=xs, out=m.moe_unpermute(s["y"], s["pos"], slots, s["slot_w"]))
    if c["kind"] == "dispatch_grad":
        slots = c["k"] + c["S"]
        dy, dw = m.moe_unpermute_grad(s["dout"], s["y"], s["pos"], slots, s["slot_w"])
        dlogits = m.route_grad(dw, s["logits"], s["ids"], c["S"], c["renorm"])
        return dict(dy=dy, dw=dw, dlogits=dlogits, dx=m.moe_permute_grad(s["dxs"], s["pos"], slots))
    if c["kind"] == "linear":
        got = m.moe_linear(s["x"], s["w"], offsets=s["offsets"], bias=s["bias"], activation=c["act"], mul=s["mul"],
                           residual=s["res"], out_dtype=_out_dtype(c), return_pre=c["keep"])
        return dict(y=got[0], pre=got[1]) if c["keep"] else dict(y=got)
    if c["kind"] == "linear_grad":
        dx, dw = m.moe_linear_grad(s["dy"], s["x"], s["w"], offsets=s["offsets"], dw_dtype=_out_dtype(c))
        return dict(dx=dx, dw=dw)
    dpre, dmul, dbias = m.moe_linear_act_grad(s["dy"], s["pre"], c["act"], mul=s["mul"], offsets=s["offsets"],
                                              bias_grad=c["bias"])
    return {n: t for n, t in (("dpre", dpre), ("dmul", dmul), ("dbias", dbias)) if t is not None}


def _act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * SQRT_HALF))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(TANH_C * (v + 0.044715 * v * v * v)))
    return v


def _act_slope(name, v):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        g = 1 / (1 + torch.exp(-v))
        return g * (1 + v * (1 - g))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * SQRT_HALF)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(TANH_C * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * TANH_C * (1 + 3 * 0.044715 * v * v)
    return torch.ones_like(v)


def _run_plain(s):
    c = s["case"]
    f = torch.float32
    dt = DTYPES[c["dtype"]]
    if c["kind"] == "dispatch":
        T, H, slots = c["T"], c["H"], c["k"] + c["S"]
        pos, kept = s["pos"].long(), s["pos"] >= 0
        token = torch.arange(T, device="cuda").repeat_interleave(slots)
        dest = torch.where(kept, pos, s["rows"])          # dropped pairs go to one spare row
        xs = torch.empty((s["rows"] + 1, H), dtype=dt, device="cuda")
        xs[dest] = s["x"][token]
        w = torch.where(kept, s["slot_w"], 0.0)
        terms = s["y"][pos.clamp(min=0)].to(f) * w[:, None]
        return dict(xs=xs[:-1], out=terms.view(T, slots, H).sum(1).to(dt))
    if c["kind"] == "dispatch_grad":
        T, H, k, slots = c["T"], c["H"], c["k"], c["k"] + c["S"]
        pos, kept = s["pos"].long(), s["pos"] >= 0
        at = pos.clamp(min=0)
        dout = s["dout"].to(f).repeat_interleave(slots, 0)
        dest = torch.where(kept, pos, s["rows"])
        dy = torch.empty((s["rows"] + 1, H), dtype=dt, device="cuda")
        dy[dest] = (dout * s["slot_w"][:, None]).to(dt)
        dw = torch.where(kept, (dout * s["y"][at].to(f)).sum(1), 0.0)
        dx = (s["dxs"][at].to(f) * kept[:, None]).view(T, slots, H).sum(1).to(dt)
        g, ids, l = dw.view(T, slots)[:, :k], s["ids"].long(), s["logits"]
        e = torch.exp(l - l.amax(1, keepdim=True))
        if c["renorm"]:
            e = torch.zeros_like(e).scatter(1, ids, e.gather(1, ids))
        p = e / e.sum(1, keepdim=True)
        wide = torch.zeros_like(l).scatter(1, ids, g)
        dlogits = p * (wide - (p * wide).sum(1, keepdim=True))
        return dict(dy=dy[:-1], dw=dw, dlogits=dlogits, dx=dx)
    spans = [(e, a, b) for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:]))]
    if c["kind"] == "linear":
        y = torch.empty((c["R"], c["N"]), dtype=_out_dtype(c), device="cuda")
        pre = torch.empty((c["R"], c["N"]), dtype=dt, device="cuda") if c["keep"] else None
        for e, a, b in spans:
            if a == b:
                continue
            v = s["x"][a:b].to(f) @ s["w"][e].to(f).t()
            if c["bias"]:
                v = v + s["bias"][e].to(f)
            if c["keep"]:
                pre[a:b] = v.to(dt)
            v = _act(c["act"], v)
            if c["mul"]:
                v = v * s["mul"][a:b].to(f)
            if c["res"]:
                v = v + s["res"][a:b].to(f)
            y[a:b] = v.to(y.dtype)
        return dict(y=y, pre=pre) if c["keep"] else dict(y=y)
    if c["kind"] == "linear_grad":
        dx = torch.empty((c["R"], c["K"]), dtype=dt, device="cuda")
        dw = torch.empty((c["E"], c["N"], c["K"]), dtype=_out_dtype(c), device="cuda")
        for e, a, b in spans:
            d = s["dy"][a:b].to(f)
            if a < b:
                dx[a:b] = (d @ s["w"][e].to(f)).to(dt)
                dw[e] = (d.t() @ s["x"][a:b].to(f)).to(dw.dtype)
            else:
                dw[e] = 0
        return dict(dx=dx, dw=dw)
    dy, v = s["dy"].to(f), s["pre"].to(f)
    slope = dy * _act_slope(c["act"], v)
    out = {}
    if c["mul"]:
        slope = slope * s["mul"].to(f)
        out["dmul"] = (dy * _act(c["act"], v)).to(dt)
    out["dpre"] = slope.to(dt)
    if c["bias"]:
        out["dbias"] = torch.stack([slope[a:b].sum(0) for _, a, b in spans])
    return out


# ------------------------------------------------------------------ cost

def work(case):
    """What one pass cannot do without: each input read once, each output written once, the products' operations."""
    c = case
    es = 4 if c["dtype"] == "fp32" else 2
    if c["kind"] in ("dispatch", "dispatch_grad"):
        P = c["T"] * (c["k"] + c["S"])
        rows = P - int(c["drop"] * P)
        T, H = c["T"], c["H"]
        if c["kind"] == "dispatch":                        # x, y in; xs, out out; positions and weights
            return dict(bytes=2 * es * H * (T + rows) + 8 * P, flops=2 * rows * H)
        # dout, y, dxs in; dy, dx out; positions, weights and their gradients, logits and theirs, picked experts
        return dict(bytes=es * H * (2 * T + 3 * rows) + 12 * P + 8 * T * c["E"] + 4 * T * c["k"],
                    flops=4 * rows * H + 8 * T * c["E"])
    R, E, N = c["R"], c["E"], c["N"]
    if c["kind"] == "act_grad":
        n = 5 if c["mul"] else 3                           # dy, pre (and mul) in, dpre (and dmul) out
        return dict(bytes=n * es * R * N + (4 * E * N if c["bias"] else 0), flops=12 * R * N)
    K = c["K"]
    outs = 4 if c["out"] == "fp32" else es
    used = E * (1 - (1 - 1 / E) ** R) if E > 1 else 1      # experts that some row picks
    if c["kind"] == "linear":
        rows = es * R * K + outs * R * N + es * R * N * (c["mul"] + c["res"] + c["keep"])
        return dict(bytes=int(rows + es * used * N * K + (es * E * N if c["bias"] else 0)), flops=2 * R * N * K)
    return dict(bytes=int(es * R * (N + 2 * K) + es * used * N * K + outs * E * N * K), flops=4 * R * N * K)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The same outputs from their definitions in float64, pair by slot and expert by expert."""
    s, c = prepare(case, seed), case
    d = torch.float64
    if c["kind"] == "dispatch":
        slots, pos = c["k"] + c["S"], s["pos"].view(c["T"], -1).long()
        xs = torch.zeros((s["rows"], c["H"]), dtype=d, device="cuda")
        out = torch.zeros((c["T"], c["H"]), dtype=d, device="cuda")
        w = s["slot_w"].view(c["T"], -1).to(d)
        for j in range(slots):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            xs[pos[t, j]] = s["x"][t].to(d)
            out[t] += w[t, j, None] * s["y"][pos[t, j]].to(d)
        return dict(xs=xs, out=out)
    if c["kind"] == "dispatch_grad":
        T, k, slots, pos = c["T"], c["k"], c["k"] + c["S"], s["pos"].view(c["T"], -1).long()
        dy = torch.zeros((s["rows"], c["H"]), dtype=d, device="cuda")
        dx = torch.zeros((T, c["H"]), dtype=d, device="cuda")
        dw = torch.zeros((T, slots), dtype=d, device="cuda")
        w = s["slot_w"].view(T, -1).to(d)
        for j in range(slots):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            r = pos[t, j]
            dy[r] = w[t, j, None] * s["dout"][t].to(d)
            dw[t, j] = (s["dout"][t].to(d) * s["y"][r].to(d)).sum(1)
            dx[t] += s["dxs"][r].to(d)
        ids, l = s["ids"].long(), s["logits"].to(d)
        dl = torch.zeros_like(l)
        if c["renorm"]:
            p = torch.softmax(l.gather(1, ids), 1)
            dl.scatter_(1, ids, p * (dw[:, :k] - (p * dw[:, :k]).sum(1, keepdim=True)))
        else:
            p = torch.softmax(l, 1)
            pk = p.gather(1, ids)
            dl -= p * (pk * dw[:, :k]).sum(1, keepdim=True)
            dl.scatter_add_(1, ids, pk * dw[:, :k])
        return dict(dy=dy, dw=dw.view(-1), dlogits=dl, dx=dx)
    if c["kind"] == "act_grad":
        dy = s["dy"].to(d)
        v = s["pre"].to(d).requires_grad_(True)
        a = _exact_act(c["act"], v)
        slope, = torch.autograd.grad(a.sum(), v)
        out = {}
        g = dy * slope
        if c["mul"]:
            g = g * s["mul"].to(d)
            out["dmul"] = dy * a.detach()
        out["dpre"] = g
        if c["bias"]:
            out["dbias"] = torch.stack([g[a0:b0].sum(0) for a0, b0 in zip(s["bounds"], s["bounds"][1:])])
        return out
    got = []
    for e in range(c["E"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        w, x = s["w"][e].to(d), s["x"][a:b].to(d)
        if c["kind"] == "linear_grad":
            g = s["dy"][a:b].to(d)
            got.append((torch.mm(g, w), torch.mm(g.t().contiguous(), x)))
            continue
        v = torch.mm(x, w.t().contiguous())
        if c["bias"]:
            v += s["bias"][e].to(d)
        y = _exact_act(c["act"], v)
        if c["mul"]:
            y = y * s["mul"][a:b].to(d)
        if c["res"]:
            y = y + s["res"][a:b].to(d)
        got.append((y, v))
    if c["kind"] == "linear_grad":
        return dict(dx=torch.cat([g[0] for g in got]), dw=torch.stack([g[1] for g in got]))
    y = torch.cat([g[0] for g in got])
    return dict(y=y, pre=torch.cat([g[1] for g in got])) if c["keep"] else dict(y=y)


def _exact_act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v * SQRT_HALF)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * TANH_C * (v + 0.044715 * v ** 3))
    return v
