"""Cases of the few-token operators: the expert layer for a few tokens (bf16 and
4-bit weights), the 4-bit matrix-vector product, the router's top-k, and the
4-bit group quantisation.

4-bit weights are row-major codes q [N, K/2] uint8 (the even column of a pair in
the low nibble) with one bf16 scale, and optionally one zero point (uint8,
0..15; 8 where there is none), for each group of G columns:
w[n, k] = (q[n, k] - zero[n, k // G]) * scale[n, k // G].
"""
import math

import torch

own = False  # False: plain torch forms; True: the package's operators


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one token through all experts of a mid-sized layer: a decode step of one request
        dict(name="moe bf16 T1", op="moe", T=1, H=2048, I=1024, E=64, El=64, rank=0, K=6, fmt="bf16", group=0,
             zeros=False, routing="uniform", unrouted=0.0, out="bf16"),
        # one rank's share of a large layer: a decode batch whose routing is skewed towards this rank
        dict(name="moe bf16 T64 rank 0 of 8", op="moe", T=64, H=7168, I=2048, E=256, El=32, rank=0, K=8, fmt="bf16",
             group=0, zeros=False, routing="zipf", unrouted=0.0, out="bf16"),
        # a full decode batch that touches every expert
        dict(name="moe bf16 T128", op="moe", T=128, H=4096, I=1536, E=128, El=128, rank=0, K=8, fmt="bf16", group=0,
             zeros=False, routing="uniform", unrouted=0.0, out="bf16"),
        # one token through a large layer whose 4-bit experts are all on this GPU
        dict(name="moe int4 T1", op="moe", T=1, H=7168, I=2048, E=256, El=256, rank=0, K=8, fmt="int4", group=128,
             zeros=False, routing="uniform", unrouted=0.0, out="bf16"),
        # a small ragged batch on one rank of four, odd sizes, masked slots, zero points, fp32 partial sums
        dict(name="moe int4 T13 rank 1 of 4", op="moe", T=13, H=4160, I=1472, E=128, El=32, rank=1, K=8, fmt="int4",
             group=64, zeros=True, routing="uniform", unrouted=0.05, out="fp32"),
        # a square projection of one token: nothing but latency
        dict(name="matvec M1 2048x2048", op="matvec", M=1, N=2048, K=2048, group=128, zeros=False, out="bf16"),
        # the output projection of one token over a vocabulary, odd row count
        dict(name="matvec M1 50021x7168", op="matvec", M=1, N=50021, K=7168, group=128, zeros=False, out="bf16"),
        # a projection of a small batch, fine groups with zero points
        dict(name="matvec M24 7168x4096", op="matvec", M=24, N=7168, K=4096, group=32, zeros=True, out="fp32"),
        # the routing of one token over many experts
        dict(name="router T1 E256", op="router", T=1, H=7168, E=256, K=8, scoring="sigmoid", bias=True, norm=True),
        # the routing of a batch of tokens
        dict(name="router T200 E64", op="router", T=200, H=2048, E=64, K=6, scoring="softmax", bias=False, norm=False),
        # laying out one expert's matrix, odd row count, zero points
        dict(name="quantize 1031x2080", op="quantize", N=1031, K=2080, group=32, zeros=True),
        # laying out one rank's experts at load time
        dict(name="quantize 98304x4096", op="quantize", N=98304, K=4096, group=128, zeros=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["moe", "moe", "moe", "matvec", "matvec", "router", "quantize"])
    if op == "moe":
        fmt = rng.choice(["bf16", "int4"])
        group = rng.choice([32, 64, 128]) if fmt == "int4" else 0
        while True:
            K = rng.randint(1, 8)
            P = rng.choice([1, 1, 2, 4, 8])
            El = max(1, _log_int(rng, 8, 256) // P)
            T = _log_int(rng, 1, 128)
            m = group or 8
            H, I = _step(_log_int(rng, 256, 7168), m), _step(_log_int(rng, 128, 2048), m)
            c = dict(op="moe", T=T, H=H, I=I, E=P * El, El=El, rank=rng.randrange(P), K=min(K, P * El), fmt=fmt,
                     group=group, zeros=bool(group) and rng.random() < 0.5, routing=rng.choice(["uniform", "zipf"]),
                     unrouted=rng.choice([0.0, 0.0, 0.1]) if T > 4 else 0.0, out=rng.choice(["bf16", "fp32"]))
            # no larger than the largest listed case, and hardly ever a batch with nothing for this rank
            if El * 3 * H * I <= 2_400_000_000 and work(c)["flops"] >= 6.0 * H * I * (1 if P == 1 else 8):
                return c
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        return dict(op="matvec", M=_log_int(rng, 1, 64), N=_log_int(rng, 256, 50000),
                    K=_step(_log_int(rng, 256, 7168), group), group=group, zeros=rng.random() < 0.5,
                    out=rng.choice(["bf16", "fp32"]))
    if op == "router":
        E = _log_int(rng, 8, 256)
        return dict(op="router", T=_log_int(rng, 1, 256), H=_step(_log_int(rng, 256, 7168), 8), E=E,
                    K=rng.randint(1, min(8, E)), scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    norm=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    return dict(op="quantize", N=_log_int(rng, 64, 60000), K=_step(_log_int(rng, 256, 4096), group), group=group,
                zeros=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --
def _randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)


def _codes(rows, cols, g):
    """Bell-shaped 4-bit codes of a rows x cols matrix, two to a byte."""
    out = torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda")
    for r in range(0, rows, 32768):
        n = min(32768, rows - r)
        v = torch.randn((n, cols), generator=g, device="cuda").mul_(2.6).add_(8.0).round_().clamp_(0, 15)
        v = v.to(torch.uint8).view(n, cols // 2, 2)
        torch.add(v[..., 0], v[..., 1], alpha=16, out=out[r:r + n])
    return out


def _w4(lead, rows, cols, group, zeros, g):
    n = lead * rows
    q = _codes(n, cols, g).view(*((lead, rows) if lead > 1 else (rows,)), cols // 2)
    shape = (*q.shape[:-1], cols // group)
    s = torch.rand(shape, generator=g, device="cuda").add_(0.5).mul_(1.0 / (2.6 * math.sqrt(cols))).to(torch.bfloat16)
    z = torch.randint(6, 11, shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q, s, z


def _routes(c, g):
    T, E, K = c["T"], c["E"], c["K"]
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-6)
    keys = -torch.log(-torch.log(u))
    if c["routing"] == "zipf":
        keys = keys - 1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    idx = keys.topk(K, dim=1).indices
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), dim=1)
    off = torch.rand((T, K), generator=g, device="cuda") < c["unrouted"]
    return idx.masked_fill(off, -1), w.masked_fill(off, 0.0)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "moe":
        El, H, I = c["El"], c["H"], c["I"]
        s["x"] = _randn((c["T"], H), g)
        s["idx"], s["w"] = _routes(c, g)
        if c["fmt"] == "bf16":
            s["w13"] = torch.empty((El, 2 * I, H), dtype=torch.bfloat16, device="cuda")
            s["w2"] = torch.empty((El, H, I), dtype=torch.bfloat16, device="cuda")
            for e in range(El):
                s["w13"][e] = _randn((2 * I, H), g, 1.0 / math.sqrt(H))
                s["w2"][e] = _randn((H, I), g, 1.0 / math.sqrt(I))
        else:
            s["w13"], s["s13"], s["z13"] = (t if t is None else t.view(El, 2 * I, -1)
                                            for t in _w4(El, 2 * I, H, c["group"], c["zeros"], g))
            s["w2"], s["s2"], s["z2"] = (t if t is None else t.view(El, H, -1)
                                         for t in _w4(El, H, I, c["group"], c["zeros"], g))
    elif c["op"] == "matvec":
        s["x"] = _randn((c["M"], c["K"]), g)
        s["q"], s["s"], s["z"] = _w4(1, c["N"], c["K"], c["group"], c["zeros"], g)
    elif c["op"] == "router":
        s["x"] = _randn((c["T"], c["H"]), g)
        s["wr"] = _randn((c["E"], c["H"]), g, 1.0 / math.sqrt(c["H"]))
        s["bias"] = torch.randn((c["E"],), generator=g, device="cuda").mul_(0.05) if c["bias"] else None
    else:
        s["wt"] = _randn((c["N"], c["K"]), g, 1.0 / math.sqrt(c["K"]))
    return s


# ------------------------------------------------------------- plain forms --
def _out(v, name):
    return v if name == "fp32" else v.to(torch.bfloat16)


def _plain_weights(q, scale, zero, group):
    """fp32 weights of 4-bit codes: [..., K/2] uint8 -> [..., K]."""
    if scale is None:
        return q.float()
    v = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float()
    z = 8.0 if zero is None else zero.float().repeat_interleave(group, dim=-1)
    return (v - z) * scale.float().repeat_interleave(group, dim=-1)


def _plain_moe(s):
    c = s["case"]
    local = s["idx"] - c["rank"] * c["El"]
    here = (local >= 0) & (local < c["El"]) & (s["idx"] >= 0)
    act = local[here].unique()
    pick = lambda name: None if s.get(name) is None else s[name][act]  # noqa: E731
    w13 = _plain_weights(pick("w13"), pick("s13"), pick("z13"), c["group"])
    gu = torch.matmul(s["x"].float(), w13.transpose(1, 2))               # [A, T, 2I]
    del w13
    gate, up = gu[..., :c["I"]], gu[..., c["I"]:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    w2 = _plain_weights(pick("w2"), pick("s2"), pick("z2"), c["group"])
    y = torch.matmul(h, w2.transpose(1, 2))                              # [A, T, H]
    hit = (local[:, :, None] == act) & here[:, :, None]                  # [T, K, A]
    coef = (s["w"][:, :, None] * hit).sum(1)                             # [T, A]
    return _out((coef.t()[:, :, None] * y).sum(0), c["out"])


def _plain_matvec(s):
    c = s["case"]
    w = _plain_weights(s["q"], s["s"], s["z"], c["group"])
    return _out(torch.matmul(s["x"].float(), w.t()), c["out"])


def _plain_router(s):
    c = s["case"]
    l = torch.matmul(s["x"].float(), s["wr"].float().t())
    if c["scoring"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = l if s["bias"] is None else p + s["bias"]
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    w = p.gather(1, idx)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(idx=idx, w=w)


def _plain_quantize(s):
    c = s["case"]
    v = s["wt"].float().view(c["N"], -1, c["group"])
    if c["zeros"]:
        lo, hi = v.amin(-1).clamp(max=0.0), v.amax(-1).clamp(min=0.0)
        scale = (hi / 15.0 - lo / 15.0).to(torch.bfloat16)
        d = scale.float()
        zero = torch.round(-lo / d).clamp(0, 15)
        q = (torch.round(v / d[..., None]) + zero[..., None]).clamp(0, 15)
    else:
        scale = (v.abs().amax(-1) / 7.0).to(torch.bfloat16)
        d, zero = scale.float(), torch.full_like(scale, 8.0).float()
        q = torch.round(v / d[..., None]).clamp(-8, 7) + 8.0
    back = ((q - zero[..., None]) * d[..., None]).view(c["N"], c["K"]).to(torch.bfloat16)
    return dict(values=back, scale=scale, zero=zero.to(torch.uint8) if c["zeros"] else None)


# --------------------------------------------------------------------- run --
def run(state):
    s, c = state, state["case"]
    if not own:
        return dict(moe=_plain_moe, matvec=_plain_matvec, router=_plain_router, quantize=_plain_quantize)[c["op"]](s)
    import combine_send_counts_gb300 as ep
    dt = torch.float32 if c.get("out") == "fp32" else torch.bfloat16
    if c["op"] == "moe":
        if "plan" not in s:  # a program keeps the layer: its weights, workspace and error word
            if c["fmt"] == "bf16":
                w13, w2 = s["w13"], s["w2"]
            else:
                w13 = ep.W4(s["w13"], s["s13"], s["z13"], c["group"])
                w2 = ep.W4(s["w2"], s["s2"], s["z2"], c["group"])
            s["plan"] = ep.MoeDecode(w13, w2, rank=c["rank"], num_experts=c["E"], topk=c["K"], max_tokens=c["T"],
                                     out_dtype=dt)
        return s["plan"](s["x"], s["idx"], s["w"])
    if c["op"] == "matvec":
        if "plan" not in s:
            s["plan"] = ep.W4(s["q"], s["s"], s["z"], c["group"])
        return ep.w4_matvec(s["x"], s["plan"], out_dtype=dt)
    if c["op"] == "router":
        if "plan" not in s:
            s["plan"] = ep.RouterTopk(s["wr"], c["K"], scoring=c["scoring"], bias=s["bias"], renormalize=c["norm"],
                                      max_tokens=c["T"])
        idx, w = s["plan"](s["x"])
        return dict(idx=idx, w=w)
    w4 = ep.w4_quantize(s["wt"], c["group"], zeros=c["zeros"])
    return dict(values=ep.w4_dequantize(w4), scale=w4.scale, zero=w4.zero)


# -------------------------------------------------------------------- work --
def _w4_bytes(n, k, group, zeros):
    return n * k // 2 + n * (k // group) * (3 if zeros else 2)


def work(case):
    c = case
    if c["op"] == "moe":
        T, H, I, K = c["T"], c["H"], c["I"], c["K"]
        # expected distinct local experts under the case's routing
        p = [1.0 / (e + 1) ** 1.2 if c["routing"] == "zipf" else 1.0 for e in range(c["E"])]
        tot = sum(p)
        # inclusion of an expert in one token's K draws: exact for uniform, a bound-respecting
        # approximation for zipf (the Poisson form with the rate that gives K in all)
        if c["routing"] == "zipf":
            lo, hi = 0.0, 1e6
            for _ in range(100):
                mid = (lo + hi) / 2
                lo, hi = (mid, hi) if sum(1 - math.exp(-mid * v / tot) for v in p) < K * (1 - 1e-9) else (lo, mid)
            inc = [1 - math.exp(-lo * v / tot) for v in p]
        else:
            inc = [K / c["E"]] * c["E"]
        keep = 1.0 - c["unrouted"]
        first = c["rank"] * c["El"]
        mine = [v * keep for v in inc[first:first + c["El"]]]
        slots = T * sum(mine)
        act = sum(1 - (1 - min(v, 1.0)) ** T for v in mine)
        one = 3 * H * I * 2 if c["fmt"] == "bf16" else (_w4_bytes(2 * I, H, c["group"], c["zeros"])
                                                       + _w4_bytes(H, I, c["group"], c["zeros"]))
        return dict(bytes=act * one + T * H * 2 + T * K * 12 + T * H * (4 if c["out"] == "fp32" else 2),
                    flops=6.0 * H * I * slots)
    if c["op"] == "matvec":
        return dict(bytes=_w4_bytes(c["N"], c["K"], c["group"], c["zeros"]) + c["M"] * c["K"] * 2
                    + c["M"] * c["N"] * (4 if c["out"] == "fp32" else 2), flops=2.0 * c["M"] * c["N"] * c["K"])
    if c["op"] == "router":
        return dict(bytes=c["E"] * c["H"] * 2 + c["T"] * c["H"] * 2 + c["T"] * c["K"] * 12 + (4 * c["E"] if c["bias"] else 0),
                    flops=2.0 * c["T"] * c["H"] * c["E"])
    n = c["N"] * c["K"]  # bf16 in, codes and scales out, and the values they stand for
    return dict(bytes=2 * n + 2 * _w4_bytes(c["N"], c["K"], c["group"], c["zeros"]) + 2 * n, flops=4.0 * n)


# ------------------------------------------------------------------- exact --
def _weights64(q, scale, zero, group):
    if scale is None:
        return q.to(torch.float64)
    rows, half = q.shape
    w = torch.empty((rows, 2 * half), dtype=torch.float64, device=q.device)
    w[:, 0::2] = torch.remainder(q, 16).to(torch.float64)
    w[:, 1::2] = torch.div(q, 16, rounding_mode="floor").to(torch.float64)
    w = w.view(rows, -1, group)
    w -= 8.0 if zero is None else zero.to(torch.float64)[:, :, None]
    w *= scale.to(torch.float64)[:, :, None]
    return w.view(rows, 2 * half)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "moe":
        x = s["x"].to(torch.float64)
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        at = lambda name, e: None if s.get(name) is None else s[name][e]  # noqa: E731
        for e in range(c["El"]):
            toks, ks = torch.nonzero(s["idx"] == e + c["rank"] * c["El"], as_tuple=True)
            if toks.numel() == 0:
                continue
            w13 = _weights64(s["w13"][e], at("s13", e), at("z13", e), c["group"])
            a = x[toks] @ w13[:c["I"]].t()
            b = x[toks] @ w13[c["I"]:].t()
            y = (a * torch.sigmoid(a) * b) @ _weights64(s["w2"][e], at("s2", e), at("z2", e), c["group"]).t()
            out.index_add_(0, toks, y * s["w"][toks, ks].to(torch.float64)[:, None])
        return out
    if c["op"] == "matvec":
        x = s["x"].to(torch.float64)
        parts = []
        for r in range(0, c["N"], 8192):
            z = None if s["z"] is None else s["z"][r:r + 8192]
            parts.append(x @ _weights64(s["q"][r:r + 8192], s["s"][r:r + 8192], z, c["group"]).t())
        return torch.cat(parts, 1)
    if c["op"] == "router":
        logits = s["x"].to(torch.float64) @ s["wr"].to(torch.float64).t()
        score = torch.softmax(logits, 1) if c["scoring"] == "softmax" else torch.sigmoid(logits)
        key = logits if s["bias"] is None else score + s["bias"].to(torch.float64)
        idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["K"]]
        w = torch.take_along_dim(score, idx, 1)
        return dict(idx=idx, w=w / w.sum(1, keepdim=True) if c["norm"] else w)
    vals, scales, zs = [], [], []
    for r in range(0, c["N"], 8192):
        v = s["wt"][r:r + 8192].to(torch.float64)
        v = v.view(v.shape[0], -1, c["group"])
        if c["zeros"]:
            lo, hi = torch.clamp(v.min(2).values, max=0), torch.clamp(v.max(2).values, min=0)
            d = ((hi - lo) / 15).to(torch.bfloat16).to(torch.float64)
            z = torch.clamp(torch.round(-lo / d), 0, 15)
            q = torch.clamp(torch.round(v / d[:, :, None]) + z[:, :, None], 0, 15) - z[:, :, None]
            zs.append(z.to(torch.uint8))
        else:
            d = (v.abs().max(2).values / 7).to(torch.bfloat16).to(torch.float64)
            q = torch.clamp(torch.round(v / d[:, :, None]), -8, 7)
        vals.append((q * d[:, :, None]).view(v.shape[0], -1))
        scales.append(d)
    return dict(values=torch.cat(vals), scale=torch.cat(scales), zero=torch.cat(zs) if zs else None)
