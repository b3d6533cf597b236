"""Cases of the operators around the routing: the norm in front of a layer with
the residual's addition and 8-bit rows, its backward pass, the choice of experts
from logits with groups, its backward pass, and low-rank adapters of many
requests beside a shared projection.

8-bit rows are e4m3 codes with one fp32 scale for each 128 columns: with a =
max(max|v|, 1e-4) of a group, scale = a / 448 and code = e4m3(v * (448 / a)).
"""
import math

import torch

own = False  # False: plain torch forms; True: the package's operators


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # a decode step of one request: the sum, the normed row for the router and its 8-bit form for the experts
        dict(name="norm T1 7168 fp8", op="norm", T=1, H=7168, residual="bf16", w="bf16", y=True, fp8="row"),
        # a ragged batch of odd width whose residual stream is kept in 32 bits, 32-bit weights
        dict(name="norm T333 4168 fp32 residual", op="norm", T=333, H=4168, residual="fp32", w="fp32", y=True, fp8=""),
        # a prefill: everything that the layer behind it reads
        dict(name="norm T16384 7168 fp8", op="norm", T=16384, H=7168, residual="bf16", w="bf16", y=True, fp8="col"),
        # fine-tuning on a short sequence
        dict(name="norm backward T257 2048", op="norm_backward", T=257, H=2048, residual="bf16", w="bf16", dres=True),
        # a training step of a large layer
        dict(name="norm backward T16384 7168", op="norm_backward", T=16384, H=7168, residual="bf16", w="bf16",
             dres=True),
        # one token's experts: sigmoid scores, a bias for balance, the best four of eight groups
        dict(name="select T1 E256 groups", op="select", T=1, E=256, K=8, dtype="fp32", scoring="sigmoid", bias=True,
             groups=8, kept=4, group_score="top2", norm=True),
        # an odd number of tokens, logits as a bf16 product leaves them, no groups
        dict(name="select T4097 E60 softmax", op="select", T=4097, E=60, K=6, dtype="bf16", scoring="softmax",
             bias=False, groups=1, kept=1, group_score="max", norm=False),
        # a prefill's tokens
        dict(name="select T16384 E256 groups", op="select", T=16384, E=256, K=8, dtype="fp32", scoring="sigmoid",
             bias=True, groups=8, kept=4, group_score="top2", norm=True),
        # fine-tuning on a short sequence
        dict(name="select backward T200 E64", op="select_backward", T=200, E=64, K=6, dtype="fp32", scoring="sigmoid",
             norm=True, empty=0.1),
        # a training step
        dict(name="select backward T16384 E256", op="select_backward", T=16384, E=256, K=8, dtype="fp32",
             scoring="softmax", norm=False, empty=0.0),
        # a decode batch in which almost every request has an adapter of its own, some none, beside a 4-bit projection
        dict(name="lora M24 L32 r16 4096x4096", op="lora", M=24, L=32, R=16, K=4096, N=4096, runs=1, none=0.1,
             base="fp32", out="bf16"),
        # a prefill of a few long requests, added to what the projection left
        dict(name="lora M8192 L8 r64 7168x4096", op="lora", M=8192, L=8, R=64, K=7168, N=4096, runs=700, none=0.1,
             base="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "select", "select", "select_backward", "lora", "lora"])
    if op == "norm":
        fp8 = rng.choice(["", "row", "row", "col"])
        return dict(op=op, T=_log_int(rng, 1, 16384), H=_step(_log_int(rng, 256, 7168), 128 if fp8 else 8),
                    residual=rng.choice(["", "bf16", "bf16"] if fp8 else ["", "bf16", "fp32"]),
                    w=rng.choice(["bf16", "fp32"]), y=not fp8 or rng.random() < 0.7, fp8=fp8)
    if op == "norm_backward":
        residual = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, T=_log_int(rng, 1, 16384 if residual == "bf16" else 8192), H=_step(_log_int(rng, 256, 7168), 8),
                    residual=residual, w=rng.choice(["bf16", "fp32"]), dres=rng.random() < 0.7)
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * max(1, _log_int(rng, 8, 512) // groups)
        kept = rng.randint(1, groups)
        most = 16384 * 256 // max(E, 256)
        return dict(op=op, T=_log_int(rng, 1, most), E=E, K=rng.randint(1, min(8, E // groups * kept)),
                    dtype=rng.choice(["bf16", "fp32"]), scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.6, groups=groups, kept=kept,
                    group_score=rng.choice(["max", "top2"]), norm=rng.random() < 0.5)
    if op == "select_backward":
        E = _log_int(rng, 8, 512)
        return dict(op=op, T=_log_int(rng, 1, 16384 * 256 // max(E, 256)), E=E, K=rng.randint(1, min(8, E)),
                    dtype=rng.choice(["bf16", "fp32"]), scoring=rng.choice(["softmax", "sigmoid"]),
                    norm=rng.random() < 0.5, empty=rng.choice([0.0, 0.1]))
    while True:
        M = _log_int(rng, 1, 8192)
        c = dict(op=op, M=M, L=_log_int(rng, 1, 64), R=rng.choice([8, 16, 16, 32, 64, 128]),
                 K=_step(_log_int(rng, 256, 7168), 8), N=_step(_log_int(rng, 256, 7168), 8),
                 runs=1 if M <= 128 else _log_int(rng, 64, M), none=rng.choice([0.0, 0.1]),
                 base=rng.choice(["", "bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]))
        w = work(c)
        if w["flops"] <= 1.2e10 and w["bytes"] <= 2.5e8 and c["M"] * c["L"] * c["R"] <= 8192 * 8 * 64:
            return c


# ------------------------------------------------------------------ inputs --
def _randn(shape, g, std=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] in ("norm", "norm_backward"):
        T, H = c["T"], c["H"]
        s["w"] = (1.0 + 0.2 * torch.randn((H,), generator=g, device="cuda")).to(_TYPES[c["w"]])
        if c["op"] == "norm":
            s["x"] = _randn((T, H), g)
            s["res"] = _randn((T, H), g, 2.0, _TYPES[c["residual"]]) if c["residual"] else None
        else:
            s["h"] = _randn((T, H), g, 2.0, _TYPES[c["residual"]])
            s["dy"] = _randn((T, H), g, 0.01)
            s["dres"] = _randn((T, H), g, 0.01, _TYPES[c["residual"]]) if c["dres"] else None
    elif c["op"] in ("select", "select_backward"):
        T, E, K = c["T"], c["E"], c["K"]
        s["logits"] = _randn((T, E), g, 1.5, _TYPES[c["dtype"]])
        if c["op"] == "select":
            s["bias"] = torch.randn((E,), generator=g, device="cuda").mul_(0.05) if c["bias"] else None
        else:
            idx = s["logits"].float().topk(K, dim=1).indices
            off = torch.rand((T, K), generator=g, device="cuda") < c["empty"]
            s["idx"] = idx.masked_fill(off, -1)
            s["dw"] = torch.randn((T, K), generator=g, device="cuda").mul_(0.1)
    else:
        M, L, R, K, N = c["M"], c["L"], c["R"], c["K"], c["N"]
        s["x"] = _randn((M, K), g)
        s["a"] = _randn((L, R, K), g, 1.0 / math.sqrt(K))
        s["b"] = _randn((L, N, R), g, 0.5 / math.sqrt(R))
        s["scaling"] = torch.rand((L,), generator=g, device="cuda").add_(0.5)
        s["base"] = _randn((M, N), g, 1.0, _TYPES[c["base"]]) if c["base"] else None
        pieces = -(-M // c["runs"])   # requests of runs rows each, one adapter or none for each
        ids = torch.randint(0, L, (pieces,), generator=g, device="cuda")
        ids = ids.masked_fill(torch.rand((pieces,), generator=g, device="cuda") < c["none"], -1)
        s["ids"] = ids.repeat_interleave(c["runs"])[:M].contiguous()
    return s


# ------------------------------------------------------------- plain forms --
_EPS, _SCALE = 1e-6, 2.5


def _plain_norm(s):
    c = s["case"]
    out = {}
    h = s["x"].float()
    if s["res"] is not None:
        out["residual"] = (h + s["res"].float()).to(s["res"].dtype)
        h = out["residual"].float()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + _EPS) * s["w"].float()
    if c["y"]:
        out["y"] = y.to(torch.bfloat16)
    if c["fp8"]:
        v = y.view(c["T"], -1, 128)
        a = v.abs().amax(2).clamp(min=1e-4)
        out["q"] = (v * (448.0 / a)[:, :, None]).clamp(-448.0, 448.0).view(c["T"], c["H"]).to(torch.float8_e4m3fn)
        scale = a / 448.0
        out["scale"] = scale if c["fp8"] == "row" else scale.t().contiguous()
    return out


def _plain_norm_backward(s):
    h, w, g = s["h"].float(), s["w"].float(), s["dy"].float()
    r = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + _EPS)
    n = h * r
    gw = g * w
    d = r * (gw - n * (gw * n).mean(1, keepdim=True))
    if s["dres"] is not None:
        d = d + s["dres"].float()
    return dict(dresidual=d.to(s["h"].dtype), dx=d.to(torch.bfloat16), dweight=(g * n).sum(0))


def _plain_scores(l, c):
    if c["scoring"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        return p / p.sum(1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-l))


def _plain_select(s):
    # in 64 bits: keys of two experts may be nearer than 32 bits tell
    c = s["case"]
    l = s["logits"].double()
    p = _plain_scores(l, c)
    key = l if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        by = (key if c["group_score"] == "max" or s["bias"] is not None else p).view(c["T"], c["groups"], -1)
        if c["group_score"] == "max":
            mark = by.amax(2)
        else:
            mark = torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(mark, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(mark).scatter_(1, best, 1.0) > 0
        keep = keep[:, :, None].expand(c["T"], c["groups"], c["E"] // c["groups"]).reshape(c["T"], c["E"])
        key = key.masked_fill(~keep, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    w = p.gather(1, idx)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(idx=idx, w=(w * _SCALE).float())


def _plain_select_backward(s):
    c = s["case"]
    p = _plain_scores(s["logits"].float(), c)
    there = (s["idx"] >= 0).float()
    at = s["idx"].clamp(min=0)
    pk = p.gather(1, at) * there
    d = s["dw"] * _SCALE * there
    if c["norm"]:
        total = pk.sum(1, keepdim=True)
        d = (d - (d * pk).sum(1, keepdim=True) / total) / total * there
        d = torch.where(total > 0, d, torch.zeros_like(d))
    dp = torch.zeros_like(p).scatter_add_(1, at, d)
    if c["scoring"] == "softmax":
        out = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        out = dp * p * (1.0 - p)
    return out.to(s["logits"].dtype)


def _plain_lora(s):
    c = s["case"]
    L, R = c["L"], c["R"]
    v = s["x"].float() @ s["a"].view(L * R, -1).float().t()
    hit = (s["ids"][:, None] == torch.arange(L, device="cuda")).float() * s["scaling"]
    v = (v.view(-1, L, R) * hit[:, :, None]).view(-1, L * R)
    y = v @ s["b"].permute(0, 2, 1).reshape(L * R, -1).float()
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(_TYPES[c["out"]])


# --------------------------------------------------------------------- run --
_PLAIN = dict(norm=_plain_norm, norm_backward=_plain_norm_backward, select=_plain_select,
              select_backward=_plain_select_backward, lora=_plain_lora)


def run(state):
    s, c = state, state["case"]
    if not own:
        return _PLAIN[c["op"]](s)
    import combine_send_counts_gb300 as ep
    if c["op"] == "norm":
        r = ep.add_rms_norm(s["x"], s["w"], s["res"], eps=_EPS, y=c["y"], fp8=c["fp8"] != "",
                            scale_fmt=ep.EP_SCALE_COL_F32 if c["fp8"] == "col" else ep.EP_SCALE_ROW_F32)
        out = {}
        if s["res"] is not None:
            out["residual"] = r["residual"]
        if c["y"]:
            out["y"] = r["y"]
        if c["fp8"]:
            out["q"], out["scale"] = r["q"].view(torch.float8_e4m3fn), r["scale"]
        return out
    if c["op"] == "norm_backward":
        r = ep.add_rms_norm_backward(s["dy"], s["h"], s["w"], s["dres"], eps=_EPS)
        return dict(dresidual=r["dresidual"], dx=r["dx"], dweight=r["dweight"])
    if c["op"] == "select":
        idx, w = ep.router_select(s["logits"], c["K"], scoring=c["scoring"], bias=s["bias"], num_groups=c["groups"],
                                  topk_groups=c["kept"], group_score=c["group_score"], renormalize=c["norm"],
                                  scale=_SCALE)
        return dict(idx=idx, w=w)
    if c["op"] == "select_backward":
        return ep.router_select_backward(s["logits"], s["idx"], s["dw"], scoring=c["scoring"], renormalize=c["norm"],
                                         scale=_SCALE)
    if "plan" not in s:  # a program keeps the adapters: their weights, workspace and error word
        s["plan"] = ep.LoraAdapters(s["a"], s["b"], s["scaling"], max_tokens=c["M"], out_dtype=_TYPES[c["out"]])
    return s["plan"](s["x"], s["ids"], s["base"])


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    size = {"": 0, "bf16": 2, "fp32": 4}
    if c["op"] == "norm":
        n, r = c["T"] * c["H"], size[c["residual"]]
        one = 2 + 2 * r + (2 if c["y"] else 0) + (1 + 4 / 128 if c["fp8"] else 0)
        return dict(bytes=n * one + c["H"] * size[c["w"]], flops=4.0 * n)
    if c["op"] == "norm_backward":
        n, r = c["T"] * c["H"], size[c["residual"]]
        # a bf16 residual's gradient is x's too
        one = 2 + r + (r if c["dres"] else 0) + r + (2 if r == 4 else 0)
        return dict(bytes=n * one + c["H"] * (size[c["w"]] + 4), flops=8.0 * n)
    if c["op"] == "select":
        T, E, K = c["T"], c["E"], c["K"]
        return dict(bytes=T * E * size[c["dtype"]] + T * K * 12 + (4 * E if c["bias"] else 0), flops=6.0 * T * E)
    if c["op"] == "select_backward":
        T, E, K = c["T"], c["E"], c["K"]
        # sigmoid scores, and softmax scores divided by their sum, need the chosen logits alone
        read = T * E if c["scoring"] == "softmax" and not c["norm"] else T * K
        return dict(bytes=(read + T * E) * size[c["dtype"]] + T * K * 12, flops=6.0 * T * E)
    M, L, R, K, N = c["M"], c["L"], c["R"], c["K"], c["N"]
    pieces = -(-M // c["runs"])
    share = 1.0 - c["none"]
    used = L * (1.0 - (1.0 - share / L) ** pieces)   # expected adapters that some row names
    rows = M * share
    return dict(bytes=rows * K * 2 + used * R * (K + N) * 2 + M * N * (size[c["base"]] + size[c["out"]]) + 8 * M,
                flops=2.0 * rows * R * (K + N))


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "norm":
        out = {k: [] for k in (["residual"] if c["residual"] else []) + (["y"] if c["y"] else [])
               + (["q", "scale"] if c["fp8"] else [])}
        w = s["w"].to(torch.float64)
        for t in range(0, c["T"], 2048):
            h = s["x"][t:t + 2048].to(torch.float64)
            if c["residual"]:
                h = (h + s["res"][t:t + 2048].to(torch.float64)).to(s["res"].dtype).to(torch.float64)
                out["residual"].append(h.to(s["res"].dtype))
            y = h * torch.rsqrt(torch.sum(h * h, 1) / c["H"] + _EPS)[:, None] * w
            if c["y"]:
                out["y"].append(y)
            if c["fp8"]:
                top = torch.clamp(torch.max(torch.abs(y.view(-1, c["H"] // 128, 128)), 2).values, min=1e-4)
                q = y / torch.repeat_interleave(top, 128, 1) * 448.0
                out["q"].append(q.to(torch.float8_e4m3fn).to(torch.float32))
                out["scale"].append(top / 448.0)
        out = {k: torch.cat(v) for k, v in out.items()}
        if c["fp8"] == "col":
            out["scale"] = out["scale"].t()
        return out
    if c["op"] == "norm_backward":
        # of f(h) = sum of dy * y: by the product rule, term by term
        ds, dw = [], torch.zeros((c["H"],), dtype=torch.float64, device="cuda")
        w = s["w"].to(torch.float64)
        for t in range(0, c["T"], 2048):
            h, g = s["h"][t:t + 2048].to(torch.float64), s["dy"][t:t + 2048].to(torch.float64)
            m = torch.sum(h * h, 1, keepdim=True) / c["H"] + _EPS
            dm = torch.sum(g * w * h, 1, keepdim=True) * (-0.5) * m ** -1.5      # through the mean square
            d = g * w * m ** -0.5 + dm * 2.0 * h / c["H"]
            dw += torch.sum(g * h * m ** -0.5, 0)
            if s["dres"] is not None:
                d += s["dres"][t:t + 2048].to(torch.float64)
            ds.append(d)
        d = torch.cat(ds)
        return dict(dresidual=d, dx=d, dweight=dw)
    if c["op"] == "select":
        l = s["logits"].to(torch.float64)
        score = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
        key = l if s["bias"] is None else score + s["bias"].to(torch.float64)
        if c["groups"] > 1:
            marks = []
            for part in torch.chunk(key if s["bias"] is not None or c["group_score"] == "max" else score, c["groups"], 1):
                marks.append(part.topk(min(2, part.shape[1]) if c["group_score"] == "top2" else 1, dim=1).values.sum(1))
            order = torch.argsort(torch.stack(marks, 1), dim=1, descending=True, stable=True)
            place = torch.argsort(order, dim=1)      # of each group
            key = torch.where(torch.repeat_interleave(place, c["E"] // c["groups"], 1) < c["kept"], key,
                              torch.full_like(key, -math.inf))
        idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["K"]]
        w = torch.take_along_dim(score, idx, 1)
        return dict(idx=idx, w=_SCALE * (w / w.sum(1, keepdim=True) if c["norm"] else w))
    if c["op"] == "select_backward":
        # the matrix of derivatives of the chosen scores by the logits, times dw
        l = s["logits"].to(torch.float64).requires_grad_(True)
        score = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
        chosen = torch.take_along_dim(score, s["idx"].clamp(min=0), 1)
        chosen = torch.where(s["idx"] >= 0, chosen, torch.zeros_like(chosen))
        if c["norm"]:
            total = chosen.sum(1, keepdim=True)
            chosen = chosen / torch.where(total > 0, total, torch.ones_like(total))
        return torch.autograd.grad((chosen * _SCALE * s["dw"].to(torch.float64)).sum(), l)[0]
    out = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    if s["base"] is not None:
        out += s["base"].to(torch.float64)
    for i in range(c["L"]):
        rows = torch.nonzero(s["ids"] == i)[:, 0]
        if rows.numel():
            v = s["x"][rows].to(torch.float64) @ s["a"][i].to(torch.float64).t()
            out[rows] += s["scaling"][i].to(torch.float64) * (v @ s["b"][i].to(torch.float64).t())
    return out
