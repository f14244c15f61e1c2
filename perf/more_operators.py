"""The operators of a mixture-of-experts block around the expert products: sizes, inputs, plain forms and 64-bit references.

Four operators, each in its directions:

  route     forward: scores s = softmax or sigmoid of the router's logits, c = s + bias decides: the best groups of experts
            (by their two largest c), in them the k largest c, ties to the lowest index; weights s, renormalised over the
            k and scaled; and the experts' row counts, the row of every (token, choice) in expert order, and its inverse.
            grad: the logits' gradient from the weights'
  rows      dispatch: out[rows[t, j]] = X[t];  combine: Y[t] = sum_j weights[t, j] O[rows[t, j]]
  gate      forward: h = silu(g) u of rows [g | u], and the rows saved in 8 bits (E4M3, a power of two per 32).
            grad: from the saved rows and dh, weighted per row by its router weight w: d[g | u], w h and dw
            save: BF16 rows to 8 bits
  wgrad     dB_g (+)= alpha dD_g^T A_g, A's rows saved in 8 bits once per token and found through the routing

Where `own` is true, run() makes the library's calls; where it is false, elementary torch operations in 32 bits (what
decides between experts in 64).
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one next token: latency
        {"name": "route 1 token", "op": "route", "tokens": 1, "experts": 128, "topk": 8, "scores": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "renormalise": True, "scale": 1.0, "f32": False, "padded": 0.0},
        # a training micro-batch with a bias for balance and a limit to four of eight groups of experts
        {"name": "route groups", "op": "route", "tokens": 4096, "experts": 256, "topk": 8, "scores": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "renormalise": True, "scale": 2.5, "f32": True, "padded": 0.0},
        # a padded batch, an odd number of experts, weights that are not renormalised
        {"name": "route grad ragged", "op": "route grad", "tokens": 10007, "experts": 60, "topk": 4, "scores": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "renormalise": False, "scale": 1.0, "f32": False, "padded": 0.3},
        # a training micro-batch into expert order
        {"name": "dispatch large", "op": "dispatch", "tokens": 8192, "experts": 64, "topk": 8, "hidden": 4096,
         "padded": 0.0},
        # the way back of a few decoded tokens
        {"name": "combine 4 tokens", "op": "combine", "tokens": 4, "experts": 128, "topk": 8, "hidden": 4096,
         "weighted": True, "padded": 0.0},
        # a padded batch, rows whose length is an odd multiple of 16 bytes
        {"name": "combine ragged", "op": "combine", "tokens": 5003, "experts": 60, "topk": 6, "hidden": 2056,
         "weighted": True, "padded": 0.3},
        # the activation of a training micro-batch, its inputs saved for the backward pass
        {"name": "gate large", "op": "gate", "rows": 65536, "inner": 2048, "save": True},
        # its backward pass on a ragged batch
        {"name": "gate grad ragged", "op": "gate grad", "tokens": 4001, "experts": 60, "topk": 4, "inner": 1408,
         "weighted": True, "padded": 0.3},
        # a block's input saved for the backward pass
        {"name": "save rows", "op": "save", "rows": 8192, "inner": 4096},
        # 8 experts with a few rows each (the repository's grouped decode workload): the gradient written bounds the time
        {"name": "wgrad few rows", "op": "wgrad", "tokens": 64, "topk": 2, "experts": 8, "empty": 1, "spare": 0, "n": 4096,
         "k": 7168, "skew": 0.7, "add": False},
        # a training batch routed unevenly over 64 small experts, one of several micro-batches accumulated in FP32
        {"name": "wgrad ragged", "op": "wgrad", "tokens": 2000, "topk": 8, "experts": 64, "empty": 4, "spare": 384,
         "n": 2048, "k": 2048, "skew": 0.7, "add": True},
        # a large training batch on 8 wide experts
        {"name": "wgrad large", "op": "wgrad", "tokens": 8192, "topk": 2, "experts": 8, "empty": 0, "spare": 0, "n": 4096,
         "k": 7168, "skew": 0.4, "add": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route grad", "dispatch", "combine", "gate", "gate grad", "save", "wgrad"])
    padded = rng.choice([0.0, 0.0, 0.1, 0.4])
    if op in ("route", "route grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        per = max(_log(rng, 8, 256) // groups, 4)
        scores = rng.choice(["softmax", "sigmoid"])
        topk_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(8, topk_groups * per))
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": groups * per, "topk": topk, "scores": scores,
                "bias": rng.random() < 0.5, "groups": groups, "topk_groups": topk_groups,
                "renormalise": topk > 1 and rng.random() < 0.6,   # (of one choice: a constant, its gradient 0)
                "scale": rng.choice([1.0, 2.5]), "f32": rng.random() < 0.5,
                "padded": padded}
    experts = _log(rng, 8, 128)
    topk = rng.randint(1, 8)
    if op in ("dispatch", "combine"):
        case = {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts, "topk": topk, "hidden": 8 * _log(rng, 64, 512),
                "padded": padded}
        if op == "combine":
            case["weighted"] = rng.random() < 0.7
        return case
    if op in ("gate", "save"):
        case = {"op": op, "rows": _log(rng, 1, 65536), "inner": 32 * rng.randint(8, 64)}
        if op == "gate":
            case["save"] = rng.random() < 0.7
        return case
    if op == "gate grad":
        return {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts, "topk": topk, "inner": 32 * rng.randint(8, 64),
                "weighted": rng.random() < 0.7, "padded": padded}
    experts = _log(rng, 2, 64)
    empty = rng.randint(0, experts // 4)
    topk = rng.randint(1, min(8, experts - empty))
    return {"op": op, "tokens": _log(rng, 16, 16384 // topk), "topk": topk, "experts": experts, "empty": empty,
            "spare": rng.choice([0, 0, 1, 130]), "n": 8 * _log(rng, 32, 512), "k": 32 * _log(rng, 8, 128),
            "skew": rng.choice([0.0, 0.4, 0.8]), "add": rng.choice([False, False, True])}


# ---------------------------------------------------------------- inputs

def _places(ids, experts):
    """Rows in expert order of the choices `ids` (tokens x topk; -1: none): sizes, rows, slots."""
    flat = ids.reshape(-1).long()
    kept = flat >= 0
    order = torch.sort(torch.where(kept, flat, experts), stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    count = kept.sum()
    slots = torch.where(torch.arange(flat.numel(), device=flat.device) < count, order, -1)
    sizes = (flat[:, None] == torch.arange(experts, device=flat.device)).sum(dim=0)
    return (sizes.to(torch.int32), torch.where(kept, rows, -1).reshape(ids.shape).to(torch.int32), slots.to(torch.int32))


def _some_choices(gen, case, bias=None):
    """Distinct experts per token, -1 for the padded tokens."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    u = torch.rand(t, e, generator=gen, device="cuda")
    if bias is not None:
        u = u.log().neg().log().neg() + bias   # uneven: the k largest of logits with that noise
    ids = u.topk(k, dim=1).indices.to(torch.int32)
    if case.get("padded"):
        ids[torch.rand(t, generator=gen, device="cuda") < case["padded"]] = -1
    return ids


def _to8(x):
    """E4M3 values and the exponent bytes (2^(byte - 127) per 32) of BF16 rows: the least power of two with which the
    largest of the 32 is at most 448."""
    b = x.float().reshape(x.shape[0], -1, 32)
    mantissa, exponent = torch.frexp(b.abs().amax(dim=2))     # amax = mantissa 2^exponent, mantissa in [0.5, 1)
    e = torch.where(mantissa > 0, exponent - 9 + (mantissa > 0.875).int(), -127).clamp(-127, 127)
    q = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn)
    return q.reshape(x.shape), (e + 127).to(torch.uint8)


def _from8(q, e, dtype=F32):
    two = torch.ldexp(torch.ones_like(e, dtype=dtype), e.int() - 127)
    return (q.to(dtype).reshape(*e.shape, 32) * two[..., None]).reshape(q.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=F32) * scale).to(dtype)

    def empty(*shape, dtype):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s, op = dict(case), case["op"]
    if op in ("route", "route grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        z = normal(t, e, dtype=F32) * 1.5 + normal(e, dtype=F32) * 0.5
        s["logits"] = z if case["f32"] else z.to(BF16)
        s["bias_values"] = normal(e, scale=0.05, dtype=F32) if case["bias"] else None
        s["keep"] = torch.rand(t, generator=gen, device="cuda") >= case["padded"] if case["padded"] else None
        if op == "route":
            s["out"] = [empty(t, k, dtype=torch.int32), empty(t, k, dtype=F32), empty(e, dtype=torch.int32),
                        empty(t, k, dtype=torch.int32), empty(t * k, dtype=torch.int32)]
        else:
            s["ids"] = _choose(s)[0].to(torch.int32)
            s["dweights"] = normal(t, k, dtype=F32)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    if op in ("dispatch", "combine", "gate grad"):
        s["sizes"], s["rows"], s["slots"] = _places(_some_choices(gen, case), case["experts"])
        t, k = case["tokens"], case["topk"]
        if case.get("weighted"):
            w = torch.rand(t, k, generator=gen, device="cuda") + 0.05
            s["weights"] = w / w.sum(dim=1, keepdim=True)
    if op == "dispatch":
        s["X"] = normal(t, case["hidden"])
        s["out"] = torch.zeros(t * k, case["hidden"], device="cuda", dtype=BF16)
    elif op == "combine":
        s["O"] = normal(t * k, case["hidden"])
        s["Y"] = empty(t, case["hidden"], dtype=BF16)
    elif op in ("gate", "save"):
        r, i = case["rows"], case["inner"]
        width = 2 * i if op == "gate" else i
        s["X"] = normal(r, width)
        s["Q"] = empty(r, width, dtype=torch.uint8)
        s["sf"] = empty(r, width // 32, dtype=torch.uint8)
        s["H"] = empty(r, i, dtype=BF16)
    elif op == "gate grad":
        r, i = t * k, case["inner"]
        q, s["sf"] = _to8(normal(r, 2 * i))
        s["Q"] = q.view(torch.uint8)
        s["dH"] = normal(r, i)
        s["dX"], s["H"] = torch.zeros(r, 2 * i, device="cuda", dtype=BF16), torch.zeros(r, i, device="cuda", dtype=BF16)
        s["dweights"] = torch.zeros(t, k, device="cuda") if case["weighted"] else None
    elif op == "wgrad":
        e, n, k = case["experts"], case["n"], case["k"]
        skew = normal(e, scale=case["skew"], dtype=F32)
        skew[torch.randperm(e, generator=gen, device="cuda")[:case["empty"]]] = -torch.inf
        s["sizes_dev"], _, s["slots"] = _places(_some_choices(gen, case, skew), e)
        s["sizes"] = s["sizes_dev"].tolist()
        rows = case["tokens"] * case["topk"]
        s["dD"] = normal(rows + case["spare"], n)
        s["slots"] = torch.nn.functional.pad(s["slots"], (0, case["spare"]), value=-1)
        q, s["sf"] = _to8(normal(case["tokens"], k))
        s["Q"] = q.view(torch.uint8)
        if case["add"]:   # what earlier micro-batches left
            s["dB"] = torch.randn(e, n, k, generator=gen, device="cuda") * math.sqrt(rows / e)
        else:
            s["dB"] = empty(e, n, k, dtype=BF16)
    return s


# ---------------------------------------------------------------- one pass

def _choose(s):
    """Choices (tokens x topk, -1 for padded tokens) and all scores, in 64 bits."""
    z = s["logits"].to(F64)
    if s["scores"] == "softmax":
        score = (z - z.amax(dim=1, keepdim=True)).exp()
        score = score / score.sum(dim=1, keepdim=True)
    else:
        score = 1 / (1 + (-z).exp())
    c = score if s["bias_values"] is None else score + s["bias_values"].to(F64)
    if s["groups"] > 1:
        by = c.reshape(c.shape[0], s["groups"], -1)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(dim=2)
        stay = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        out = torch.ones_like(best, dtype=torch.bool).scatter_(1, stay, False)
        c = by.masked_fill(out[:, :, None], -torch.inf).reshape(c.shape)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    return ids if s["keep"] is None else torch.where(s["keep"][:, None], ids, -1), score


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "route":
        ids, score = _choose(s)
        w = score.gather(1, ids.clamp(min=0)).float()
        if s["renormalise"]:
            w = w / w.sum(dim=1, keepdim=True)
        w = torch.where(ids >= 0, w * s["scale"], 0.0)
        sizes, rows, slots = _places(ids, s["experts"])
        return {"ids": ids.to(torch.int32), "weights": w, "sizes": sizes, "rows": rows, "slots": slots}
    if op == "route grad":
        z, ids, dw = s["logits"].float(), s["ids"].clamp(min=0).long(), s["dweights"]
        if s["scores"] == "softmax":
            score = (z - z.amax(dim=1, keepdim=True)).exp()
            score = score / score.sum(dim=1, keepdim=True)
        else:
            score = 1 / (1 + (-z).exp())
        a = score.gather(1, ids)
        if s["renormalise"]:
            total = a.sum(dim=1, keepdim=True)
            da = (dw - (dw * a).sum(dim=1, keepdim=True) / total) / total
        else:
            da = dw
        da = torch.where(s["ids"] >= 0, da * s["scale"], 0.0)
        ds = torch.zeros_like(score).scatter_(1, ids, da)
        if s["scores"] == "softmax":
            dz = score * (ds - (da * a).sum(dim=1, keepdim=True))
        else:
            dz = ds * score * (1 - score)
        return {"dlogits": dz.to(s["logits"].dtype)}
    if op == "dispatch":
        token = s["slots"].clamp(min=0).long() // s["topk"]
        return {"out": torch.where((s["slots"] >= 0)[:, None], s["X"][token], s["out"])}
    if op == "combine":
        there = (s["rows"] >= 0)[:, :, None]
        o = torch.where(there, s["O"][s["rows"].clamp(min=0).long()].float(), 0.0)
        if s["weighted"]:
            o = o * s["weights"][:, :, None]
        return {"Y": o.sum(dim=1).to(BF16)}
    if op in ("gate", "save"):
        got = {}
        if op == "save" or s["save"]:
            got["saved"], got["exponents"] = _to8(s["X"])
        if op == "gate":
            g, u = s["X"].float().chunk(2, dim=1)
            got["H"] = (g / (1 + (-g).exp()) * u).to(BF16)
        return got
    if op == "gate grad":
        g, u = _from8(s["Q"].view(torch.float8_e4m3fn), s["sf"]).chunk(2, dim=1)
        dh = s["dH"].float()
        sg = 1 / (1 + (-g).exp())
        h = g * sg * u
        there = (s["slots"] >= 0)[:, None]
        dg, du = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
        dw = None
        if s["weighted"]:
            at = s["slots"].clamp(min=0).long()
            w = s["weights"].reshape(-1)[at][:, None]
            each = (dh * h).sum(dim=1)
            h, dg, du = h * w, dg * w, du * w
            dw = torch.zeros_like(s["weights"]).reshape(-1).index_add_(0, at, torch.where(there[:, 0], each, 0.0))
            dw = dw.reshape(s["weights"].shape)
        dx = torch.where(there, torch.cat([dg, du], dim=1), 0.0).to(BF16)
        return {"dX": dx, "H": torch.where(there, h, 0.0).to(BF16), "dweights": dw}
    a = _from8(s["Q"].view(torch.float8_e4m3fn), s["sf"])
    rows = s["tokens"] * s["topk"]
    a = a[s["slots"][:rows].long() // s["topk"]].split(s["sizes"])
    d = s["dD"][:rows].float().split(s["sizes"])
    if s["add"]:
        return {"dB": s["dB"].add_(torch.stack([x.T @ y for x, y in zip(d, a)]))}
    return {"dB": torch.stack([(x.T @ y).to(BF16) for x, y in zip(d, a)])}


def _run_own(s):
    from dense_block_scaled_gb300 import tkg
    op = s["op"]
    if op == "route":
        tkg.moe_route(s["logits"], *s["out"], bias=s["bias_values"], keep=s["keep"], scores=s["scores"], groups=s["groups"],
                      topk_groups=s["topk_groups"], renormalise=s["renormalise"], scale=s["scale"])
        return dict(zip(("ids", "weights", "sizes", "rows", "slots"), s["out"]))
    if op == "route grad":
        tkg.moe_route_grad(s["logits"], s["ids"], s["dweights"], s["dlogits"], scores=s["scores"],
                           renormalise=s["renormalise"], scale=s["scale"])
        return {"dlogits": s["dlogits"]}
    if op == "dispatch":
        tkg.moe_dispatch(s["X"], s["rows"], s["out"])
        return {"out": s["out"]}
    if op == "combine":
        tkg.moe_combine(s["O"], s["rows"], s["Y"], weights=s.get("weights"))
        return {"Y": s["Y"]}
    if op == "save":
        tkg.checkpoint_mxfp8(s["X"], s["Q"], s["sf"])
        return {"saved": s["Q"].view(torch.float8_e4m3fn), "exponents": s["sf"]}
    if op == "gate":
        if not s["save"]:
            tkg.swiglu(s["X"], s["H"])
            return {"H": s["H"]}
        tkg.swiglu(s["X"], s["H"], s["Q"], s["sf"])
        return {"saved": s["Q"].view(torch.float8_e4m3fn), "exponents": s["sf"], "H": s["H"]}
    if op == "gate grad":
        tkg.swiglu_grad(s["Q"], s["sf"], s["dH"], s["dX"], s["H"], slots=s["slots"], weights=s.get("weights"),
                        dweights=s["dweights"])
        return {"dX": s["dX"], "H": s["H"], "dweights": s["dweights"]}
    tkg.gemm_grouped_dev_mxfp8_wgrad(s["sizes_dev"], s["dD"], s["Q"], s["sf"], s["dB"], slots=s["slots"], topk=s["topk"],
                                     accumulate=s["add"])
    return {"dB": s["dB"]}


def work(case):
    op = case["op"]
    if op in ("route", "route grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        size = 4 if case["f32"] else 2
        if op == "route":
            return {"bytes": t * e * size + 16 * t * k + 4 * e * (1 + case["bias"]), "flops": 4 * t * e}
        read = t * e if case["scores"] == "softmax" and not case["renormalise"] else t * k
        return {"bytes": (read + t * e) * size + 8 * t * k, "flops": 6 * t * e}
    if op in ("dispatch", "combine"):
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        tokens = t * (1 - case["padded"])
        whole = t if op == "combine" else tokens     # a padded token's Y is written, its X not read
        return {"bytes": 2 * h * (whole + tokens * k) + 4 * t * k * (2 if case.get("weighted") else 1),
                "flops": 2 * tokens * k * h if op == "combine" else 0}
    if op in ("gate", "save"):
        r, i = case["rows"], case["inner"]
        if op == "save":
            return {"bytes": r * i * (2 + 33 / 32), "flops": 2 * r * i}
        return {"bytes": r * i * (6 + (2 * 33 / 32 if case["save"] else 0)), "flops": 10 * r * i}
    if op == "gate grad":
        r = case["tokens"] * case["topk"]
        there = r * (1 - case["padded"])
        return {"bytes": there * case["inner"] * (2 * 33 / 32 + 2 + 6) + 4 * r + (8 * there if case["weighted"] else 0),
                "flops": 20 * there * case["inner"]}
    t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
    r = t * case["topk"]
    # read and written back in FP32 where there are rows, or written for every expert
    matrices = 8 * (e - case["empty"]) if case["add"] else 2 * e
    return {"bytes": 2 * r * n + t * k * 33 / 32 + 4 * r + matrices * n * k, "flops": 2 * r * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("route", "route grad"):
        z = s["logits"].to(F64)
        p = torch.softmax(z, dim=1) if case["scores"] == "softmax" else torch.sigmoid(z)
        if op == "route":
            value = p if s["bias_values"] is None else p + s["bias_values"].to(F64)
            if case["groups"] > 1:
                grouped = value.unflatten(1, (case["groups"], -1))
                score = grouped.topk(2, dim=2).values.sum(dim=2)
                least = score.topk(case["topk_groups"], dim=1).values[:, -1:]
                value = torch.where((score >= least)[:, :, None], grouped, torch.full_like(grouped, -9.0)).flatten(1)
            w = p.gather(1, value.topk(case["topk"], dim=1).indices)
            w = case["scale"] * (w / w.sum(dim=1, keepdim=True) if case["renormalise"] else w)
            if s["keep"] is not None:
                w = w * s["keep"][:, None]
            return {"ids": None, "weights": w, "sizes": None, "rows": None, "slots": None}
        kept = s["ids"] >= 0
        at = s["ids"].long().clamp(min=0)
        z.requires_grad_(True)
        p = torch.softmax(z, dim=1) if case["scores"] == "softmax" else torch.sigmoid(z)
        w = p.gather(1, at)
        w = case["scale"] * (w / w.sum(dim=1, keepdim=True) if case["renormalise"] else w)
        (torch.where(kept, w, torch.zeros_like(w)) * s["dweights"].to(F64)).sum().backward()
        return {"dlogits": z.grad}
    if op == "dispatch":
        out = torch.zeros(s["out"].shape, dtype=F64, device="cuda")
        for j in range(case["topk"]):
            r = s["rows"][:, j].long()
            out[r[r >= 0]] = s["X"][r >= 0].to(F64)
        return {"out": out}
    if op == "combine":
        Y = torch.zeros(s["Y"].shape, dtype=F64, device="cuda")
        for j in range(case["topk"]):
            r = s["rows"][:, j].long()
            o = s["O"][r[r >= 0]].to(F64)
            Y[r >= 0] += o * s["weights"][r >= 0, j:j + 1].to(F64) if case["weighted"] else o
        return {"Y": Y}
    if op in ("gate", "save"):
        got = {}
        if op == "save" or case["save"]:
            b = s["X"].to(F64).unflatten(1, (-1, 32))
            e = torch.full(b.shape[:2], -127, dtype=torch.int64, device="cuda")
            for i in range(-40, 41):   # the least exponent with which the largest is at most 448 (inputs are near 1)
                e = torch.where((b.abs().amax(dim=2) > 448 * 2.0 ** (i - 1)), i, e)
            got["saved"], got["exponents"] = torch.ldexp(b, -e[..., None]).flatten(1), None
        if op == "gate":
            x, i = s["X"].to(F64), case["inner"]
            got["H"] = torch.nn.functional.silu(x[:, :i]) * x[:, i:]
        return got
    if op == "gate grad":
        x = _from8(s["Q"].view(torch.float8_e4m3fn), s["sf"], F64).requires_grad_(True)
        i, kept = case["inner"], s["slots"] >= 0
        w = torch.ones(x.shape[0], dtype=F64, device="cuda")
        if case["weighted"]:
            w = s["weights"].reshape(-1).to(F64)[s["slots"].long().clamp(min=0)]
        w = torch.where(kept, w, torch.zeros_like(w)).requires_grad_(True)
        h = w[:, None] * torch.nn.functional.silu(x[:, :i]) * x[:, i:]
        (h * s["dH"].to(F64))[kept].sum().backward()
        dw = None
        if case["weighted"]:
            dw = torch.zeros(s["weights"].numel(), dtype=F64, device="cuda")
            dw[s["slots"][kept].long()] = w.grad[kept]
            dw = dw.reshape(s["weights"].shape)
        return {"dX": x.grad, "H": h.detach(), "dweights": dw}
    rows = case["tokens"] * case["topk"]
    A = _from8(s["Q"].view(torch.float8_e4m3fn), s["sf"], F64)
    token = s["slots"][:rows].long() // case["topk"]
    dB, o = torch.zeros(s["dB"].shape, dtype=F64, device="cuda"), 0
    for g, m in enumerate(s["sizes"]):
        dB[g] = torch.einsum("in,ik->nk", s["dD"][o:o + m].to(F64), A[token[o:o + m]])
        o += m
    return {"dB": dB + s["dB"].to(F64) if case["add"] else dB}
