"""The training-side operators as a user calls them: sizes, inputs, plain forms and 64-bit references.

Four operators, all on BF16 operands:

  loss    softmax cross entropy of a linear head over a large vocabulary: z = alpha X W^T (tokens x vocab, never kept),
          lse_t = log sum_v exp z_tv, loss_t = lse_t - z_t,label(t); a label outside [0, vocab) ignores its row (loss 0)
  grad    its gradient: g_tv = alpha dloss_t (exp(z_tv - lse_t) - [v = label(t)]), dX = g W, dW = g^T X
  dgrad   expert products D = A B_g^T with row counts in device memory: gradient to the rows, dA = alpha dD B_g
  wgrad   the same products: gradient to the experts' matrices, dB_g = alpha dD_g^T A_g (dense training: one group),
          written in BF16 or added to FP32 values (accumulation over micro-batches)

Where `own` is true, run() makes the library's calls; where it is false, elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one next token scored against a mid-size vocabulary: W is read once, latency and bandwidth count
        {"name": "loss 1 token", "op": "loss", "tokens": 1, "vocab": 32768, "hidden": 2048, "ignored": 0.0, "alpha": 1.0},
        # a few answer tokens of a small model: all operands fit in L2, launches count
        {"name": "loss small", "op": "loss", "tokens": 16, "vocab": 4000, "hidden": 512, "ignored": 0.0, "alpha": 1.0},
        # evaluation of a ragged batch with padding, an odd vocabulary and a logit scale
        {"name": "loss ragged", "op": "loss", "tokens": 777, "vocab": 50001, "hidden": 2048, "ignored": 0.3, "alpha": 0.5},
        # a training micro-batch of a large-vocabulary model
        {"name": "loss large", "op": "loss", "tokens": 8192, "vocab": 131072, "hidden": 4096, "ignored": 0.0, "alpha": 1.0},
        # fine-tuning on a short sequence: the head's matrix and its gradient bound the time
        {"name": "grad short", "op": "grad", "tokens": 128, "vocab": 32768, "hidden": 2048, "ignored": 0.0, "alpha": 1.0},
        # a ragged batch with half of its tokens masked (prompts), odd sizes
        {"name": "grad ragged", "op": "grad", "tokens": 1333, "vocab": 50001, "hidden": 2048, "ignored": 0.5, "alpha": 0.5},
        # the training micro-batch above
        {"name": "grad large", "op": "grad", "tokens": 8192, "vocab": 131072, "hidden": 4096, "ignored": 0.0, "alpha": 1.0},
        # 8 experts with a few rows each (the repository's grouped decode workload): the experts' matrices bound the time
        {"name": "dgrad few rows", "op": "dgrad", "groups": 8, "empty": 0, "rows": 128, "spare": 0, "n": 4096, "k": 7168,
         "skew": 0.0},
        # a training batch routed unevenly over 64 small experts, four of them without rows, rows to spare in the buffers
        {"name": "dgrad ragged", "op": "dgrad", "groups": 64, "empty": 4, "rows": 16000, "spare": 384, "n": 2048,
         "k": 2048, "skew": 0.7},
        # the same few rows: the gradient written for every expert bounds the time
        {"name": "wgrad few rows", "op": "wgrad", "groups": 8, "empty": 1, "rows": 128, "spare": 0, "n": 4096, "k": 7168,
         "skew": 0.7, "add": False},
        # the uneven training batch above, one of several micro-batches accumulated in FP32
        {"name": "wgrad ragged", "op": "wgrad", "groups": 64, "empty": 4, "rows": 16000, "spare": 384, "n": 2048,
         "k": 2048, "skew": 0.7, "add": True},
        # a large training batch on 8 wide experts
        {"name": "wgrad large", "op": "wgrad", "groups": 8, "empty": 0, "rows": 16384, "spare": 0, "n": 4096, "k": 7168,
         "skew": 0.4, "add": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "grad", "dgrad", "wgrad"])
    if op in ("loss", "grad"):
        return {"op": op, "tokens": _log(rng, 1 if op == "loss" else 16, 8192), "vocab": _log(rng, 1000, 131072),
                "hidden": 8 * _log(rng, 32, 512), "ignored": rng.choice([0.0, 0.0, 0.2, 0.6]),
                "alpha": rng.choice([1.0, 1.0, 0.5])}
    groups = _log(rng, 1, 64)
    empty = rng.randint(0, groups // 4)
    case = {"op": op, "groups": groups, "empty": empty, "rows": _log(rng, max(16, groups), 16384),
            "spare": rng.choice([0, 0, 1, 130]), "n": 8 * _log(rng, 32, 512), "k": 8 * _log(rng, 32, 512),
            "skew": rng.choice([0.0, 0.4, 0.8])}
    if op == "wgrad":
        case["add"] = rng.choice([False, False, True])
    return case


def _sizes(case, seed):
    """Row counts per expert: `empty` of them zero, the others uneven by `skew`, summing to `rows`."""
    rng = random.Random(seed)
    groups, rows = case["groups"], case["rows"]
    idle = set(rng.sample(range(groups), case["empty"]))
    busy = [g for g in range(groups) if g not in idle]
    w = [math.exp(case["skew"] * rng.gauss(0.0, 1.0)) for _ in busy]
    total = sum(w)
    spread = rows - len(busy)   # every busy expert has a row
    take = [1 + int(spread * x / total) for x in w]
    for i in range(rows - sum(take)):
        take[i % len(take)] += 1
    sizes = [0] * groups
    for g, t in zip(busy, take):
        sizes[g] = t
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(BF16)

    s = dict(case)
    if case["op"] in ("loss", "grad"):
        t, v, h = case["tokens"], case["vocab"], case["hidden"]
        s["X"] = normal(t, h)
        s["W"] = normal(v, h, scale=2.0 / (math.sqrt(h) * case["alpha"]))   # logits of spread 2
        labels = torch.randint(0, v, (t,), generator=gen, device="cuda")
        if case["ignored"]:
            labels[torch.rand(t, generator=gen, device="cuda") < case["ignored"]] = -100
        s["labels"] = labels
        if case["op"] == "loss":
            s["loss"] = torch.empty(t, device="cuda")
            s["lse"] = torch.empty(t, device="cuda")
        else:
            # what the forward pass left, and the gradient of the mean over the kept rows
            s["lse"] = torch.logsumexp(case["alpha"] * (s["X"].float() @ s["W"].float().T), dim=1)
            kept = labels >= 0
            s["dloss"] = kept.float() / kept.sum().clamp(min=1)
            s["dX"] = torch.empty(t, h, device="cuda", dtype=BF16)
            s["dW"] = torch.empty(v, h, device="cuda", dtype=BF16)
        return s
    sizes = _sizes(case, seed)
    rows, cap, n, k = case["rows"], case["rows"] + case["spare"], case["n"], case["k"]
    s["sizes"] = sizes
    s["sizes_dev"] = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    s["dD"] = normal(cap, n)
    if case["op"] == "dgrad":
        s["B"] = normal(case["groups"], n, k, scale=1.0 / math.sqrt(n))
        s["dA"] = torch.empty(cap, k, device="cuda", dtype=BF16)
    else:
        s["A"] = normal(cap, k)
        if case["add"]:   # what earlier micro-batches left
            s["dB"] = torch.randn(case["groups"], n, k, generator=gen, device="cuda") * math.sqrt(rows / case["groups"])
        else:
            s["dB"] = torch.empty(case["groups"], n, k, device="cuda", dtype=BF16)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op in ("loss", "grad"):
        X, W, labels = s["X"].float(), s["W"].float(), s["labels"]
        kept = (labels >= 0) & (labels < s["vocab"])
        at = labels.clamp(0, s["vocab"] - 1)[:, None]
        z = (X @ W.T).mul_(s["alpha"])
        if op == "loss":
            top = z.max(dim=1).values
            lse = (z - top[:, None]).exp_().sum(dim=1).log() + top
            loss = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
            return {"loss": loss, "lse": lse}
        g = z.sub_(s["lse"][:, None]).exp_()
        g.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        g.mul_(torch.where(kept, s["dloss"] * s["alpha"], 0.0)[:, None])
        return {"dX": (g @ W).to(BF16), "dW": (g.T @ X).to(BF16)}
    dDs = s["dD"][:s["rows"]].split(s["sizes"])
    if op == "dgrad":
        return {"dA": torch.cat([d.float() @ b.float() for d, b in zip(dDs, s["B"])]).to(BF16)}
    As = s["A"][:s["rows"]].split(s["sizes"])
    if s["add"]:
        return {"dB": s["dB"].add_(torch.stack([d.float().T @ a.float() for d, a in zip(dDs, As)]))}
    return {"dB": torch.stack([(d.float().T @ a.float()).to(BF16) for d, a in zip(dDs, As)])}


def _run_own(s):
    from dense_block_scaled_gb300 import tkg
    op = s["op"]
    if op == "loss":
        tkg.linear_ce_loss(s["X"], s["W"], s["labels"], s["loss"], s["lse"], alpha=s["alpha"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "grad":
        tkg.linear_ce_grad(s["X"], s["W"], s["labels"], s["lse"], s["dloss"], s["dX"], s["dW"], alpha=s["alpha"])
        return {"dX": s["dX"], "dW": s["dW"]}
    if op == "dgrad":
        tkg.gemm_grouped_dev_bf16_dgrad(s["sizes_dev"], s["dD"], s["B"], s["dA"])
        return {"dA": s["dA"][:s["rows"]]}
    tkg.gemm_grouped_dev_bf16_wgrad(s["sizes_dev"], s["dD"], s["A"], s["dB"], accumulate=s["add"])
    return {"dB": s["dB"]}


def work(case):
    if case["op"] in ("loss", "grad"):
        t, v, h = case["tokens"], case["vocab"], case["hidden"]
        if case["op"] == "loss":
            return {"bytes": 2 * (t + v) * h + 16 * t, "flops": 2 * t * v * h}
        return {"bytes": 4 * (t + v) * h + 16 * t, "flops": 6 * t * v * h}
    g, r, n, k = case["groups"], case["rows"], case["n"], case["k"]
    if case["op"] == "dgrad":
        matrices = 2 * (g - case["empty"])          # read for the experts that have rows
    elif case["add"]:
        matrices = 8 * (g - case["empty"])          # read and written back in FP32 where there are rows
    else:
        matrices = 2 * g                            # written for every expert
    return {"bytes": 2 * r * (n + k) + matrices * n * k + 4 * g, "flops": 2 * r * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 1.2e13:   # over about 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("loss", "grad"):
        X, labels, alpha, v = s["X"].to(f64), s["labels"], case["alpha"], case["vocab"]
        kept = (labels >= 0) & (labels < v)
        blocks = [(v0, s["W"][v0:v0 + 8192]) for v0 in range(0, v, 8192)]   # vocabulary entries at a time
        if case["op"] == "loss":
            parts, hit = [], torch.zeros(case["tokens"], dtype=f64, device="cuda")
            for v0, Wp in blocks:
                z = alpha * torch.einsum("th,vh->tv", X, Wp.to(f64))
                parts.append(torch.logsumexp(z, dim=1))
                at = ((labels >= v0) & (labels < v0 + Wp.shape[0])).nonzero()[:, 0]
                hit[at] = z[at, labels[at] - v0]
            lse = torch.logsumexp(torch.stack(parts), dim=0)
            return {"loss": torch.where(kept, lse - hit, torch.zeros_like(lse)), "lse": lse}
        scale = torch.where(kept, s["dloss"].to(f64) * alpha, torch.zeros_like(X[:, 0]))[:, None]
        dX, dW, lse = torch.zeros_like(X), [], s["lse"].to(f64)[:, None]
        for v0, Wp in blocks:
            p = torch.exp(alpha * torch.einsum("th,vh->tv", X, Wp.to(f64)) - lse)
            onehot = labels[:, None] == torch.arange(v0, v0 + Wp.shape[0], device="cuda")[None, :]
            g = scale * (p - onehot.to(f64))
            dX += torch.einsum("tv,vh->th", g, Wp.to(f64))
            dW.append(torch.einsum("tv,th->vh", g, X))
        return {"dX": dX, "dW": torch.cat(dW)}
    off = [0]
    for m in s["sizes"]:
        off.append(off[-1] + m)
    if case["op"] == "dgrad":
        out = torch.zeros(case["rows"], case["k"], dtype=f64, device="cuda")
        for g, B in enumerate(s["B"]):
            out[off[g]:off[g + 1]] = torch.einsum("in,nk->ik", s["dD"][off[g]:off[g + 1]].to(f64), B.to(f64))
        return {"dA": out}
    dB = torch.stack([torch.einsum("in,ik->nk", s["dD"][off[g]:off[g + 1]].to(f64),
                                   s["A"][off[g]:off[g + 1]].to(f64)) for g in range(case["groups"])])
    return {"dB": dB + s["dB"].to(f64) if case["add"] else dB}
