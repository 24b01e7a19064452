"""Cases of the head's loss and of the expert router, for timing and comparison.

Two operators, each with its gradient:

- the head's loss: the softmax cross entropy of bf16(hidden) @ bf16(weight).T
  against a target column per row, over a large vocabulary, without storing the
  logits; its gradient for the hidden states and for the weight;
- expert routing: softmax or sigmoid scores of a token's expert logits, a
  balance bias that only moves the choice, groups of experts, the best k
  (ties to the lower expert), renormalised weights; the experts' load; the
  gradient of the weights for the logits.

``run`` computes them from elementary torch operations, or, with ``own`` set,
through ``wide_bf16_row_gb300.topk``.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

IGNORE = -100  # the target of a row that takes no part in the loss
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LARGEST_TRAIN = (4096, 2048, 98592)
LARGEST_ROUTE = (65536, 256)


def listed():
    return [
        # one draft's log-probability over a small vocabulary: latency
        {"name": "score 1x2048x4096", "op": "score", "rows": 1, "dim": 2048, "vocab": 4096, "ignored": 0.0},
        # the draft window scored against the draft head
        {"name": "score 15x2048x98592", "op": "score", "rows": 15, "dim": 2048, "vocab": 98592, "ignored": 0.0},
        # a prompt's loss under the full vocabulary (evaluation)
        {"name": "score 1000x2048x248320", "op": "score", "rows": 1000, "dim": 2048, "vocab": 248320, "ignored": 0.2},
        # a drafter trained under a frozen head: only the hidden states' gradient
        {"name": "frozen 256x2048x248320", "op": "frozen", "rows": 256, "dim": 2048, "vocab": 248320, "ignored": 0.0},
        # a short padded batch, odd sizes, half of its rows ignored
        {"name": "train 333x1032x32771", "op": "train", "rows": 333, "dim": 1032, "vocab": 32771, "ignored": 0.5},
        # a training step of the draft head
        {"name": "train 4096x2048x98592", "op": "train", "rows": 4096, "dim": 2048, "vocab": 98592, "ignored": 0.1},
        # one decoded token: latency
        {"name": "route 1x256 sigmoid", "op": "route", "tokens": 1, "experts": 256, "k": 8, "score": "sigmoid",
         "groups": 8, "kept": 4, "bias": True, "renorm": True, "type": "bf16", "masked": 0.0},
        # a prompt through a softmax router, renormalised over the chosen experts
        {"name": "route 8192x128 softmax", "op": "route", "tokens": 8192, "experts": 128, "k": 8, "score": "softmax",
         "groups": 1, "kept": 1, "bias": False, "renorm": True, "type": "bf16", "masked": 0.0},
        # a training step's routing: grouped sigmoid scores with a balance bias, forward, load and gradient
        {"name": "route step 65536x256", "op": "route step", "tokens": 65536, "experts": 256, "k": 8,
         "score": "sigmoid", "groups": 8, "kept": 4, "bias": True, "renorm": True, "type": "fp32", "masked": 0.02},
        # plain softmax weights (dense gradient), an odd count of experts, some of them masked
        {"name": "route step 20001x60", "op": "route step", "tokens": 20001, "experts": 60, "k": 4,
         "score": "softmax", "groups": 1, "kept": 1, "bias": False, "renorm": False, "type": "fp16", "masked": 0.1},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    if rng.random() < 0.55:
        op = rng.choice(("score", "frozen", "train"))
        dim, vocab = 8 * _log(rng, 16, 512), _log(rng, 1000, 248320)
        passes = {"score": 1, "frozen": 2, "train": 3}[op]
        n, d, v = LARGEST_TRAIN
        most = min(n, max(1, 3 * n * d * v // (passes * dim * vocab)))
        return {"op": op, "rows": _log(rng, 1, most), "dim": dim, "vocab": vocab,
                "ignored": rng.choice((0.0, 0.1, 0.5))}
    groups = rng.choice((1, 1, 2, 4, 8))
    experts = groups * max(2, _log(rng, 8, 256) // groups)
    kept = rng.randint(max(1, groups // 2), groups)
    k = rng.randint(1, min(8, kept * (experts // groups)))
    tokens = _log(rng, 1, LARGEST_ROUTE[0] * LARGEST_ROUTE[1] // max(experts, LARGEST_ROUTE[1]))
    return {"op": rng.choice(("route", "route step")), "tokens": tokens, "experts": experts, "k": k,
            "score": rng.choice(("softmax", "sigmoid")), "groups": groups, "kept": kept, "bias": rng.random() < 0.5,
            "renorm": rng.random() < 0.6, "type": rng.choice(("bf16", "fp16", "fp32")),
            "masked": rng.choice((0.0, 0.02, 0.2))}


def _is_head(case):
    return case["op"] in ("score", "frozen", "train")


def _scale(case):
    return 2.5 if case["renorm"] and case["score"] == "sigmoid" else 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    if _is_head(case):
        n, d, v = case["rows"], case["dim"], case["vocab"]
        weight = torch.empty((v, d), dtype=torch.bfloat16, device=dev)
        for at in range(0, v, 32768):
            stop = min(v, at + 32768)
            weight[at:stop] = normal(stop - at, d) * d ** -0.5
        target = torch.randint(0, v, (n,), generator=gen, device=dev)
        # hidden states that lean toward their targets, from not at all to quite surely
        lean = (math.log(v) + 2) * uniform(n, 1)
        hidden = (normal(n, d) + lean * weight[target].float()).to(torch.bfloat16)
        target = torch.where(uniform(n) < case["ignored"], IGNORE, target)
        # the gradient of the mean over the rows that count
        valid = (target != IGNORE).float()
        grad = valid / valid.sum().clamp(min=1)
        return {"case": case, "hidden": hidden, "weight": weight, "target": target, "grad": grad}

    t, e = case["tokens"], case["experts"]
    logits = 1.5 * normal(t, e) + 0.5 * normal(e)
    if case["masked"] > 0:  # experts out of reach for a token, and padded tokens that have none
        logits.masked_fill_(uniform(t, e) < case["masked"], -math.inf)
        logits.masked_fill_(uniform(t, 1) < 0.01, -math.inf)
    bias = 0.1 * normal(e) if case["bias"] else None
    return {"case": case, "logits": logits.to(TYPES[case["type"]]), "bias": bias, "grad": normal(t, case["k"])}


# ------------------------------------------------------------------ plain forms


def _plain_head(s):
    case, target = s["case"], s["target"]
    h, w = s["hidden"].float(), s["weight"].float()
    x = h @ w.t()
    valid = target != IGNORE
    column = target.clamp(min=0)[:, None]
    # over the target's logit, so that a loss near 0 keeps its digits: log(1 + sum over the others of exp(x - x_t))
    hit = x.gather(1, column)
    rest = x.scatter(1, column, -math.inf)
    top = rest.amax(1, keepdim=True)
    above = top - hit + (rest - top).exp_().sum(1, keepdim=True).log()
    loss = above.clamp(min=0) + (-above.abs()).exp().log1p()
    lse = hit + loss
    loss = torch.where(valid, loss[:, 0], 0.0)
    if case["op"] == "score":
        return {"loss": loss, "lse": torch.where(valid, lse[:, 0], 0.0)}
    p = (x - lse).exp()
    p.scatter_add_(1, column, -torch.ones_like(lse))
    p *= torch.where(valid, s["grad"], 0.0)[:, None]
    out = {"loss": loss, "d_hidden": (p @ w).to(torch.bfloat16)}
    if case["op"] == "train":
        out["d_weight"] = (p.t() @ h).to(torch.bfloat16)
    return out


def _plain_scores(x, valid, score):
    if score == "sigmoid":
        return torch.where(valid, 1 / (1 + (-x).exp()), 0.0)
    x = torch.where(valid, x, -math.inf)
    top = x.amax(1, keepdim=True)
    p = torch.where(valid, (x - top).exp(), 0.0)
    return p / p.sum(1, keepdim=True).clamp(min=torch.finfo(x.dtype).tiny)


def _plain_route(s):
    case = s["case"]
    x = s["logits"].float()
    t, e = x.shape
    valid = (x == x) & (x > -math.inf)
    # the choice in 64 bits: scores next to a border
    wide = _plain_scores(x.double(), valid, case["score"])
    biased = wide if s["bias"] is None else wide + s["bias"].double()
    choice = torch.where(valid, x.double() if s["bias"] is None else biased, -math.inf)
    if case["groups"] > 1:
        each = torch.where(valid, biased, -math.inf).view(t, case["groups"], -1)
        best = each.sort(-1, descending=True).values[..., :2]
        group = torch.where(best > -math.inf, best, 0.0).sum(-1)
        group = torch.where(best[..., 0] > -math.inf, group, -math.inf)
        order = group.sort(dim=-1, descending=True, stable=True).indices[:, : case["kept"]]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order, True)
        choice = torch.where(kept.repeat_interleave(e // case["groups"], 1), choice, -math.inf)
    value, idx = choice.sort(dim=-1, descending=True, stable=True)
    taken = value[:, : case["k"]] > -math.inf
    idx = torch.where(taken, idx[:, : case["k"]], -1)
    scores = _plain_scores(x, valid, case["score"])
    weight = torch.where(taken, scores.gather(1, idx.clamp(min=0)), 0.0)
    if case["renorm"]:
        weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-30)
    out = {"idx": idx.int(), "weight": weight * _scale(case)}
    if case["op"] == "route":
        return out
    load = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
    load.scatter_add_(0, torch.where(taken, idx, e).view(-1), torch.ones_like(idx, dtype=torch.int32).view(-1))
    out["load"] = load[:e]
    chosen = torch.where(taken, scores.gather(1, idx.clamp(min=0)), 0.0)
    g = torch.where(taken, s["grad"], 0.0) * _scale(case)
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-30)
        g = torch.where(taken, (g - (g * chosen).sum(1, keepdim=True) / total) / total, 0.0)
    dense = torch.zeros_like(scores).scatter_add_(1, idx.clamp(min=0), g)
    if case["score"] == "sigmoid":
        d = dense * scores / (1 + x.exp())
    else:
        d = scores * (dense - (dense * scores).sum(1, keepdim=True))
    out["d_logits"] = torch.where(valid, d, 0.0).to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------ the framework's calls


def _own_head(s):
    from wide_bf16_row_gb300 import topk

    op = s["case"]["op"]
    loss, lse = topk.head_loss_bf16(s["hidden"], s["weight"], s["target"], ignore_index=IGNORE)
    if op == "score":
        return {"loss": loss, "lse": lse}
    d_hidden, d_weight = topk.head_loss_grad_bf16(s["hidden"], s["weight"], s["target"], lse, s["grad"],
                                                  ignore_index=IGNORE, weight_grad=op == "train")
    out = {"loss": loss, "d_hidden": d_hidden}
    if op == "train":
        out["d_weight"] = d_weight
    return out


def _own_route(s):
    from wide_bf16_row_gb300 import topk

    case = s["case"]
    how = {"score": case["score"], "renormalize": case["renorm"], "scale": _scale(case)}
    step = case["op"] == "route step"
    load = torch.zeros(case["experts"], dtype=torch.int32, device="cuda") if step else None
    idx, weight = topk.route_experts(s["logits"], case["k"], bias=s["bias"], groups=case["groups"],
                                     groups_kept=case["kept"], load=load, **how)
    out = {"idx": idx, "weight": weight}
    if step:
        out["load"] = load
        out["d_logits"] = topk.route_experts_grad(s["logits"], idx, s["grad"], **how)
    return out


def run(state):
    if own:
        return _own_head(state) if _is_head(state["case"]) else _own_route(state)
    return _plain_head(state) if _is_head(state["case"]) else _plain_route(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if _is_head(case):
        n, d, v = case["rows"], case["dim"], case["vocab"]
        product = 2 * n * d * v
        read = 2 * n * d + 2 * v * d + 8 * n
        if case["op"] == "score":
            return {"bytes": read + 8 * n, "flops": product}
        read += 4 * n
        if case["op"] == "frozen":
            return {"bytes": read + 4 * n + 2 * n * d, "flops": 2 * product}
        return {"bytes": read + 4 * n + 2 * n * d + 2 * v * d, "flops": 3 * product}
    t, e, k = case["tokens"], case["experts"], case["k"]
    size = 4 if case["type"] == "fp32" else 2
    total = t * e * size + (4 * e if case["bias"] else 0) + 8 * t * k
    flops = 8 * t * e
    if case["op"] == "route step":
        total += 4 * e + 4 * t * k + t * e * size
        flops += 8 * t * e
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_head(case, s):
    n, v = case["rows"], case["vocab"]
    h, target = s["hidden"].double(), s["target"]
    step = max(1, min(v, (1 << 28) // max(n, case["dim"])))
    pieces = [(at, min(v, at + step)) for at in range(0, v, step)]
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
    hit = torch.zeros(n, dtype=torch.float64, device="cuda")
    rows = torch.arange(n, device="cuda")
    for lo, hi in pieces:
        x = torch.mm(h, s["weight"][lo:hi].double().t())
        lse = torch.logaddexp(lse, torch.logsumexp(x, 1))
        here = (target >= lo) & (target < hi)
        hit = torch.where(here, x[rows, torch.where(here, target - lo, 0)], hit)
    counts = target != IGNORE
    loss = torch.where(counts, lse - hit, 0.0)
    if case["op"] == "score":
        return {"loss": loss, "lse": torch.where(counts, lse, 0.0)}
    g = torch.where(counts, s["grad"].double(), 0.0)
    dh = torch.zeros_like(h)
    dw = torch.empty(s["weight"].shape, dtype=torch.float32, device="cuda") if case["op"] == "train" else None
    for lo, hi in pieces:
        w = s["weight"][lo:hi].double()
        q = torch.exp(torch.mm(h, w.t()) - lse[:, None]) * g[:, None]
        here = (target >= lo) & (target < hi)
        q[rows, torch.where(here, target - lo, 0)] -= torch.where(here, g, 0.0)
        dh += torch.mm(q, w)
        if dw is not None:
            dw[lo:hi] = torch.mm(q.t(), h)
    out = {"loss": loss, "d_hidden": dh}
    if dw is not None:
        out["d_weight"] = dw
    return out


def _exact_route(case, s):
    x = s["logits"].double().cpu().numpy()
    t, e = x.shape
    k, groups = case["k"], case["groups"]
    out_of_reach = np.isnan(x) | (x == -np.inf)
    safe = np.where(out_of_reach, 0.0, x)
    if case["score"] == "sigmoid":
        score = np.where(safe >= 0, 1 / (1 + np.exp(-np.abs(safe))), np.exp(-np.abs(safe)) / (1 + np.exp(-np.abs(safe))))
    else:
        top = np.where(out_of_reach, -np.inf, x).max(1, keepdims=True)
        score = np.exp(safe - np.where(np.isfinite(top), top, 0.0))
        score = np.where(out_of_reach, 0.0, score)
        score = score / np.maximum(score.sum(1, keepdims=True), 1e-300)
    score = np.where(out_of_reach, 0.0, score)
    lifted = score if s["bias"] is None else score + s["bias"].double().cpu().numpy()
    rank = np.where(out_of_reach, -np.inf, safe if s["bias"] is None else lifted)
    if groups > 1:
        each = np.sort(np.where(out_of_reach, -np.inf, lifted).reshape(t, groups, -1), axis=2)[:, :, ::-1][:, :, :2]
        total = np.where(np.isinf(each[:, :, 0]), -np.inf, np.where(np.isinf(each), 0.0, each).sum(2))
        place = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
        rank = np.where(np.repeat(place < case["kept"], e // groups, axis=1), rank, -np.inf)
    idx = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    taken = np.take_along_axis(rank, idx, 1) > -np.inf
    chosen = np.where(taken, np.take_along_axis(score, idx, 1), 0.0)
    total = np.maximum(chosen.sum(1, keepdims=True), 1e-300) if case["renorm"] else 1.0
    out = {"idx": np.where(taken, idx, -1), "weight": _scale(case) * chosen / total}
    if case["op"] == "route":
        return out
    out["load"] = np.bincount(idx[taken], minlength=e)
    g = np.where(taken, s["grad"].double().cpu().numpy(), 0.0) * _scale(case)
    if case["renorm"]:
        g = np.where(taken, (g - (g * chosen).sum(1, keepdims=True) / total) / total, 0.0)
    d = np.zeros((t, e))
    np.put_along_axis(d, np.where(taken, idx, 0), 0.0, 1)
    row = np.broadcast_to(np.arange(t)[:, None], idx.shape)
    d[row[taken], idx[taken]] = g[taken]
    if case["score"] == "sigmoid":
        d = d * score * (1 - score)
    else:
        d = score * (d - (d * score).sum(1, keepdims=True))
    out["d_logits"] = np.where(out_of_reach, 0.0, d)
    return out


def exact(case, seed):
    if _is_head(case):
        products = {"score": 1, "frozen": 3, "train": 4}[case["op"]]
        if products * 2 * case["rows"] * case["dim"] * case["vocab"] > 1.2e13:
            return None
        return _exact_head(case, prepare(case, seed))
    return _exact_route(case, prepare(case, seed))
