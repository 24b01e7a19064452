"""Cases of the operators around an expert layer and before sampling, for timing and comparison.

Four operators:

- tokens sorted by the experts that routing chose for them, and back: the
  order of the choices by expert (stable), the tokens' rows gathered in it,
  the experts' rows combined with the routing weights, and the gradients of both;
- rows in 8 bits: e4m3 values with a scale for each 128 of a row, gathered by
  expert in the same pass;
- the product of such rows with weights in 8 bits (a scale for each block of
  128 x 128), of one matrix or of the experts' matrices over their rows;
- logits made ready for sampling: repetition, presence and frequency
  penalties, biases and a grammar's mask.

``run`` computes them from elementary torch operations, or, with ``own`` set,
through ``wide_bf16_row_gb300.topk``.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128  # values that share a scale
LARGEST_ROWS = 16384 * 8 * 2048  # values of the sorted rows
LARGEST_PRODUCT = 16384 * 8 * 2048 * 1536  # multiplications
LARGEST_LOGITS = 256 * 248320


def listed():
    return [
        # one decoded token to its eight experts and back: latency
        {"name": "sort 1x2048 k8", "op": "sort", "tokens": 1, "dim": 2048, "experts": 256, "k": 8, "type": "bf16",
         "dropped": 0.0},
        # a prompt's tokens to the experts and back
        {"name": "sort 8192x2048 k8", "op": "sort", "tokens": 8192, "dim": 2048, "experts": 128, "k": 8,
         "type": "bf16", "dropped": 0.0},
        # an odd batch with padded tokens and dropped choices, forward and backward
        {"name": "sort step 5001x1001 k3", "op": "sort step", "tokens": 5001, "dim": 1001, "experts": 60, "k": 3,
         "type": "fp32", "dropped": 0.1},
        # a training step's tokens: forward and backward
        {"name": "sort step 16384x2048 k8", "op": "sort step", "tokens": 16384, "dim": 2048, "experts": 256, "k": 8,
         "type": "bf16", "dropped": 0.0},
        # one decoded token through its experts' first matrix: latency
        {"name": "experts 1x2048x1536 k8", "op": "experts", "tokens": 1, "dim": 2048, "out": 1536, "experts": 128,
         "k": 8, "type": "bf16", "dropped": 0.0},
        # a batch of decoding requests: every expert's weight is read for a few rows
        {"name": "experts 64x2048x1536 k8", "op": "experts", "tokens": 64, "dim": 2048, "out": 1536, "experts": 128,
         "k": 8, "type": "bf16", "dropped": 0.0},
        # a long prompt through the experts, some tokens padded
        {"name": "experts 16384x2048x1536 k8", "op": "experts", "tokens": 16384, "dim": 2048, "out": 1536,
         "experts": 128, "k": 8, "type": "bf16", "dropped": 0.02},
        # the draft window through the draft head in 8 bits
        {"name": "product 15x2048x98592", "op": "product", "tokens": 15, "dim": 2048, "out": 98592, "type": "bf16"},
        # a prompt through one matrix of odd sizes, sums kept in 32 bits
        {"name": "product 4001x1040x4099", "op": "product", "tokens": 4001, "dim": 1040, "out": 4099, "type": "fp32"},
        # one request's draft logits: latency
        {"name": "logits 1x98592", "op": "logits", "rows": 1, "cols": 98592, "type": "bf16", "history": 500,
         "biases": 4, "mask": False},
        # a batch under the full vocabulary, half of it under a grammar
        {"name": "logits 256x248320", "op": "logits", "rows": 256, "cols": 248320, "type": "bf16", "history": 4000,
         "biases": 16, "mask": True},
        # long conversations in 32 bits over an odd vocabulary
        {"name": "logits 33x32771", "op": "logits", "rows": 33, "cols": 32771, "type": "fp32", "history": 40000,
         "biases": 0, "mask": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(("sort", "sort step", "experts", "experts", "product", "logits"))
    dropped = rng.choice((0.0, 0.0, 0.02, 0.2))
    if op in ("sort", "sort step"):
        experts, dim = _log(rng, 4, 512), _log(rng, 64, 8192)
        k = rng.randint(1, min(8, experts))
        most = min(65536, LARGEST_ROWS // (dim * k))
        return {"op": op, "tokens": _log(rng, 1, most), "dim": dim, "experts": experts, "k": k,
                "type": rng.choice(("bf16", "bf16", "fp16", "fp32")), "dropped": dropped}
    if op == "experts":
        experts, dim, out = _log(rng, 4, 256), 16 * _log(rng, 16, 448), _log(rng, 64, 4096)
        k = rng.randint(1, min(8, experts))
        while experts * dim * out > 1 << 30:
            out //= 2
        most = min(16384, LARGEST_PRODUCT // (dim * out * k))
        return {"op": op, "tokens": _log(rng, 1, most), "dim": dim, "out": out, "experts": experts, "k": k,
                "type": rng.choice(("bf16", "bf16", "fp32")), "dropped": dropped}
    if op == "product":
        dim, out = 16 * _log(rng, 8, 448), _log(rng, 128, 248320)
        most = min(16384, LARGEST_PRODUCT // (dim * out), 600_000_000 // out)
        return {"op": op, "tokens": _log(rng, 1, most), "dim": dim, "out": out, "type": rng.choice(("bf16", "fp32"))}
    cols = _log(rng, 1000, 248320)
    kind = rng.choice(("bf16", "fp16", "fp32"))
    rows = _log(rng, 1, min(256, LARGEST_LOGITS // (cols * (2 if kind == "fp32" else 1))))
    return {"op": op, "rows": rows, "cols": cols, "type": kind, "history": rng.choice((0, _log(rng, 10, 40000))),
            "biases": rng.choice((0, _log(rng, 1, 300))), "mask": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _choices(case, gen):
    """[tokens, k] distinct experts of each token, some experts more popular than others; -1 where there is none."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    popular = 0.5 * torch.randn(e, generator=gen, device="cuda")
    idx = (popular + torch.randn(t, e, generator=gen, device="cuda")).topk(k, 1).indices
    if case["dropped"] > 0:  # padded tokens have no expert, and a full expert drops single choices
        lost = torch.rand(t, k, generator=gen, device="cuda") < case["dropped"] / 2
        lost |= torch.rand(t, 1, generator=gen, device="cuda") < case["dropped"] / 2
        idx = torch.where(lost, -1, idx)
    return idx.int()


def _order(idx, experts):
    """(slot [tokens, k], source [tokens * k], offsets [experts + 1]) of the choices sorted by expert."""
    flat = idx.reshape(-1).long()
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts)
    source = key.sort(stable=True).indices
    slot = torch.empty_like(source).scatter_(0, source, torch.arange(len(flat), device=flat.device))
    count = torch.zeros(experts + 1, dtype=torch.long, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    ends = count[:experts].cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    source = torch.where(valid[source], source, -1)
    slot = torch.where(valid, slot, -1).view(idx.shape)
    return slot, source, offsets


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    op = case["op"]
    if op in ("sort", "sort step"):
        t, k, d, kind = case["tokens"], case["k"], case["dim"], TYPES[case["type"]]
        s = {"case": case, "idx": _choices(case, gen), "x": normal(t, d).to(kind), "y": normal(t * k, d).to(kind)}
        score = uniform(t, k) + 0.05
        s["weight"] = 2.5 * score / score.sum(1, keepdim=True)
        if op == "sort step":
            s["d_out"] = normal(t, d).to(kind)
            s["d_rows"] = normal(t * k, d).to(kind)
        return s
    if op in ("experts", "product"):
        t, d, n = case["tokens"], case["dim"], case["out"]
        e = case.get("experts", 1)
        # hidden states with a few large channels, as they come
        channel = torch.exp(0.5 * normal(d))
        s = {"case": case, "x": (normal(t, d) * channel).to(torch.bfloat16)}
        weight = torch.empty((e, n, d), dtype=torch.float8_e4m3fn, device=dev)
        rows = max(1, (1 << 26) // d)
        flat = weight.view(e * n, d)
        for at in range(0, e * n, rows):
            stop = min(e * n, at + rows)
            flat[at:stop] = (100 * normal(stop - at, d)).clamp(-448, 448).to(torch.float8_e4m3fn)
        shape = (e, -(-n // BLOCK), -(-d // BLOCK))
        s["w_scale"] = torch.exp(0.3 * normal(*shape)) * (0.01 * d ** -0.5)
        s["weight"] = weight
        if op == "experts":
            s["idx"] = _choices(case, gen)
            s["most"] = int(torch.bincount(s["idx"].clamp(min=-1).view(-1) + 1, minlength=2)[1:].max())
        return s
    rows, cols, length = case["rows"], case["cols"], case["history"]
    s = {"case": case, "logits": (3 * normal(rows, cols)).to(TYPES[case["type"]])}
    if length:
        # tokens of a conversation: a few common ones, many rare ones; the first part is the prompt
        s["tokens"] = (cols * uniform(rows, length) ** 4).long().clamp(max=cols - 1).int()
        s["lengths"] = (length * uniform(rows)).long().clamp(max=length).int() + (length > 1)
        s["lengths"] = s["lengths"].clamp(max=length)
        s["prompts"] = (s["lengths"] * uniform(rows)).int()
        s["repetition"] = 1 + 0.3 * uniform(rows)
        s["presence"] = 0.5 * uniform(rows)
        s["frequency"] = 0.2 * uniform(rows)
        s["repetition"][::4] = 1.0  # requests that ask for none
        s["frequency"][::4] = 0.0
        s["presence"][::4] = 0.0
    if case["biases"]:
        s["bias_tokens"] = (cols * uniform(rows, case["biases"])).long().clamp(max=cols - 1).int()
        s["bias_tokens"][:, -1:] = -1  # a request with fewer biases than the widest
        s["bias_values"] = 5 * normal(rows, case["biases"])
        s["bias_values"][:, 1::7] = -100.0
    if case["mask"]:
        # half of the requests under a grammar that allows few tokens
        allow = uniform(rows, cols) < torch.where(uniform(rows, 1) < 0.5, 0.02, 1.1)
        bits = torch.nn.functional.pad(allow, (0, -cols % 32)).view(rows, -1, 32).long()
        words = (bits << torch.arange(32, device=dev)).sum(2)
        s["allowed"] = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    return s


# ------------------------------------------------------------------ plain forms


def _plain_gather(x, source, k):
    rows = x[(source // k).clamp(min=0)]
    return torch.where(source[:, None] >= 0, rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _plain_combine(y, slot, weight):
    each = torch.where(slot[..., None] >= 0, y[slot.clamp(min=0)].float(), 0.0)
    return (each if weight is None else each * weight[..., None]).sum(1).to(y.dtype)


def _plain_sort(s):
    case = s["case"]
    slot, source, offsets = _order(s["idx"], case["experts"])
    out = {"slot": slot.int(), "source": source.int(), "offsets": offsets.int(),
           "rows": _plain_gather(s["x"], source, case["k"]), "out": _plain_combine(s["y"], slot, s["weight"])}
    if case["op"] == "sort":
        return out
    d = s["d_out"].float()
    token, used = (source // case["k"]).clamp(min=0), source >= 0
    share = s["weight"].view(-1)[source.clamp(min=0)]
    out["d_y"] = torch.where(used[:, None], d[token] * share[:, None], 0.0).to(s["y"].dtype)
    each = torch.where(slot[..., None] >= 0, s["y"][slot.clamp(min=0)].float(), 0.0)
    out["d_weight"] = (each * d[:, None]).sum(2)
    out["d_x"] = _plain_combine(s["d_rows"], slot, None)
    return out


def _plain_quantize(x):
    """The rows' values as their 8 bits and scales stand for them, in 32 bits."""
    rows, d = x.shape
    blocks = torch.nn.functional.pad(x.float(), (0, -d % BLOCK)).view(rows, -1, BLOCK)
    scale = blocks.abs().amax(2, keepdim=True).clamp(min=2.0 ** -100) / 448
    q = (blocks / scale).to(torch.float8_e4m3fn).float()
    return (q * scale).view(rows, -1)[:, :d]


def _plain_weight(weight, scale):
    e, n, d = weight.shape
    wide = scale.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :d]
    return weight.float() * wide


def _plain_product(s):
    case = s["case"]
    x, w = _plain_quantize(s["x"]), _plain_weight(s["weight"], s["w_scale"])
    if case["op"] == "product":
        return {"y": (x @ w[0].t()).to(TYPES[case["type"]])}
    e, most = case["experts"], max(1, s["most"])
    slot, source, offsets = _order(s["idx"], e)
    used = source >= 0
    # each expert's rows in a padded batch of their own
    at = torch.arange(len(source), device=source.device)
    expert = torch.searchsorted(offsets, at, right=True) - 1
    place = torch.where(used, expert * most + at - offsets[expert.clamp(0, e - 1)], e * most)
    padded = torch.zeros((e * most + 1, case["dim"]), device=x.device)
    padded.index_copy_(0, place, torch.where(used[:, None], x[(source // case["k"]).clamp(min=0)], 0.0))
    y = torch.bmm(padded[:-1].view(e, most, -1), w.transpose(1, 2)).view(e * most, -1)
    y = torch.where(used[:, None], y[place.clamp(max=e * most - 1)], 0.0)
    return {"offsets": offsets.int(), "y": y.to(TYPES[case["type"]])}


def _plain_logits(s):
    x = s["logits"].float()
    rows, cols = x.shape
    if "tokens" in s:
        at = torch.arange(s["tokens"].shape[1], device=x.device)[None]
        token = s["tokens"].long()
        here = at < s["lengths"][:, None]
        answered = here & (at >= s["prompts"][:, None])
        count = torch.zeros((rows, cols + 1), device=x.device)
        seen = torch.zeros_like(count).scatter_add_(1, torch.where(here, token, cols), torch.ones_like(token).float())
        count.scatter_add_(1, torch.where(answered, token, cols), torch.ones_like(token).float())
        seen, count = seen[:, :cols] > 0, count[:, :cols]
        r = s["repetition"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None] * count
        x = torch.where(count > 0, x - s["presence"][:, None], x)
    if "bias_tokens" in s:
        token = s["bias_tokens"].long()
        valid = (token >= 0) & (token < cols)
        place = torch.arange(token.shape[1], device=x.device).expand_as(token) + 1
        last = torch.zeros((rows, cols + 1), dtype=torch.long, device=x.device)
        last.scatter_reduce_(1, torch.where(valid, token, cols), place, "amax")
        last = last[:, :cols]
        value = s["bias_values"].gather(1, (last - 1).clamp(min=0))
        x = torch.where(last > 0, x + value, x)
    if "allowed" in s:
        bit = torch.arange(32, device=x.device, dtype=torch.int32)
        allow = ((s["allowed"][..., None] >> bit) & 1).view(rows, -1)[:, :cols]
        x = torch.where(allow > 0, x, -math.inf)
    return {"logits": x.to(s["logits"].dtype)}


# ------------------------------------------------------------------ the framework's calls


def _own_sort(s):
    from wide_bf16_row_gb300 import topk

    case = s["case"]
    order = topk.sort_by_expert(s["idx"], case["experts"])
    out = {"slot": order.slot, "source": order.source, "offsets": order.offsets,
           "rows": topk.gather_tokens(s["x"], order), "out": topk.combine_tokens(s["y"], order, s["weight"])}
    if case["op"] == "sort step":
        out["d_y"], out["d_weight"] = topk.combine_tokens_grad(s["d_out"], s["y"], order, s["weight"])
        out["d_x"] = topk.gather_tokens_grad(s["d_rows"], order)
    return out


def _own_product(s):
    from wide_bf16_row_gb300 import topk

    case = s["case"]
    dtype = TYPES[case["type"]]
    if case["op"] == "product":
        q, scale = topk.quantize_tokens_fp8(s["x"])
        return {"y": topk.product_fp8(q, scale, s["weight"][0], s["w_scale"][0], dtype=dtype)}
    order = topk.sort_by_expert(s["idx"], case["experts"])
    q, scale = topk.quantize_tokens_fp8(s["x"], order)
    return {"offsets": order.offsets,
            "y": topk.product_fp8(q, scale, s["weight"], s["w_scale"], offsets=order.offsets, dtype=dtype)}


def _own_logits(s):
    from wide_bf16_row_gb300 import topk

    return {"logits": topk.penalize_logits(
        s["logits"], tokens=s.get("tokens"), lengths=s.get("lengths"), prompts=s.get("prompts"),
        repetition=s.get("repetition"), presence=s.get("presence"), frequency=s.get("frequency"),
        bias_tokens=s.get("bias_tokens"), bias_values=s.get("bias_values"), allowed=s.get("allowed"))}


def run(state):
    op = state["case"]["op"]
    if op in ("sort", "sort step"):
        return _own_sort(state) if own else _plain_sort(state)
    if op in ("experts", "product"):
        return _own_product(state) if own else _plain_product(state)
    return _own_logits(state) if own else _plain_logits(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op = case["op"]
    size = 4 if case["type"] == "fp32" else 2
    if op in ("sort", "sort step"):
        t, k, d, e = case["tokens"], case["k"], case["dim"], case["experts"]
        n = t * k
        total = 4 * n + 8 * n + 4 * (e + 1) + 4 * n + 2 * (t * d + n * d) * size
        flops = 2 * n * d
        if op == "sort step":
            total += 4 * n + (t * d + n * d + n * d + t * d) * size
            flops += 4 * n * d
        return {"bytes": total, "flops": flops}
    if op in ("experts", "product"):
        t, d, n = case["tokens"], case["dim"], case["out"]
        rows, e = (t * case["k"], case["experts"]) if op == "experts" else (t, 1)
        read = min(e, rows) * (n * d + 4 * -(-n // BLOCK) * -(-d // BLOCK))  # the experts that have rows
        order = 4 * rows + 4 * (e + 1) if op == "experts" else 0
        return {"bytes": 2 * t * d + read + order + rows * n * size, "flops": 2 * rows * d * n}
    rows, cols = case["rows"], case["cols"]
    total = 2 * rows * cols * size
    if case["history"]:
        total += rows * (2 * case["history"] + 20)  # half of it on average, 4 bytes a token
    total += 8 * rows * case["biases"] + (rows * -(-cols // 32) * 4 if case["mask"] else 0)
    return {"bytes": total, "flops": 4 * rows * cols}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_sorted(case, idx):
    """Sorted by hand: the flat places of each expert's choices in turn."""
    flat = idx.cpu().numpy().reshape(-1)
    places = [np.flatnonzero(flat == e) for e in range(case["experts"])]
    ends = np.cumsum([0] + [len(p) for p in places])
    used = np.concatenate(places)
    source = np.full(len(flat), -1, dtype=np.int64)
    source[:len(used)] = used
    slot = np.full(len(flat), -1, dtype=np.int64)
    slot[used] = np.arange(len(used))
    return slot.reshape(idx.shape), source, ends


def _exact_sort(case, s):
    slot, source, offsets = _exact_sorted(case, s["idx"])
    k, used = case["k"], int(offsets[-1])
    token = torch.from_numpy(source[:used] // k).cuda()
    out = {"slot": slot, "source": source, "offsets": offsets}
    rows = torch.zeros((len(source), case["dim"]), dtype=torch.float64, device="cuda")
    rows[:used] = s["x"][token].double()
    out["rows"] = rows
    at = torch.from_numpy(slot).cuda()
    weight = s["weight"].double()

    def back(y, share):
        total = torch.zeros((case["tokens"], case["dim"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            have = torch.nonzero(at[:, j] >= 0)[:, 0]
            part = y[at[have, j]].double()
            total[have] += part * weight[have, j, None] if share else part
        return total

    out["out"] = back(s["y"], True)
    if case["op"] == "sort":
        return out
    d = s["d_out"].double()
    d_y = torch.zeros_like(rows)
    d_y[:used] = d[token] * weight.reshape(-1)[torch.from_numpy(source[:used]).cuda(), None]
    d_weight = torch.zeros_like(weight)
    for j in range(k):
        have = torch.nonzero(at[:, j] >= 0)[:, 0]
        d_weight[have, j] = torch.einsum("td,td->t", d[have], s["y"][at[have, j]].double())
    out.update(d_y=d_y, d_weight=d_weight, d_x=back(s["d_rows"], False))
    return out


def _exact_quantize(x):
    """e4m3 by hand: four significant bits, half to even, steps no finer than 2^-9, at most 448."""
    rows, d = x.shape
    out = torch.empty((rows, d), dtype=torch.float64, device="cuda")
    for at in range(0, d, BLOCK):
        part = x[:, at:at + BLOCK].float()
        # the scale and the quotient are defined in 32 bits
        scale = torch.clamp(part.abs().max(1, keepdim=True).values, min=2.0 ** -100) / 448
        v = (part / scale).double()
        step = torch.ldexp(torch.ones_like(v), torch.clamp(torch.frexp(v).exponent - 4, min=-9))
        out[:, at:at + BLOCK] = torch.clamp(torch.round(v / step) * step, -448, 448) * scale.double()
    return out


def _exact_product(case, s):
    x = _exact_quantize(s["x"])

    def weight(e):
        w, n, d = s["weight"][e].double(), case["out"], case["dim"]
        for i in range(0, n, BLOCK):
            scale = s["w_scale"][e, i // BLOCK].double()
            w[i:i + BLOCK] *= torch.repeat_interleave(scale, BLOCK)[:d]
        return w

    if case["op"] == "product":
        return {"y": x @ weight(0).t()}
    _, source, offsets = _exact_sorted(case, s["idx"])
    y = torch.zeros((len(source), case["out"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = x[torch.from_numpy(source[lo:hi] // case["k"]).cuda()] @ weight(e).t()
    return {"offsets": offsets, "y": y}


def _exact_logits(case, s):
    rows, cols = case["rows"], case["cols"]
    x = s["logits"].double().cpu().numpy()
    host = {name: t.cpu().numpy() for name, t in s.items() if torch.is_tensor(t) and name != "logits"}
    for r in range(rows):
        v = x[r]
        if "tokens" in host:
            said = host["tokens"][r, :host["lengths"][r]]
            seen = np.unique(said)
            rep = float(host["repetition"][r])
            v[seen] = np.where(v[seen] > 0, v[seen] / rep, v[seen] * rep)
            answered, times = np.unique(said[host["prompts"][r]:], return_counts=True)
            v[answered] -= times * float(host["frequency"][r]) + float(host["presence"][r])
        if "bias_tokens" in host:
            biases = dict(zip(host["bias_tokens"][r].tolist(), host["bias_values"][r].tolist()))
            for token, value in biases.items():
                if 0 <= token < cols:
                    v[token] += value
        if "allowed" in host:
            bits = np.unpackbits(host["allowed"][r].astype("<i4").view(np.uint8), bitorder="little")[:cols]
            v[bits == 0] = -np.inf
    return {"logits": x}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("sort", "sort step"):
        return _exact_sort(case, s)
    if case["op"] in ("experts", "product"):
        return _exact_product(case, s)
    return _exact_logits(case, s)
