"""Measured cases of the expert-layer operators (partitioned_chip_accumulation_amd.experts).

A mixture-of-experts layer sends each token to its top_k experts. Its operators are

  group         count the (token, choice) pairs of each expert and sort them by expert;
  matmul        y[p] = x[token(p)] w[e(p)]^T, the rows of one expert after another;
  matmul_dx     the gradient of its rows, dx[p] = dy[p] w[e(p)];
  matmul_dw     the gradient of its weights, dw[e] = sum over e's rows of dy[p]^T x[token(p)];
  combine       out[t] = sum over choices j of weight[t, j] y[place(t, j)];
  combine_grad  its gradients with respect to y and to the weights;
  int8          rows of x quantised to 8 bits with a scale each, times an 8-bit weight with a
                scale for each output channel, dense or by expert.

A pair whose expert id lies outside [0, experts) is dropped: it has no place (-1), its row adds
nothing, and the rows of the sorted arrays past the last kept pair are zero.

``own`` selects between the plain form below and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# The largest amount of work of a drawn case (the largest listed ones).
MOST_FLOPS = 2 * 8192 * 4 * 4096 * 4096
MOST_PAIRS = 65536 * 8
MOST_COMBINE = 16384 * 4 * 4096


def listed():
    return [
        # one decode step of 32 sequences: what counts is the latency of the call
        dict(name="group_decode", op="group", tokens=32, top_k=8, experts=256, skew=0.5, pad=0.0),
        # a long prompt batch, 3% of it padding without an expert
        dict(name="group_prompt", op="group", tokens=65521, top_k=8, experts=256, skew=0.5,
             pad=0.03),
        # expert outputs back to the tokens of a prompt batch
        dict(name="combine_prompt", op="combine", tokens=16384, top_k=4, experts=32, n=4096,
             dtype="bf16", skew=0.5, pad=0.0),
        # the same step's backward pass in training, odd token count, some padding
        dict(name="combine_train", op="combine_grad", tokens=8191, top_k=8, experts=64, n=2048,
             dtype="fp16", skew=0.5, pad=0.02),
        # a decode step of 4 sequences: few rows, bound by reading the weights it touches
        dict(name="matmul_decode", op="matmul", tokens=4, top_k=8, experts=64, n=2560, k=2048,
             dtype="bf16", skew=0.5, pad=0.0),
        # a small prompt: about a hundred rows an expert, every group ragged
        dict(name="matmul_ragged", op="matmul", tokens=1021, top_k=4, experts=32, n=1344, k=2048,
             dtype="fp16", skew=0.7, pad=0.02),
        # a training or prompt batch: bound by the matrix cores
        dict(name="matmul_batch", op="matmul", tokens=8192, top_k=4, experts=16, n=4096, k=4096,
             dtype="bf16", skew=0.3, pad=0.0),
        # the gradient of a training batch's rows
        dict(name="matmul_dx_train", op="matmul_dx", tokens=8192, top_k=4, experts=16, n=2560,
             k=4096, dtype="bf16", skew=0.3, pad=0.0),
        # the gradient of many experts' weights, some of them with few rows
        dict(name="matmul_dw_train", op="matmul_dw", tokens=8192, top_k=2, experts=32, n=2560,
             k=2048, dtype="fp16", skew=1.0, pad=0.01),
        # one token through an 8-bit dense layer
        dict(name="int8_decode", op="int8", tokens=1, top_k=1, experts=0, n=8192, k=4096,
             dtype="bf16", skew=0.0, pad=0.0),
        # a prompt through an 8-bit dense layer
        dict(name="int8_prompt", op="int8", tokens=8192, top_k=1, experts=0, n=8192, k=4096,
             dtype="bf16", skew=0.0, pad=0.0),
        # a batch of decode steps through 8-bit experts: some tens of rows an expert
        dict(name="int8_experts", op="int8", tokens=512, top_k=4, experts=32, n=2560, k=2048,
             dtype="fp16", skew=0.5, pad=0.0),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["group", "combine", "combine_grad", "matmul", "matmul", "matmul_dx",
                     "matmul_dw", "int8", "int8"])
    case = dict(op=op, skew=round(rng.uniform(0.0, 1.0), 2),
                pad=rng.choice([0.0, 0.0, 0.02, 0.1]))
    experts = _spread(rng, 2, 256)
    top_k = min(experts, rng.choice([1, 2, 4, 6, 8]))
    if op == "group":
        return dict(case, tokens=_spread(rng, 1, MOST_PAIRS // top_k), top_k=top_k,
                    experts=experts)
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("combine"):
        n = _spread(rng, 16, 1024) * 8 + rng.choice([0, 0, 0, 1, 4])
        tokens = _spread(rng, 1, min(32768, MOST_COMBINE // (n * top_k)))
        return dict(case, tokens=tokens, top_k=top_k, experts=experts, n=n, dtype=dtype)
    # layer widths in steps of 16 mostly, as layers are built, and odd ones besides
    n = _spread(rng, 8, 512) * 16 + rng.choice([0, 0, 0, 0, 2, 7])
    k = _spread(rng, 8, 512) * 16 + rng.choice([0, 0, 0, 0, 8, 5])
    if op == "int8":
        dense = rng.random() < 0.5
        experts, top_k = (0, 1) if dense else (min(experts, 64), top_k)
        case["pad"] = 0.0 if dense else case["pad"]
    else:
        experts = min(experts, 64)
    if experts:
        top_k = min(top_k, experts)
        while experts * n * k > 64 * 2560 * 2048:
            n = max(128, n // 2)
            k = max(128, k // 2)
    tokens = _spread(rng, 1, max(1, min(16384, MOST_FLOPS // (2 * n * k * top_k))))
    return dict(case, tokens=tokens, top_k=top_k, experts=experts, n=n, k=k, dtype=dtype)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * (int(seed) + 1))


def _route(case, g):
    """Expert ids as a router picks them: distinct experts for a token, some experts more popular
    than others, padding tokens without one (-1)."""
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    rank = torch.randperm(experts, generator=g, device="cuda").float()
    uniform = torch.rand(tokens, experts, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    score = -torch.log(-torch.log(uniform)) - case["skew"] * torch.log1p(rank)
    ids = score.topk(top_k, dim=1).indices.int()
    gone = torch.rand(tokens, 1, generator=g, device="cuda") < case["pad"]
    return torch.where(gone, -1, ids).contiguous()


def _sorted(ids, experts):
    """counts, offsets, order and place of the pairs sorted by expert, for a prepared case."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    sorted_key, at = torch.sort(key, stable=True)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    kept = sorted_key < experts
    order = torch.where(kept, at, -1)
    place = torch.empty_like(at)
    place[at] = torch.where(kept, torch.arange(at.numel(), device="cuda"), -1)
    return [t.int().contiguous() for t in (counts, offsets, order, place.view_as(ids))]


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case=case)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if case["experts"]:
        s["ids"] = _route(case, g)
        if op == "group":
            return s
        s["counts"], s["offsets"], s["order"], s["place"] = _sorted(s["ids"], case["experts"])
    tokens, pairs, n = case["tokens"], case["tokens"] * case["top_k"], case["n"]
    dtype = DTYPES[case["dtype"]]
    kept = None if not case["experts"] else (s["order"] >= 0).view(-1, 1)
    if op.startswith("combine"):
        s["y"] = torch.where(kept, normal(pairs, n), 0.0).to(dtype)
        s["weights"] = normal(tokens, case["top_k"]).softmax(dim=1)
        if op == "combine_grad":
            s["dout"] = normal(tokens, n, dtype=dtype)
        return s
    k = case["k"]
    if op == "int8":
        # activations with a few channels larger than the rest, weights quantised by channel
        s["x"] = (normal(tokens, k) * (1.0 + 8.0 * (normal(k).abs() > 2.5))).to(dtype)
        shape = (case["experts"], n, k) if case["experts"] else (n, k)
        s["wq"] = normal(*shape, scale=40.0).round_().clamp_(-127, 127).to(torch.int8)
        s["sw"] = (torch.rand(*shape[:-1], generator=g, device="cuda") + 0.5) / (40 * k ** 0.5)
        return s
    if op in ("matmul", "matmul_dw"):
        s["x"] = normal(tokens, k, dtype=dtype)
    if op in ("matmul", "matmul_dx"):
        s["w"] = normal(case["experts"], n, k, scale=k ** -0.5, dtype=dtype)
    if op in ("matmul_dx", "matmul_dw"):
        s["dy"] = torch.where(kept, normal(pairs, n), 0.0).to(dtype)
    return s


# ---------------------------------------------------------------------------
# The library's calls.

def _run_own(s):
    from partitioned_chip_accumulation_amd import experts
    case = s["case"]
    op = case["op"]
    if op == "group":
        g = experts.group_rows(s["ids"], case["experts"])
        return g.counts, g.offsets, g.order, g.place
    g = experts.Groups(s["counts"], s["offsets"], s["order"], s["place"]) \
        if case["experts"] else None
    if op == "combine":
        return experts.combine(s["y"], g, s["weights"])
    if op == "combine_grad":
        return experts.combine_backward(s["dout"], s["y"], g, s["weights"])
    if op == "matmul":
        return experts.matmul(s["x"], s["w"], g, gather=True)
    if op == "matmul_dx":
        return experts.matmul_dx(s["dy"], s["w"], g)
    if op == "matmul_dw":
        return experts.matmul_dw(s["dy"], s["x"], g, gather=True)
    xq, sx = experts.quantize_rows(s["x"])
    y = experts.int8_matmul(xq, sx, s["wq"], s["sw"], g, gather=g is not None,
                            out_dtype=DTYPES[case["dtype"]])
    return y, sx


# ---------------------------------------------------------------------------
# The plain form.

def _plain_group(s):
    experts = s["case"]["experts"]
    flat = s["ids"].reshape(-1).long()
    m = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = counts.cumsum(0) - counts
    at = torch.argsort(key, stable=True)
    kept = key[at] < experts
    order = torch.where(kept, at, -1)
    place = torch.empty_like(at)
    place[at] = torch.where(kept, torch.arange(m, device="cuda"), -1)
    return (counts[:experts].int(), offsets.int(), order.int(),
            place.view_as(s["ids"]).int())


def _padded_places(s):
    """Each sorted pair's expert and its place within the expert's rows, and the largest group."""
    counts, offsets = s["counts"].long(), s["offsets"].long()
    kept = int(offsets[-1])
    at = torch.arange(kept, device="cuda")
    expert = (at.view(-1, 1) >= offsets[1:].view(1, -1)).sum(1) if kept else at
    return kept, expert, at - offsets[expert], int(counts.max())


def _padded(rows, s, where):
    """Rows of the sorted pairs as one [experts, largest group, width] array, zeros after each."""
    kept, expert, within, most = where
    out = torch.zeros(s["case"]["experts"], max(1, most), rows.shape[1], dtype=rows.dtype,
                      device="cuda")
    out[expert, within] = rows[:kept]
    return out


def _rows(padded, s, where):
    """The sorted pairs' rows out of the padded array; zero past the last kept pair."""
    kept, expert, within, _ = where
    out = torch.zeros(s["order"].numel(), padded.shape[2], dtype=padded.dtype, device="cuda")
    out[:kept] = padded[expert, within]
    return out


def _gathered(x, s):
    token = (s["order"].long().clamp(min=0)) // s["case"]["top_k"]
    return x[token]


def _plain_matmul(s, dtype):
    where = _padded_places(s)
    x = _padded(_gathered(s["x"], s).float(), s, where)
    w = s["w"].float().transpose(1, 2).contiguous()
    return _rows(torch.bmm(x, w), s, where).to(dtype)


def _plain_dx(s, dtype):
    where = _padded_places(s)
    return _rows(torch.bmm(_padded(s["dy"].float(), s, where), s["w"].float()), s, where).to(dtype)


def _plain_dw(s, dtype):
    where = _padded_places(s)
    x = _padded(_gathered(s["x"], s).float(), s, where)
    dy = _padded(s["dy"].float(), s, where).transpose(1, 2).contiguous()
    return torch.bmm(dy, x).to(dtype)


def _plain_combine(s, dtype):
    place = s["place"].long()
    y = s["y"].float()[place.clamp(min=0)]
    weight = torch.where(place >= 0, s["weights"], 0.0)
    return (y * weight.unsqueeze(2)).sum(1).to(dtype)


def _plain_combine_grad(s, dtype):
    place, top_k = s["place"].long(), s["case"]["top_k"]
    dout = s["dout"].float()
    dot = (s["y"].float()[place.clamp(min=0)] * dout.unsqueeze(1)).sum(2)
    dweights = torch.where(place >= 0, dot, 0.0)
    order = s["order"].long()
    weight = torch.where(order >= 0, s["weights"].reshape(-1)[order.clamp(min=0)], 0.0)
    dy = dout[order.clamp(min=0) // top_k] * weight.view(-1, 1)
    return dy.to(dtype), dweights


def _plain_int8(s, dtype):
    # 64 bits: the quotient rounded once, a value next to the middle of two steps, sums past 2^24
    x = s["x"].float()
    scale = (x.abs().amax(1).double() / 127.0).float()
    q = torch.where(scale.view(-1, 1) > 0,
                    (x.double() / scale.double().view(-1, 1)).round().clamp(-127, 127), 0.0)
    if not s["case"]["experts"]:
        y = q @ s["wq"].t().contiguous().double()
        return (y * scale.double().view(-1, 1) * s["sw"].double()).to(dtype), scale
    where = _padded_places(s)
    y = torch.bmm(_padded(_gathered(q, s), s, where),
                  s["wq"].transpose(1, 2).contiguous().double())
    y = y * _padded(_gathered(scale.view(-1, 1), s).double(), s, where)
    return _rows(y * s["sw"].double().unsqueeze(1), s, where).to(dtype), scale


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "group":
        return _plain_group(state)
    plain = {"matmul": _plain_matmul, "matmul_dx": _plain_dx, "matmul_dw": _plain_dw,
             "combine": _plain_combine, "combine_grad": _plain_combine_grad, "int8": _plain_int8}
    return plain[op](state, DTYPES[state["case"]["dtype"]])


# ---------------------------------------------------------------------------
# What a pass cannot do without.

def work(case):
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    pairs = tokens * top_k
    op = case["op"]
    if op == "group":
        return {"bytes": 12.0 * pairs + 8.0 * experts + 4, "flops": 0.0}
    n = case["n"]
    kept = pairs * (1.0 - case["pad"])
    if op == "combine":
        return {"bytes": 2.0 * n * (kept + tokens) + 8.0 * pairs, "flops": 2.0 * kept * n}
    if op == "combine_grad":
        return {"bytes": 2.0 * n * (kept + tokens + pairs) + 16.0 * pairs,
                "flops": 3.0 * kept * n}
    k = case["k"]
    flops = 2.0 * kept * n * k
    # the experts that the tokens can be expected to touch
    touched = experts * (1.0 - (1.0 - top_k / experts) ** tokens) if experts else 1.0
    index = 4.0 * pairs if experts else 0.0
    if op == "matmul":
        moved = 2.0 * (tokens * k + touched * n * k + pairs * n)
    elif op == "matmul_dx":
        moved = 2.0 * (pairs * n + touched * n * k + pairs * k)
        index = 0.0
    elif op == "matmul_dw":
        moved = 2.0 * (pairs * n + tokens * k + experts * n * k)
    else:
        moved = 2.0 * tokens * k + touched * (n * k + 4.0 * n) + 2.0 * pairs * n + 4.0 * tokens
    return {"bytes": moved + index, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, expert by expert.

def _exact_group(s):
    experts = s["case"]["experts"]
    ids = s["ids"].cpu().numpy()
    flat = ids.reshape(-1)
    lists = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(lists, kind="stable")
    counts = np.array([np.count_nonzero(lists == e) for e in range(experts)], dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    order[offsets[-1]:] = -1
    place = np.full(flat.size, -1, dtype=np.int32)
    place[order[:offsets[-1]]] = np.arange(offsets[-1])
    return counts, offsets, order.astype(np.int32), place.reshape(ids.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "group":
        return _exact_group(s)
    top_k, tokens = case["top_k"], case["tokens"]
    if op == "combine":
        out = torch.zeros(tokens, case["n"], dtype=torch.float64, device="cuda")
        for j in range(top_k):
            p = s["place"][:, j].long()
            t = torch.nonzero(p >= 0).view(-1)
            out[t] += s["weights"][t, j].double().view(-1, 1) * s["y"][p[t]].double()
        return out
    if op == "combine_grad":
        dy = torch.zeros(tokens * top_k, case["n"], dtype=torch.float64, device="cuda")
        dweights = torch.zeros(tokens, top_k, dtype=torch.float64, device="cuda")
        for j in range(top_k):
            p = s["place"][:, j].long()
            t = torch.nonzero(p >= 0).view(-1)
            d = s["dout"][t].double()
            dy[p[t]] = d * s["weights"][t, j].double().view(-1, 1)
            dweights[t, j] = (d * s["y"][p[t]].double()).sum(1)
        return dy, dweights
    if op == "int8":
        top = s["x"].double().abs().amax(1)
        # the scale is held in 32 bits by definition: the nearest 32-bit value of top / 127
        scale = (top / 127.0).float().double().view(-1, 1)
        steps = s["x"].double() / torch.where(scale == 0, 1.0, scale)
        low = steps.floor()
        up = (steps - low > 0.5) | ((steps - low == 0.5) & (low % 2 != 0))
        value = (low + up.double()).clamp(-127, 127) * scale
        if not case["experts"]:
            weight = s["wq"].double() * s["sw"].double().view(-1, 1)
            return value @ weight.t().contiguous(), scale.view(-1)
    pairs = tokens * top_k
    n, k = case["n"], case["k"]
    shape = {"matmul": (pairs, n), "int8": (pairs, n), "matmul_dx": (pairs, k),
             "matmul_dw": (case["experts"], n, k)}[op]
    out = torch.zeros(*shape, dtype=torch.float64, device="cuda")
    first = s["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        token = s["order"][a:b].long() // top_k
        if op == "matmul":
            out[a:b] = s["x"][token].double() @ s["w"][e].double().t().contiguous()
        elif op == "matmul_dx":
            out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
        elif op == "matmul_dw":
            out[e] = s["dy"][a:b].double().t().contiguous() @ s["x"][token].double()
        else:
            weight = s["wq"][e].double() * s["sw"][e].double().view(-1, 1)
            out[a:b] = value[token] @ weight.t().contiguous()
    return (out, scale.view(-1)) if op == "int8" else out
