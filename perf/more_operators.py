"""Measured cases of the operators around an expert layer and of its forms for serving
(partitioned_chip_accumulation_amd.experts).

  norm       h = x + residual (in the rows' type), y = h / sqrt(mean h^2 + eps) weight, row by row;
  norm_int8  the same with y in 8 bits and a scale a row, as the 8-bit products take it;
  norm_grad  the gradients of norm: for its rows (x's and the residual's are one) and its weight,
             from dy and from what arrives at h itself;
  mx4        rows of x quantised to 4 bits (blocks of 32 values with a power of two each), times a
             weight in the same form, dense or by expert;
  few        a whole expert layer for a few tokens: out[t] = sum over its experts j of
             weight[t, j] down[e] act(up[e] x[t]), act(a) = silu(a), or silu(a) b for the two halves
             a and b of up's rows (gated). Weights in 16 bits, in 8 bits with a scale for each
             output channel, or in 4 bits with a power of two for each block of 32.

The 4-bit form: a block's power of two is 2^(floor(log2 max |x|) - 2), and each value of it, divided by
that, the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with its sign, ties to the even code, beyond 6 it is 6.
Two values share a byte, the first one in its lower half; a power of two is a byte, its exponent plus 127.
A row's powers of two start at a multiple of 16 bytes.

A pair whose expert id lies outside [0, experts) is dropped: it adds nothing. ``own`` selects between
the plain form below and the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5

# The largest amount of work of a drawn case (the largest listed ones).
MOST_NORM = 16384 * 4096
MOST_FLOPS = 2 * 8192 * 4 * 4096 * 4096
MOST_FEW = 64 * 3 * 1280 * 2048


def listed():
    return [
        # the norm before an 8-bit layer, one decode step of 32 sequences: the call's latency
        dict(name="norm_decode", op="norm_int8", rows=32, n=4096, dtype="bf16", residual=True),
        # the same for a prompt
        dict(name="norm_int8_prompt", op="norm_int8", rows=8192, n=4096, dtype="fp16",
             residual=True),
        # the norm of a prompt or training batch, with the residual's addition
        dict(name="norm_batch", op="norm", rows=16384, n=4096, dtype="bf16", residual=True),
        # its backward pass in training, odd number of tokens
        dict(name="norm_train", op="norm_grad", rows=8191, n=2048, dtype="bf16", residual=True),
        # one token through a 4-bit dense layer
        dict(name="mx4_decode", op="mx4", tokens=1, top_k=1, experts=0, n=8192, k=4096,
             dtype="bf16", skew=0.0, pad=0.0),
        # a batch of decode steps through 4-bit experts: some tens of rows an expert
        dict(name="mx4_experts", op="mx4", tokens=512, top_k=4, experts=32, n=2560, k=2048,
             dtype="fp16", skew=0.5, pad=0.0),
        # a prompt through a 4-bit dense layer
        dict(name="mx4_prompt", op="mx4", tokens=8192, top_k=1, experts=0, n=8192, k=4096,
             dtype="bf16", skew=0.0, pad=0.0),
        # a prompt batch through 4-bit experts, some padding: bound by the matrix cores
        dict(name="mx4_batch", op="mx4", tokens=8191, top_k=4, experts=16, n=4096, k=4096,
             dtype="bf16", skew=0.3, pad=0.02),
        # a decode step of one sequence through a gated expert layer: bound by reading its weights
        dict(name="few_one", op="few", tokens=1, top_k=8, experts=64, width=2048, hidden=1280,
             weights="16", gated=True, dtype="bf16", skew=0.5, pad=0.0),
        # four sequences, weights in 8 bits
        dict(name="few_int8", op="few", tokens=4, top_k=8, experts=64, width=2048, hidden=1280,
             weights="int8", gated=True, dtype="bf16", skew=0.5, pad=0.0),
        # sixteen sequences, one of them ended, weights in 4 bits
        dict(name="few_mx4", op="few", tokens=16, top_k=4, experts=32, width=2048, hidden=2560,
             weights="mx4", gated=True, dtype="bf16", skew=0.5, pad=0.05),
        # the most tokens that are few, odd sizes, a layer without a gate
        dict(name="few_most", op="few", tokens=63, top_k=2, experts=32, width=2050, hidden=1337,
             weights="16", gated=False, dtype="fp16", skew=0.5, pad=0.0),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_int8", "norm_grad", "mx4", "mx4", "few", "few", "few"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("norm"):
        n = _spread(rng, 16, 2048) * 8 + rng.choice([0, 0, 0, 1, 4])
        return dict(op=op, rows=_spread(rng, 1, min(32768, MOST_NORM // n)), n=n, dtype=dtype,
                    residual=rng.random() < 0.75)
    experts = _spread(rng, 2, 64)
    top_k = min(experts, rng.choice([1, 2, 4, 6, 8]))
    case = dict(op=op, dtype=dtype, skew=round(rng.uniform(0.0, 1.0), 2),
                pad=rng.choice([0.0, 0.0, 0.02, 0.1]))
    # layer widths in steps of 16 mostly, as layers are built, and odd ones besides
    if op == "few":
        width = _spread(rng, 16, 256) * 16 + rng.choice([0, 0, 0, 0, 2, 7])
        hidden = _spread(rng, 8, 256) * 16 + rng.choice([0, 0, 0, 0, 8, 5])
        while 3 * experts * width * hidden > MOST_FEW:
            width, hidden = max(128, width // 2), max(128, hidden // 2)
        return dict(case, tokens=_spread(rng, 1, 64), top_k=top_k, experts=experts, width=width,
                    hidden=hidden, weights=rng.choice(["16", "int8", "mx4"]),
                    gated=rng.random() < 0.75)
    n = _spread(rng, 8, 512) * 16 + rng.choice([0, 0, 0, 0, 2, 7])
    k = _spread(rng, 8, 512) * 16 + rng.choice([0, 0, 0, 0, 8, 5])
    if rng.random() < 0.5:
        experts, top_k, case["pad"] = 0, 1, 0.0
    while experts * n * k > 16 * 4096 * 4096:
        n, k = max(128, n // 2), max(128, k // 2)
    tokens = _spread(rng, 1, max(1, min(16384, MOST_FLOPS // (2 * n * k * top_k))))
    return dict(case, tokens=tokens, top_k=top_k, experts=experts, n=n, k=k)


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
    """counts, offsets, order and place of the pairs sorted by expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    sorted_key, at = torch.sort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    counts = counts.index_add_(0, key, torch.ones_like(key))[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    kept = sorted_key < experts
    order = torch.where(kept, at, -1)
    place = torch.empty_like(at)
    place[at] = torch.where(kept, torch.arange(at.numel(), device="cuda"), -1)
    return [t.int().contiguous() for t in (counts, offsets, order, place.view_as(ids))]


def _in_blocks(x):
    """Rows in blocks of 32, zeros past the end."""
    more = -x.shape[-1] % 32
    if more:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], more)], -1)
    return x.reshape(*x.shape[:-1], -1, 32)


def _quantized_mx4(x):
    """The 4-bit form of rows (32 bits): the values, the codes and the exponents plus 127."""
    blocks = _in_blocks(x)
    top = blocks.abs().amax(-1, keepdim=True)
    exponent = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    a = torch.ldexp(blocks.abs(), -exponent)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = ((a / step).round() * step).clamp(max=6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + (torch.signbit(blocks) * 8).to(torch.uint8)
    values = torch.ldexp(torch.where(torch.signbit(blocks), -a, a), exponent).flatten(-2)
    codes = (code[..., 0::2] + code[..., 1::2] * 16).flatten(-2)
    return values, codes, (exponent.squeeze(-1) + 127).to(torch.uint8)


def _stack(case, g, kind, rows, k):
    """Weights of every expert, or of the one dense layer, as a program holds them. A weight is a
    tensor, or a pair of codes and scales."""
    shape = (case["experts"], rows, k) if case["experts"] else (rows, k)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if kind == "int8":
        q = (normal(*shape) * 40.0).round_().clamp_(-127, 127).to(torch.int8)
        scale = torch.rand(*shape[:-1], generator=g, device="cuda") + 0.5
        return q, scale / (40 * k ** 0.5)
    if kind == "mx4":
        each = [_quantized_mx4(normal(rows, k) * k ** -0.5)[1:]
                for _ in range(max(1, case["experts"]))]
        codes, powers = (torch.stack(t) if case["experts"] else t[0] for t in zip(*each))
        blocks = powers.shape[-1]
        return codes, torch.nn.functional.pad(powers, (0, -blocks % 16))[..., :blocks]
    return (normal(*shape) * k ** -0.5).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if op.startswith("norm"):
        rows, n = case["rows"], case["n"]
        # a residual stream: a few channels larger than the rest, rows of different size
        wide = 1.0 + 8.0 * (torch.randn(n, generator=g, device="cuda").abs() > 2.5)
        high = torch.rand(rows, 1, generator=g, device="cuda") + 0.5
        s["x"] = normal(rows, n)
        s["residual"] = normal(rows, n, scale=wide * high) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dtype)
        if op == "norm_grad":
            s["h"] = s.pop("x") if s["residual"] is None else s.pop("x") + s.pop("residual")
            s["dy"] = normal(rows, n)
            s["dh"] = normal(rows, n) if case["residual"] else None
        return s
    if case["experts"]:
        s["ids"] = _route(case, g)
    if op == "few":
        width, hidden = case["width"], case["hidden"]
        s["x"] = normal(case["tokens"], width)
        s["up"] = _stack(case, g, case["weights"], hidden * (2 if case["gated"] else 1), width)
        s["down"] = _stack(case, g, case["weights"], width, hidden)
        s["by"] = normal(case["tokens"], case["top_k"]).float().softmax(dim=1)
        return s
    if case["experts"]:
        s["counts"], s["offsets"], s["order"], s["place"] = _sorted(s["ids"], case["experts"])
    # activations with a few channels larger than the rest
    k = case["k"]
    wide = 1.0 + 8.0 * (torch.randn(k, generator=g, device="cuda").abs() > 2.5)
    s["x"] = normal(case["tokens"], k, scale=wide)
    s["wq"], s["ws"] = _stack(case, g, "mx4", case["n"], k)
    return s


# ---------------------------------------------------------------------------
# The library's calls.

def _run_own(s):
    from partitioned_chip_accumulation_amd import experts
    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, h = experts.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        return (y, h) if case["residual"] else y
    if op == "norm_int8":
        xq, sx, h = experts.rms_norm_int8(s["x"], s["weight"], s["residual"], eps=EPS)
        # the values that the 8 bits stand for, in the rows' type
        values = torch.mul(xq, sx.view(-1, 1), out=torch.empty_like(s["x"]))
        return (values, sx, h) if case["residual"] else (values, sx)
    if op == "norm_grad":
        return experts.rms_norm_backward(s["dy"], s["h"], s["weight"], s["dh"], eps=EPS)
    if op == "few":
        return experts.few_tokens(s["x"], s["up"], s["down"], s["ids"], s["by"],
                                  gated=case["gated"])
    g = experts.Groups(s["counts"], s["offsets"], s["order"], s["place"]) \
        if case["experts"] else None
    xq, xs = experts.quantize_mx4(s["x"])
    return experts.mx4_matmul(xq, xs, s["wq"], s["ws"], g, gather=g is not None,
                              out_dtype=DTYPES[case["dtype"]])


# ---------------------------------------------------------------------------
# The plain form.

def _plain_norm(s, dtype):
    x = s["x"].float()
    h = x if s["residual"] is None else (x + s["residual"].float()).to(dtype).float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    return h, y


def _plain_norm_grad(s, dtype):
    h, dy, w = s["h"].float(), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    dn = dy * w
    dx = r * dn - h * (r * r * r * (dn * h).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(dtype), (dy * h * r).sum(0).to(dtype)


def _plain_int8(s, dtype):
    h, y = _plain_norm(s, dtype)
    scale = y.abs().amax(1) / 127.0
    # 64 bits: the quotient rounded once, a value next to the middle of two steps
    q = (y.double() / scale.double().view(-1, 1)).round().clamp(-127, 127)
    values = torch.where(scale.view(-1, 1) > 0, q * scale.double().view(-1, 1), 0.0).to(dtype)
    return (values, scale) if s["residual"] is None else (values, scale, h.to(dtype))


def _weight(w, k):
    """A stack of weights as 32-bit values, [..., rows, k]."""
    if isinstance(w, torch.Tensor):
        return w.float()
    q, scale = w
    if q.dtype == torch.int8:
        return q.float() * scale.unsqueeze(-1)
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    values = torch.cat([grid, -grid])[codes].unflatten(-1, (-1, 32))
    return torch.ldexp(values, scale.int().unsqueeze(-1) - 127).flatten(-2)[..., :k]


def _padded_places(counts, offsets):
    """Each sorted pair's expert and its place within the expert's rows, and the largest group."""
    offsets = offsets.long()
    kept = int(offsets[-1])
    at = torch.arange(kept, device="cuda")
    expert = (at.view(-1, 1) >= offsets[1:].view(1, -1)).sum(1) if kept else at
    return kept, expert, at - offsets[expert], max(1, int(counts.max()))


def _by_expert(rows, w, where):
    """Sorted rows times their experts' weights [experts, n, k], as [kept, n]."""
    kept, expert, within, most = where
    padded = torch.zeros(w.shape[0], most, rows.shape[1], device="cuda")
    padded[expert, within] = rows[:kept]
    return torch.bmm(padded, w.transpose(1, 2).contiguous())[expert, within]


def _plain_mx4(s, dtype):
    case = s["case"]
    k = case["k"]
    x = _quantized_mx4(s["x"].float())[0][:, :k]
    w = _weight((s["wq"], s["ws"]), k)
    if not case["experts"]:
        return (x @ w.t().contiguous()).to(dtype)
    where = _padded_places(s["counts"], s["offsets"])
    y = torch.zeros(s["order"].numel(), case["n"], dtype=dtype, device="cuda")
    token = s["order"][:where[0]].long() // case["top_k"]
    y[:where[0]] = _by_expert(x[token], w, where).to(dtype)
    return y


def _plain_few(s, dtype):
    case = s["case"]
    hidden, top_k = case["hidden"], case["top_k"]
    # the experts that have a token, numbered anew: no other's weights are used
    ids = s["ids"].long()
    valid = (ids >= 0) & (ids < case["experts"])
    used, again = torch.unique(torch.where(valid, ids, 0), return_inverse=True)

    def picked(w):
        return w[used] if isinstance(w, torch.Tensor) else tuple(t[used] for t in w)

    counts, offsets, order, _ = _sorted(torch.where(valid, again, -1), used.numel())
    where = _padded_places(counts, offsets)
    pair = order[:where[0]].long()
    a = _by_expert(s["x"].float()[pair // top_k], _weight(picked(s["up"]), case["width"]), where)
    h = a[:, :hidden] * torch.sigmoid(a[:, :hidden])
    if case["gated"]:
        h = h * a[:, hidden:]
    y = _by_expert(h, _weight(picked(s["down"]), hidden), where)
    each = torch.zeros(ids.numel(), case["width"], device="cuda")
    each[pair] = y * s["by"].reshape(-1)[pair].unsqueeze(1)
    return each.view(case["tokens"], top_k, -1).sum(1).to(dtype)


def run(state):
    if own:
        return _run_own(state)
    dtype = DTYPES[state["case"]["dtype"]]
    op = state["case"]["op"]
    if op == "norm":
        h, y = _plain_norm(state, dtype)
        return y.to(dtype) if state["residual"] is None else (y.to(dtype), h.to(dtype))
    plain = {"norm_int8": _plain_int8, "norm_grad": _plain_norm_grad, "mx4": _plain_mx4,
             "few": _plain_few}
    return plain[op](state, dtype)


# ---------------------------------------------------------------------------
# What a pass cannot do without.

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        rows, n = case["rows"], case["n"]
        added = 2 if case["residual"] else 0
        if op == "norm_grad":
            return {"bytes": rows * n * (6.0 + added) + 4.0 * n, "flops": 11.0 * rows * n}
        out = 2.0 if op == "norm" else 1.0 + 4.0 / n
        return {"bytes": rows * n * (2.0 + 2 * added + out) + 2.0 * n, "flops": 5.0 * rows * n}
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    pairs = tokens * top_k
    kept = pairs * (1.0 - case["pad"])
    # the experts that the tokens can be expected to touch
    touched = experts * (1.0 - (1.0 - top_k / experts) ** tokens) if experts else 1.0
    if op == "few":
        width, hidden = case["width"], case["hidden"]
        values = width * hidden * (3 if case["gated"] else 2)
        each = {"16": 2.0, "int8": 1.0, "mx4": 0.5 + 1 / 32}[case["weights"]]
        return {"bytes": touched * values * each + 4.0 * tokens * width + 8.0 * pairs,
                "flops": 2.0 * kept * values}
    n, k = case["n"], case["k"]
    moved = 2.0 * tokens * k + touched * n * k * (0.5 + 1 / 32) + 2.0 * pairs * n
    return {"bytes": moved + (4.0 * pairs if experts else 0.0), "flops": 2.0 * kept * n * k}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.

def _exact_values(w, k):
    if isinstance(w, torch.Tensor):
        return w.double()
    q, scale = w
    if q.dtype == torch.int8:
        return q.double() * scale.double().unsqueeze(-1)
    out = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device="cuda")
    for half in (0, 1):
        code = (q.int() >> (4 * half)) & 15
        # one bit of fraction, two of exponent (of bias 1, 0: no hidden bit), the sign
        exponent, fraction = (code >> 1) & 3, (code & 1).double()
        size = torch.where(exponent == 0, fraction / 2,
                           (1 + fraction / 2) * 2.0 ** (exponent.double() - 1))
        out[..., half::2] = torch.where(code >= 8, -size, size)
    out *= (2.0 ** (scale.double() - 127)).repeat_interleave(32, -1)
    return out[..., :k]


def _exact_mx4(x):
    """Rows after quantising, by the middles between two values of the 4-bit form."""
    blocks = _in_blocks(x)
    top = blocks.abs().amax(-1, keepdim=True)
    power = torch.where(top > 0, 2.0 ** torch.floor(torch.log2(top)), 1.0) / 4
    a = blocks.abs() / power
    out = torch.zeros_like(a)
    grid = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    for code in range(1, 8):
        middle = (grid[code - 1] + grid[code]) / 2
        reached = a >= middle if code % 2 == 0 else a > middle
        out = torch.where(reached, grid[code], out)
    return (out * power * blocks.sign()).flatten(-2)[:, :x.shape[1]]


def _exact_norm(s, dtype):
    x = s["x"].double()
    h = x if s["residual"] is None else (x + s["residual"].double()).to(dtype).double()
    size = torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS)
    return h, h / size * s["weight"].double()


def _exact_silu(a):
    return a / (1 + torch.exp(-a))


def exact(case, seed):
    s = prepare(case, seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "norm":
        h, y = _exact_norm(s, dtype)
        return (y, h) if case["residual"] else y
    if op == "norm_int8":
        h, y = _exact_norm(s, dtype)
        # the scale is held in 32 bits by definition: the nearest 32-bit value of max / 127
        scale = (y.abs().amax(1) / 127).float().double()
        steps = y / torch.where(scale > 0, scale, 1.0).view(-1, 1)
        values = torch.round(steps).clamp(-127, 127) * scale.view(-1, 1)
        return (values, scale, h) if case["residual"] else (values, scale)
    if op == "norm_grad":
        h, dy, w = s["h"].double(), s["dy"].double(), s["weight"].double()
        size = torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS)
        unit = h / size
        along = (dy * w * unit).sum(1, keepdim=True) / h.shape[1]
        dx = (dy * w - unit * along) / size
        return dx if s["dh"] is None else dx + s["dh"].double(), (dy * unit).sum(0)
    top_k = case["top_k"]
    if op == "few":
        width, hidden = case["width"], case["hidden"]
        out = torch.zeros(case["tokens"], width, dtype=torch.float64, device="cuda")
        for e in sorted(set(s["ids"].reshape(-1).tolist())):
            if not 0 <= e < case["experts"]:
                continue
            pick = [w[e] if isinstance(w, torch.Tensor) else (w[0][e], w[1][e])
                    for w in (s["up"], s["down"])]
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            a = s["x"][t].double() @ _exact_values(pick[0], width).t().contiguous()
            h = _exact_silu(a[:, :hidden]) * (a[:, hidden:] if case["gated"] else 1.0)
            y = h @ _exact_values(pick[1], hidden).t().contiguous()
            out.index_add_(0, t, y * s["by"][t, j].double().unsqueeze(1))
        return out
    n, k = case["n"], case["k"]
    x = _exact_mx4(s["x"].double())
    if not case["experts"]:
        return x @ _exact_values((s["wq"], s["ws"]), k).t().contiguous()
    out = torch.zeros(case["tokens"] * top_k, n, dtype=torch.float64, device="cuda")
    first = s["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = first[e], first[e + 1]
        if a < b:
            w = _exact_values((s["wq"][e], s["ws"][e]), k)
            out[a:b] = x[s["order"][a:b].long() // top_k] @ w.t().contiguous()
    return out
