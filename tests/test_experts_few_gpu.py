"""The whole layer for a few tokens against its definition in 64 bits, expert by expert.

Tolerances, from the arithmetic alone. A 32-bit sum of m products is off by at most m steps of 2^-23 of
the sum of their magnitudes (twice as many products where float16 tokens are split in two parts); each
scale or weight is one more rounding of 2^-24. silu's slope is at most 1.1, and exp, the sum, the
division and the product after it are within 8 + |a| steps of 2^-24 of their result. The result is
rounded to the type once: half a step of the value, or half the smallest subnormal. h is allowed as much;
test_h_keeps_what_the_type_does_not holds it to two values of the type, of which the second is off by half a
step of at most half a step.
"""
from __future__ import annotations

import pytest
import torch

import mx4_reference
from partitioned_chip_accumulation_amd import experts, hist
from test_experts_gpu import normal, route

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
KINDS = ["16", "int8", "mx4"]


def make(seed, kind, num, rows, k, dtype):
    """A weight as few_tokens takes it, and its values in 64 bits."""
    if kind == "16":
        w = normal(seed, num, rows, k, dtype=dtype, scale=k**-0.5)
        return w, w.double()
    if kind == "int8":
        q = normal(seed, num, rows, k, scale=40).round().clamp(-127, 127).to(torch.int8)
        scale = (normal(seed + 1, num, rows).abs() + 0.5) / (40 * k**0.5)
        return (q, scale), q.double() * scale.double().unsqueeze(2)
    w = normal(seed, num * rows, k, dtype=torch.bfloat16, scale=k**-0.5)
    q, powers = (t.view(num, rows, -1) for t in experts.quantize_mx4(w))
    values = mx4_reference.values(q.cpu().numpy(), powers.cpu().numpy())[..., :k]
    return (q, powers), torch.from_numpy(values.copy()).cuda()


def layer(x, up, down, ids, by, gated, split, step=None):
    """The result in 64 bits and how far a result may be off before its own rounding; step: h's own,
    relative to it."""
    dtype, num, hidden = x.dtype, up.shape[0], down.shape[2]
    info = torch.finfo(dtype)
    step = info.eps / 2 if step is None else step
    out = torch.zeros(x.shape[0], down.shape[1], dtype=torch.float64, device="cuda")
    room, u = torch.zeros_like(out), 2.0**-24
    d = x.double()
    for e in range(num):
        for j in range(ids.shape[1]):
            t = torch.nonzero(ids[:, j] == e).view(-1)
            if t.numel() == 0:
                continue
            a = d[t] @ up[e].t().contiguous()
            off = (d[t].abs() @ up[e].abs().t().contiguous()) * ((2 * split * x.shape[1] + 2) * u)
            gate = a[:, :hidden]
            s = gate * torch.sigmoid(gate)
            off_s = 1.1 * off[:, :hidden] + s.abs() * (8 + gate.abs()) * u
            h, off_h = s, off_s
            if gated:
                h = s * a[:, hidden:]
                off_h = off_s * (a[:, hidden:].abs() + off[:, hidden:]) + s.abs() * off[:, hidden:]
            off_h = off_h * (1 + info.eps) + h.abs() * step + info.smallest_normal * info.eps
            w, size = by[t, j].double().unsqueeze(1), down[e].abs().t().contiguous()
            out.index_add_(0, t, w * (h @ down[e].t().contiguous()))
            terms = 2 * split * hidden * ids.shape[1] + 2 * ids.shape[1] + 8
            room.index_add_(0, t, w.abs() * (off_h @ size + (h.abs() + off_h) @ size * (terms * u)))
    return out, room


def check(got, want, room):
    info = torch.finfo(got.dtype)
    room = room * (1 + info.eps) + want.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2
    assert got.shape == want.shape
    bad = ~((got.double() - want).abs() <= room)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], room[bad][:4],
                           torch.nonzero(bad)[:4].tolist())


def case(seed, tokens, top_k, num, width, hidden, n, kind, dtype, gated, routing="mixed",
         down_kind=None):
    x = normal(seed, tokens, width, dtype=dtype)
    up, up_values = make(seed + 1, kind, num, hidden * (2 if gated else 1), width, dtype)
    down, down_values = make(seed + 3, down_kind or kind, num, n, hidden, dtype)
    ids = route(seed + 5, tokens, top_k, num, routing)
    by = normal(seed + 6, tokens, top_k).softmax(dim=1)
    return (x, up, down, ids, by), (x, up_values, down_values, ids, by)


# tokens, top_k, experts, width, hidden, columns of the result
SIZES = [(1, 1, 1, 16, 16, 1), (1, 8, 64, 128, 64, 128), (3, 2, 5, 17, 19, 11), (4, 2, 3, 33, 31, 70),
         (16, 4, 8, 256, 96, 200), (17, 2, 4, 130, 70, 90), (33, 3, 6, 512, 257, 300),
         (64, 8, 16, 264, 136, 520), (64, 2, 2, 100, 60, 40), (5, 2, 1024, 64, 32, 48),
         (64, 64, 64, 40, 24, 33), (2, 2, 3, 2050, 1337, 700), (1, 2, 4, 4096, 2048, 2048),
         (20, 2, 3, 2048, 520, 260)]


@pytest.mark.parametrize("size", SIZES, ids=["-".join(map(str, s)) for s in SIZES])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_layer(size, kind, dtype):
    for gated in (True, False):
        for routing in ("all", "mixed"):
            args, values = case(sum(size), *size, kind, dtype, gated, routing)
            check(experts.few_tokens(*args, gated=gated),
                  *layer(*values, gated, 2 if kind == "mx4" and dtype == torch.float16 else 1))


@pytest.mark.parametrize("kind", ["16", "mx4"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_narrowest_layers(kind, dtype):
    """16 bytes of a token's row and of h's are the least."""
    for width, hidden in ((8, 8), (9, 15), (15, 9)):
        args, values = case(12, 5, 2, 3, width, hidden, 7, kind, dtype, True)
        check(experts.few_tokens(*args), *layer(*values, True, 2))
    args, _ = case(12, 5, 2, 3, 7, 8, 7, kind, dtype, True)
    with pytest.raises(hist.HistError):
        experts.few_tokens(*args)
    args, _ = case(12, 5, 2, 3, 15, 16, 7, "int8", dtype, True)
    with pytest.raises(hist.HistError):
        experts.few_tokens(*args)


@pytest.mark.parametrize("up,down", [("16", "int8"), ("int8", "mx4"), ("mx4", "16")])
def test_weights_of_two_kinds(up, down):
    args, values = case(1, 9, 2, 6, 300, 200, 150, up, torch.float16, True, down_kind=down)
    check(experts.few_tokens(*args), *layer(*values, True, 2))


def sharing(tokens, top_k, num, hidden, n, kind):
    """The most workgroups that have a part of 16 columns (of 32, of up to 16 tokens in 4 bits) of the
    result, from the size of their sums in the workspace."""
    at = KINDS.index(kind)
    wide = 32 if kind == "mx4" and tokens <= 16 else 16
    tiles, step = -(-n // wide), 64 << at
    rest = experts._workspace("experts_few_tokens_workspace_size", tokens, top_k, num, hidden, n, at)
    for part in (tokens * top_k * 2 * -(-hidden // step) * step * 2, tiles * 4):
        rest -= -(-part // 256) * 256
    assert rest % (tiles * -(-tokens // 16) * wide * 64) == 0
    return tiles, rest // (tiles * -(-tokens // 16) * wide * 64)


@pytest.mark.parametrize("tokens,kind,dtype", [
    (t, k, d) for t in (1, 12, 40) for k in KINDS for d in DTYPES])
def test_h_keeps_what_the_type_does_not(tokens, kind, dtype):
    """(4-bit weights take h in bfloat16 whatever the tokens' type.)"""
    args, values = case(21, tokens, 2, 3, 64, 96, 40, kind, dtype, True)
    eps = torch.finfo(torch.bfloat16 if kind == "mx4" else dtype).eps
    check(experts.few_tokens(*args), *layer(*values, True, 2, (eps / 2)**2))


# 256 workgroups that divide the tiles evenly: the ends of their shares lie within tiles.
@pytest.mark.parametrize("kind,tokens,num,hidden,n,want", [
    ("16", 40, 16, 1337, 2064, (129, 3)),
    ("16", 9, 8, 2680, 2050, (129, 3)),
    ("16", 40, 8, 1344, 5120, (320, 2)),
    ("int8", 40, 16, 2677, 2064, (129, 3)),
    ("int8", 5, 8, 2688, 2050, (129, 3)),
    ("mx4", 40, 16, 2677, 5120, (320, 2)),
    ("mx4", 16, 16, 2688, 4112, (129, 3)),
    ("16", 3, 2, 64, 65552, (4097, 2)),
])
def test_equal_shares(kind, tokens, num, hidden, n, want):
    assert sharing(tokens, 2, num, hidden, n, kind) == want
    args, values = case(31, tokens, 2, num, 64, hidden, n, kind, torch.bfloat16, False, "all")
    # (h's two parts: twice the products)
    check(experts.few_tokens(*args, gated=False), *layer(*values, False, 2))


@pytest.mark.parametrize("routing", ["one", "none"])
@pytest.mark.parametrize("tokens", [1, 16, 64])
def test_one_expert_for_all_and_none_at_all(routing, tokens):
    """Every pair with one expert is also the same expert several times for a token."""
    args, values = case(2, tokens, 3, 5, 200, 120, 330, "16", torch.bfloat16, True, routing)
    out = experts.few_tokens(*args)
    check(out, *layer(*values, True, 1))
    assert out.any() == (routing == "one")


def test_ids_of_64_bits_and_extreme_ones():
    args, values = case(3, 6, 2, 8, 96, 64, 128, "16", torch.bfloat16, True, "all")
    x, up, down, ids, by = args
    wide = ids.long()
    assert torch.equal(experts.few_tokens(x, up, down, wide, by), experts.few_tokens(*args))
    wide[0, 0], wide[1, 1], wide[2, 0] = 2**32 + 1, -2**40, 2**63 - 1
    gone = ids.clone()
    gone[0, 0], gone[1, 1], gone[2, 0] = 2**31 - 1, -2**31, 8
    a = experts.few_tokens(x, up, down, wide, by)
    assert torch.equal(a, experts.few_tokens(x, up, down, gone, by))
    check(a, *layer(x, *values[1:3], gone, by, True, 1))


def shifted(t, by):
    longer = torch.full((*t.shape[:-2], t.shape[-2] + 1, t.shape[-1] + 2 * by + 3), 1,
                        device=t.device).to(t.dtype)
    view = longer[..., :t.shape[-2], by:by + t.shape[-1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("by", [1, 5])
def test_views(kind, by):
    """Rows and experts with gaps between them, off 16 bytes: the same bits."""
    args, _ = case(4, 7, 2, 5, 200, 130, 90, kind, torch.bfloat16, True)
    x, up, down, ids, weights = args

    def moved(w):
        if isinstance(w, torch.Tensor):
            return shifted(w, by)
        return shifted(w[0], by), (shifted(w[1], by) if kind == "mx4" else w[1])

    got = experts.few_tokens(shifted(x, by), moved(up), moved(down), ids, weights)
    assert torch.equal(got, experts.few_tokens(*args))


@pytest.mark.parametrize("kind", ["16", "mx4"])
def test_an_expert_with_infinities_keeps_them(kind):
    """Its tokens only; an expert without a token is not even looked at."""
    args, values = case(5, 20, 2, 6, 160, 96, 64, kind, torch.bfloat16, True, "all")
    x, up, down, ids, by = args
    clean = experts.few_tokens(*args)
    for w in (up, down):
        if kind == "16":
            w[2] = float("inf")
        else:
            w[1][2] = 255
    out = experts.few_tokens(*args)
    has = (ids == 2).any(1)
    assert has.any() and not has.all()
    assert torch.equal(out[~has], clean[~has])
    assert not torch.isfinite(out[has]).any()
    without = torch.where(ids == 2, (ids + 1) % 6, ids)
    assert torch.isfinite(experts.few_tokens(x, up, down, without, by)).all()


@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("dtype", DTYPES)
def test_an_infinite_weight_of_the_second_product_keeps_its_sign(dtype, tokens):
    """Whatever the type leaves of h, and of whichever sign that is."""
    x = normal(11, tokens, 64, dtype=dtype)
    up, down = (normal(s, 2, 64, 64, dtype=dtype, scale=0.125) for s in (12, 13))
    down[1, 5, 7] = float("inf")
    ids = torch.ones(tokens, 1, dtype=torch.int32, device="cuda")
    out = experts.few_tokens(x, up, down, ids, torch.ones(tokens, 1, device="cuda"), gated=False)
    a = x.double() @ up[1].double().t().contiguous()
    h = a[:, 7] * torch.sigmoid(a[:, 7])
    assert (h.abs() > 1e-3).all()  # (signs that rounding cannot change)
    assert torch.equal(out[:, 5].double(), torch.sign(h) * float("inf"))
    assert torch.isfinite(out[:, [c for c in range(64) if c != 5]]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_column_that_the_type_rounds_to_infinity_is_one(dtype):
    """h is finite in 32 bits and past the type's last value: what is left of it adds no NaN."""
    width = hidden = 16
    x = torch.zeros(3, width, dtype=dtype, device="cuda")
    up = torch.zeros(1, hidden, width, dtype=dtype, device="cuda")
    if dtype == torch.float16:
        x[1, 0] = up[0, 0, 0] = 300.0  # 90,000 > 65,520
    else:
        # 2^127 (255 / 128 + 1.5 / 256): past 2^127 (2 - 1 / 256), below 2^128
        x[1, 0], up[0, 0, 0] = 2.0**64 * 255 / 128, 2.0**63
        x[1, 1], up[0, 0, 1] = 2.0**55 * 1.5, 2.0**64
    down = torch.ones(1, 8, hidden, dtype=dtype, device="cuda")
    ids = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    out = experts.few_tokens(x, up, down, ids, torch.ones(3, 1, device="cuda"), gated=False)
    assert torch.isposinf(out[1]).all() and (out[0] == 0).all() and (out[2] == 0).all()


def test_infinities_and_nan_of_a_token_stay_in_its_row():
    for kind in KINDS:
        for dtype in DTYPES:
            args, _ = case(6, 20, 2, 6, 160, 96, 64, kind, dtype, True, "all")
            x = args[0]
            clean = experts.few_tokens(*args)
            x[3, 7], x[11, 0] = float("nan"), float("inf")
            out = experts.few_tokens(*args)
            fine = [t for t in range(20) if t not in (3, 11)]
            assert torch.equal(out[fine], clean[fine])
            assert torch.isnan(out[3]).all() and not torch.isfinite(out[11]).any()


def test_small_weights_of_a_block_and_a_token():
    """4-bit powers far below float16's range count in full for float16 tokens."""
    args, values = case(7, 3, 1, 2, 64, 64, 64, "mx4", torch.float16, False, "all")
    x, (uq, us), (dq, ds), ids, by = args
    us -= 30
    ds += 30
    up, down = values[1] * 2.0**-30, values[2] * 2.0**30
    want, room = layer(x, up, down, ids, by, False, 2)
    # (h itself is then near 2^-30, below float16's least value 2^-24: rounded to 0 or near it)
    check(experts.few_tokens(x, (uq, us), (dq, ds), ids, by, gated=False), want, room)


def test_no_tokens():
    args, _ = case(8, 2, 2, 4, 64, 32, 48, "16", torch.bfloat16, True)
    x, up, down, ids, by = args
    assert experts.few_tokens(x[:0], up, down, ids[:0], by[:0]).shape == (0, 48)


def test_refused():
    args, _ = case(9, 4, 2, 4, 64, 32, 48, "16", torch.bfloat16, True)
    x, up, down, ids, by = args
    many = torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(4, 64, 64, dtype=torch.int8, device="cuda"), torch.ones(4, 64, device="cuda")
    for change in ({0: x.half()}, {0: x.cpu()}, {0: x[:, :32]}, {1: up[:3]}, {1: up[:, :63]},
                   {2: down.half()}, {2: down[:, :, :16]}, {3: ids.float()}, {3: ids[:3]},
                   {3: ids.cpu()}, {4: by.half()}, {4: by[:, :1]}, {1: (q, s[:3])}, {1: (q, s.half())},
                   {1: (q.view(torch.uint8), s)}, {1: (q[:, :, :32], s)},
                   {0: many, 3: ids.new_zeros(65, 2), 4: by.new_zeros(65, 2)}):
        bad = list(args)
        for at, value in change.items():
            bad[at] = value
        with pytest.raises(ValueError):
            experts.few_tokens(*bad)


@pytest.mark.parametrize("other", [None, 3, (), (None,), (None, None)])
def test_weights_that_are_none(other):
    x, up, down, ids, by = case(1, 2, 2, 3, 32, 32, 32, "int8", torch.bfloat16, False)[0]
    for args in ((x, other, down, ids, by), (x, up, other, ids, by)):
        with pytest.raises(ValueError):
            experts.few_tokens(*args, gated=False)
    with pytest.raises(ValueError):
        experts.few_tokens(x, (up[0], other), down, ids, by, gated=False)


def test_captured_twice_and_on_another_stream():
    """Two graphs of one layer, replayed in turn, with eager calls on another stream between: every
    result the same bits."""
    args, _ = case(10, 12, 4, 16, 1024, 512, 1000, "16", torch.bfloat16, True, "all")
    want = experts.few_tokens(*args)
    torch.cuda.synchronize()
    captured = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = experts.few_tokens(*args)
        captured.append((graph, out))
    stream = torch.cuda.Stream()
    for _ in range(4):
        for graph, out in captured:
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            again = [experts.few_tokens(*args) for _ in range(3)]
        here = experts.few_tokens(*args)
        stream.synchronize()
        assert all(torch.equal(t, want) for t in again + [here])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_decode_step_of_all_of_them(dtype):
    """Norm, then the layer by both roads: for a few tokens at once, and grouped with 4-bit products;
    and the 8-bit norm into the 8-bit product."""
    tokens, num, width, hidden = 24, 8, 192, 160
    args, values = case(11, tokens, 2, num, width, hidden, width, "mx4", dtype, False, "all")
    x, up, down, ids, by = args
    weight = (1 + 0.1 * normal(20, width)).to(dtype)
    residual = normal(21, tokens, width, dtype=dtype)
    y, h = experts.rms_norm(x, weight, residual)
    out = experts.few_tokens(y, up, down, ids, by, gated=False)
    check(out, *layer(y, *values[1:], False, 2))
    # the same with tokens quantised to 4 bits too: 24 rows through the grouped products
    g = experts.group_rows(ids, num)
    a = experts.mx4_matmul(*experts.quantize_mx4(y), *up, g, gather=True, out_dtype=dtype)
    s = torch.nn.functional.silu(a)
    grouped = experts.combine(experts.mx4_matmul(*experts.quantize_mx4(s), *down, g, out_dtype=dtype),
                              g, by)
    # (4-bit activations: a value is off by at most a quarter of itself, or a twelfth of the block's largest
    # one; the two layers' results differ by less than their own size)
    assert float((grouped - out).float().norm() / out.float().norm()) < 0.5
    xq, sx, again = experts.rms_norm_int8(x, weight, residual)
    assert torch.equal(again, h)
    wq = normal(22, 100, width, scale=40).round().clamp(-127, 127).to(torch.int8)
    product = experts.int8_matmul(xq, sx, wq, torch.ones(100, device="cuda"), out_dtype=dtype)
    want = (xq.double() * sx.double().view(-1, 1)) @ wq.double().t().contiguous()
    info = torch.finfo(dtype)
    assert ((product.double() - want).abs() <= want.abs() * (info.eps / 2 + 4 * 2.0**-24) +
            info.smallest_normal).all()


def test_the_example_serves_by_every_road():
    """Few tokens at once and a batch, in 8 and in 4 bits: by the size of a value's step (half of 1/127
    of its row's largest one, about 4 of its standard deviations, in 8 bits: 1% of the norm; in 4
    bits, with steps of a sixth at the least, some 12%), for one operand or two, twice."""
    from test_experts_example_gpu import example
    got = example().main(steps=2)
    assert got["error"] < 0.05 and got["batch"] < 0.05
    assert got["mx4"] < 0.3 and got["mx4_batch"] < 0.4
