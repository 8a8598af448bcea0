"""Cases of the operators around products over experts: routing, 8-bit quantisation, the block-scaled 8-bit product
(dense and over experts), and the weighted sum of the experts' outputs.

``run`` computes them in plain torch operations, or, where ``own`` is true, through the library's entry points.
Layouts: an 8-bit operand of a product is rows x K with K contiguous (rows padded to 16 bytes); its scales are
[K block][row], or for weights [row block][K block]; a block is 128 long.
"""

import math

import torch

own = False

BLOCK = 128
TOP = 448.0                # largest e4m3 value
LEAST = 2.0 ** -96         # a block's largest value counts as at least this
FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # Routing of a decode batch: a few tokens, sigmoid scores, a balance bias, groups ranked by their two best.
        dict(name="route_decode", op="route", T=8, E=64, k=6, score="sigmoid", bias=True, groups=8, kept=4, two=True,
             renorm=True, scale=2.5, dtype="f32", backward=False),
        # Routing of a training batch, with its gradient: softmax over 128 experts, an odd number of tokens.
        dict(name="route_train", op="route", T=16383, E=128, k=8, score="softmax", bias=False, groups=1, kept=1,
             two=False, renorm=True, scale=1.0, dtype="f32", backward=True),
        # The rows of a decode batch, gathered for their experts and quantised for the product.
        dict(name="quantize_decode", op="quantize", form="rows", rows=96, cols=2048, src=16, dtype="bf16", groups=1),
        # An output gradient of a training step: quantised along its rows for the input gradient and along the
        # tokens of each expert for the weight gradient; odd counts.
        dict(name="quantize_train", op="quantize", form="rows+cols", rows=16383, cols=4096, src=0, dtype="bf16", groups=16),
        # One decode step of a linear layer: 16 tokens.
        dict(name="product_decode", op="product", M=16, N=4096, K=4096, form="blocks", out="bf16"),
        # The odd rectangle, both operands scaled per row: the weight gradient of a dense layer, kept in 32 bits.
        dict(name="product_odd", op="product", M=4097, N=3001, K=2049, form="rows", out="f32"),
        # A long batch of prompts through a square layer.
        dict(name="product_prompts", op="product", M=16384, N=4096, K=4096, form="blocks", out="bf16"),
        # A decode step's rows over the experts they went to.
        dict(name="experts_decode", op="experts", mode="rows", E=64, active=48, rows=96, N=2048, K=2048, out="bf16"),
        # A prompt batch over the experts; ragged counts, some experts empty.
        dict(name="experts_prompts", op="experts", mode="rows", E=64, active=60, rows=16384, N=2048, K=2048, out="bf16"),
        # The weight gradients of the experts of a training step, in 32 bits.
        dict(name="experts_weight_gradient", op="experts", mode="weights", E=16, active=15, rows=16383, N=2048, K=2048, out="f32"),
        # The experts' outputs of a decode batch summed per token.
        dict(name="combine_decode", op="combine", T=16, k=6, cols=2048, dtype="bf16", weights=True, backward=False),
        # The same of a training step, with the gradients of the outputs and of the weights.
        dict(name="combine_train", op="combine", T=8191, k=6, cols=2048, dtype="bf16", weights=True, backward=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "product", "experts", "experts", "combine"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([4, 8, 16, 20, 32]) if groups > 1 else rng.choice([8, 16, 60, 64, 128, 160, 256])
        # A bias is drawn with sigmoid scores and groups of softmax scores rank by their best: there the order of
        # the softmax's sum cannot decide which of two nearly equal keys is larger.
        score = rng.choice(["softmax", "sigmoid"])
        kept = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E // groups * kept)), score=score,
                    bias=score == "sigmoid" and rng.random() < 0.7, groups=groups, kept=kept,
                    two=groups > 1 and score == "sigmoid" and rng.random() < 0.5, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=dtype, backward=rng.random() < 0.5)
    if op == "quantize":
        form = rng.choice(["rows", "rows+cols", "blocks"])
        rows, cols = _log(rng, 1, 16384), _log(rng, 16, 4096)
        groups = rng.choice([1, 1, 8, 60]) if form == "rows+cols" else 1
        src = _log(rng, 1, rows) if form == "rows" and rng.random() < 0.5 else 0
        return dict(op=op, form=form, rows=rows, cols=cols, src=src, dtype=dtype, groups=groups)
    if op == "product":
        M, N, K = _log(rng, 1, 16384), _log(rng, 16, 4096), _log(rng, 16, 4096)
        return dict(op=op, M=M, N=N, K=K, form=rng.choice(["blocks", "blocks", "rows"]), out=dtype)
    if op == "experts":
        mode = rng.choice(["rows", "rows", "weights"])
        E = rng.choice([4, 8, 16, 32, 64])
        rows = _log(rng, 1, 16384)
        active = rng.randint(1, min(E, rows))
        return dict(op=op, mode=mode, E=E, active=active, rows=rows, N=_log(rng, 64, 2048), K=_log(rng, 64, 2048), out=dtype)
    return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 8), cols=_log(rng, 16, 2048), dtype=dtype,
                weights=rng.random() < 0.8, backward=rng.random() < 0.5)


def _up(x, m):
    return (x + m - 1) // m * m


# ---------------------------------------------------------------- plain forms


def _blocks_of_columns(x):
    """x (rows x cols) in 32 bits as rows x blocks x 128, filled with zeros."""
    rows, cols = x.shape
    full = x.new_zeros(rows, _up(cols, BLOCK))
    full[:, :cols] = x
    return full.view(rows, -1, BLOCK)


def _rounded(x, most):
    """x in 8 bits, where `most` is its block's largest magnitude, and the block's scale."""
    most = most.clamp(min=LEAST)
    return (x * (TOP / most)).clamp(-TOP, TOP).to(FP8), most / TOP


def _plain_rows(x):
    b = _blocks_of_columns(x)
    q, s = _rounded(b, b.abs().amax(2, keepdim=True))
    return q.view(x.shape[0], -1)[:, :x.shape[1]], s[:, :, 0].t().contiguous()


def _padded_places(offsets, rows):
    """Of each row, its place when every group starts on a multiple of 128."""
    counts = offsets[1:] - offsets[:-1]
    padded = (counts + BLOCK - 1) // BLOCK * BLOCK
    start = torch.cumsum(padded, 0) - padded
    at = torch.arange(rows, device=offsets.device)
    g = torch.searchsorted(offsets[1:].contiguous(), at, right=True)
    return at - offsets[g] + start[g]


def _plain_cols(x, offsets, padded):
    """Transposed, each group's rows from a multiple of 128 on, zeros between: cols x padded, scales [block][col]."""
    full = x.new_zeros(padded, x.shape[1])
    full[_padded_places(offsets.long(), x.shape[0])] = x
    b = full.view(-1, BLOCK, x.shape[1])
    q, s = _rounded(b, b.abs().amax(1, keepdim=True))
    return q.view(padded, -1).t().contiguous(), s[:, 0, :].contiguous()


def _plain_blocks(x):
    """128 x 128 blocks: q rows x cols, scales [row block][column block]."""
    rows, cols = x.shape
    full = x.new_zeros(_up(rows, BLOCK), _up(cols, BLOCK))
    full[:rows, :cols] = x
    b = full.view(full.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    q, s = _rounded(b, b.abs().amax((1, 3), keepdim=True))
    return q.view(full.shape)[:rows, :cols], s[:, 0, :, 0].contiguous()


def _wide_rows(q, s, dtype=torch.float32):
    """The values that q (rows x K) with scales [K block][row] stands for."""
    return q.to(dtype) * s.to(dtype).t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _wide_blocks(q, s, dtype=torch.float32):
    """The same with scales [..., row block, K block]."""
    wide = s.to(dtype).repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]
    return q.to(dtype) * wide.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]


def _plain_scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    l = s["logits"].float()
    T, E = l.shape
    p = _plain_scores(l, s["score"])
    key = p + s["bias"] if s["bias"] is not None else p if s["two"] else l
    if s["kept"] < s["groups"]:
        g = key.view(T, s["groups"], -1).sort(dim=2, descending=True, stable=True)[0]
        rank = g[:, :, 0] + g[:, :, 1] if s["two"] else g[:, :, 0]
        keep = torch.zeros_like(rank, dtype=torch.bool)
        keep.scatter_(1, rank.sort(dim=1, descending=True, stable=True)[1][:, :s["kept"]], True)
        key = torch.where(keep.repeat_interleave(E // s["groups"], 1), key, -math.inf)
    indices = key.sort(dim=1, descending=True, stable=True)[1][:, :s["k"]]
    w = p.gather(1, indices)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return w * s["scale"], indices.to(torch.int32)


def _plain_route_backward(s, indices):
    l, g, c = s["logits"].float(), s["grad_w"], s["scale"]
    p = _plain_scores(l, s["score"])
    at = indices.long()
    chosen = p.gather(1, at)
    d = torch.zeros_like(p)
    if s["score"] == "softmax":
        if s["renorm"]:
            w = chosen / chosen.sum(1, keepdim=True)
            d.scatter_(1, at, c * w * (g - (w * g).sum(1, keepdim=True)))
        else:
            d.scatter_(1, at, g)
            d = c * p * (d - (chosen * g).sum(1, keepdim=True))
    else:
        slope = chosen * (1.0 / (1.0 + torch.exp(l.gather(1, at))))
        if s["renorm"]:
            D = chosen.sum(1, keepdim=True)
            d.scatter_(1, at, c / D * (g - (g * chosen).sum(1, keepdim=True) / D) * slope)
        else:
            d.scatter_(1, at, c * g * slope)
    return d.to(s["logits"].dtype)


def _plain_dispatch(indices, E):
    flat = indices.reshape(-1).long()
    order = torch.sort(flat, stable=True)[1]
    counts = torch.zeros(E, dtype=torch.long, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(E + 1, dtype=torch.long, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    row_of = torch.empty_like(flat).scatter_(0, order, torch.arange(flat.numel(), device=flat.device))
    return (offsets.to(torch.int32), row_of.view(indices.shape).to(torch.int32),
            (order // indices.shape[1]).to(torch.int32))


def _padded_groups(s, places_start):
    """(E x cap places of the groups' members, which of them are some)."""
    counts = s["offsets"][1:].long() - s["offsets"][:-1].long()
    at = torch.arange(s["cap"], device=counts.device)
    there = at[None, :] < counts[:, None]
    return torch.where(there, places_start[:, None] + at[None, :], 0), there


def _plain_experts_rows(s):
    at, there = _padded_groups(s, s["offsets"][:-1].long())
    x = _wide_rows(s["A"], s["sa"])[at] * there[:, :, None]
    y = torch.bmm(x, _wide_blocks(s["B"], s["sb"]).transpose(1, 2))
    return y[there].to(s["out"])


def _plain_experts_weights(s):
    counts = s["offsets"][1:].long() - s["offsets"][:-1].long()
    padded = (counts + BLOCK - 1) // BLOCK * BLOCK
    at, there = _padded_groups(s, torch.cumsum(padded, 0) - padded)
    a = _wide_rows(s["A"], s["sa"])[:, at] * there
    b = _wide_rows(s["B"], s["sb"])[:, at] * there
    return torch.bmm(a.transpose(0, 1), b.permute(1, 2, 0)).to(s["out"])


def _plain_combine(s):
    picked = s["Y"][s["row_of"].long()].float()
    w = s["weights"][:, :, None] if s["weights"] is not None else 1.0
    got = dict(out=(picked * w).sum(1).to(s["Y"].dtype))
    if s["backward"]:
        g = s["grad_out"].float()[:, None, :]
        at = s["row_of"].long().reshape(-1)
        spread = (g * w).expand_as(picked).reshape(-1, picked.shape[2])
        got["grad_y"] = torch.zeros_like(s["Y"]).index_copy_(0, at, spread.to(s["Y"].dtype))
        if s["weights"] is not None:
            got["grad_w"] = (g * picked).sum(2)
    return got


def _run_plain(s):
    if s["op"] == "route":
        w, indices = _plain_route(s)
        offsets, row_of, token_of = _plain_dispatch(indices, s["logits"].shape[1])
        got = dict(weights=w, indices=indices, offsets=offsets, row_of=row_of, token_of=token_of)
        if s["backward"]:
            got["grad_logits"] = _plain_route_backward(s, indices)
        return got
    if s["op"] == "quantize":
        x = s["x"].float()
        if s["gather"] is not None:
            x = x[s["gather"].long()]
        if s["form"] == "blocks":
            (q, c), (qt, ct) = _plain_blocks(x), _plain_blocks(x.t())
            return dict(q=q, scales=c, q_t=qt, scales_t=ct)
        q, c = _plain_rows(x)
        got = dict(q=q, scales=c)
        if s["form"] == "rows+cols":
            got["q_t"], got["scales_t"] = _plain_cols(x, s["offsets"], s["padded"])
        return got
    if s["op"] == "product":
        b = _wide_rows(s["B"], s["sb"]) if s["form"] == "rows" else _wide_blocks(s["B"], s["sb"])
        return (_wide_rows(s["A"], s["sa"]) @ b.t()).to(s["out"])
    if s["op"] == "experts":
        return _plain_experts_rows(s) if s["mode"] == "rows" else _plain_experts_weights(s)
    return _plain_combine(s)


# ------------------------------------------------------- the library's calls


def _ok(sg, code):
    if code != sg.SGEMM_OK:
        raise sg.SgemmError(code, "perf")


def _type(sg, dtype):
    return sg.SGEMM_F32 if dtype == torch.float32 else sg.SGEMM_BF16


def _new(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _own_route(sg, s, st):
    l = s["logits"]
    (T, E), k = l.shape, s["k"]
    score = sg.SGEMM_SCORE_SOFTMAX if s["score"] == "softmax" else sg.SGEMM_SCORE_SIGMOID
    w, indices = _new((T, k), torch.float32), _new((T, k), torch.int32)
    _ok(sg, sg.sgemm_route(T, E, l.data_ptr(), _type(sg, l.dtype), l.stride(0), _ptr(s["bias"]), score, s["groups"],
                           s["kept"], int(s["two"]), k, int(s["renorm"]), s["scale"], w.data_ptr(), indices.data_ptr(), st))
    offsets, row_of, token_of = _new(E + 1, torch.int32), _new((T, k), torch.int32), _new(T * k, torch.int32)
    _ok(sg, sg.sgemm_dispatch(T, k, E, indices.data_ptr(), offsets.data_ptr(), row_of.data_ptr(), token_of.data_ptr(), st))
    got = dict(weights=w, indices=indices, offsets=offsets, row_of=row_of, token_of=token_of)
    if s["backward"]:
        d = torch.empty_like(l)
        _ok(sg, sg.sgemm_route_backward(T, E, l.data_ptr(), _type(sg, l.dtype), l.stride(0), score, k, int(s["renorm"]),
                                        s["scale"], indices.data_ptr(), s["grad_w"].data_ptr(), d.data_ptr(), E, st))
        got["grad_logits"] = d
    return got


def _own_quantize(sg, s, st):
    x, gather = s["x"], s["gather"]
    cols, kind = x.shape[1], _type(sg, x.dtype)
    rows = x.shape[0] if gather is None else gather.numel()
    ld = _up(cols, 16)
    q = _new((rows, ld), FP8)
    if s["form"] == "blocks":
        nr, nc, ldt = _up(rows, BLOCK) // BLOCK, _up(cols, BLOCK) // BLOCK, _up(rows, 16)
        c, qt, ct = _new((nr, nc), torch.float32), _new((cols, ldt), FP8), _new((nc, nr), torch.float32)
        _ok(sg, sg.sgemm_fp8_quantize_blocks(rows, cols, x.data_ptr(), kind, x.stride(0), 0, 0, q.data_ptr(), ld, 0,
                                             c.data_ptr(), nc, 0, 1, st))
        _ok(sg, sg.sgemm_fp8_quantize_blocks(rows, cols, x.data_ptr(), kind, x.stride(0), 0, 1, qt.data_ptr(), ldt, 0,
                                             ct.data_ptr(), nr, 0, 1, st))
        return dict(q=q[:, :cols], scales=c, q_t=qt[:, :rows], scales_t=ct)
    c = _new((_up(cols, BLOCK) // BLOCK, rows), torch.float32)
    if s["form"] == "rows":
        _ok(sg, sg.sgemm_fp8_quantize_rows(rows, cols, x.data_ptr(), kind, x.stride(0), _ptr(gather), x.shape[0],
                                           q.data_ptr(), ld, c.data_ptr(), rows, st))
        return dict(q=q[:, :cols], scales=c)
    padded = s["padded"]
    qt, ct = _new((cols, padded), FP8), _new((padded // BLOCK, cols), torch.float32)
    _ok(sg, sg.sgemm_fp8_quantize_both(rows, cols, x.data_ptr(), kind, x.stride(0), _ptr(gather), x.shape[0],
                                       s["offsets"].numel() - 1, s["offsets"].data_ptr(), padded, q.data_ptr(), ld,
                                       c.data_ptr(), rows, qt.data_ptr(), padded, ct.data_ptr(), cols, st))
    return dict(q=q[:, :cols], scales=c, q_t=qt, scales_t=ct)


def _own_product(sg, s, st):
    A, B, sa, sb = s["A"], s["B"], s["sa"], s["sb"]
    (M, K), N = A.shape, B.shape[0]
    C = _new((M, N), s["out"])
    form = sg.SGEMM_SCALE_ROWS if s["form"] == "rows" else sg.SGEMM_SCALE_BLOCKS
    _ok(sg, sg.sgemm_fp8(form, M, N, K, A.data_ptr(), A.stride(0), sa.data_ptr(), sa.stride(0), B.data_ptr(),
                         B.stride(0), sb.data_ptr(), sb.stride(0), 0.0, C.data_ptr(), _type(sg, C.dtype), N, st))
    return C


def _own_experts(sg, s, st):
    A, B, sa, sb, offsets = s["A"], s["B"], s["sa"], s["sb"], s["offsets"]
    E = offsets.numel() - 1
    if s["mode"] == "rows":
        (R, K), N = A.shape, B.shape[1]
        C = _new((R, N), s["out"])
        _ok(sg, sg.sgemm_fp8_grouped(E, offsets.data_ptr(), R, N, K, A.data_ptr(), A.stride(0), sa.data_ptr(),
                                     sa.stride(0), B.data_ptr(), B.stride(1), B.stride(0), sb.data_ptr(), sb.stride(1),
                                     sb.stride(0), 0.0, C.data_ptr(), _type(sg, C.dtype), N, st))
        return C
    M, N = A.shape[0], B.shape[0]
    C = _new((E, M, N), s["out"])
    _ok(sg, sg.sgemm_fp8_grouped_k(E, offsets.data_ptr(), s["padded"], M, N, A.data_ptr(), A.stride(0), sa.data_ptr(),
                                   sa.stride(0), B.data_ptr(), B.stride(0), sb.data_ptr(), sb.stride(0), 0.0,
                                   C.data_ptr(), _type(sg, C.dtype), N, M * N, st))
    return C


def _own_combine(sg, s, st):
    Y, row_of, w = s["Y"], s["row_of"], s["weights"]
    (T, k), (R, cols), kind = row_of.shape, Y.shape, _type(sg, Y.dtype)
    out = _new((T, cols), Y.dtype)
    _ok(sg, sg.sgemm_combine(T, k, cols, R, Y.data_ptr(), kind, cols, row_of.data_ptr(), _ptr(w), out.data_ptr(), cols, st))
    got = dict(out=out)
    if s["backward"]:
        gy = torch.empty_like(Y)
        gw = torch.empty_like(w) if w is not None else None
        _ok(sg, sg.sgemm_combine_backward(T, k, cols, R, s["grad_out"].data_ptr(), kind, cols, Y.data_ptr(), cols,
                                          row_of.data_ptr(), _ptr(w), gy.data_ptr(), cols, _ptr(gw), st))
        got["grad_y"] = gy
        if gw is not None:
            got["grad_w"] = gw
    return got


def run(state):
    if not own:
        return _run_plain(state)
    import dense_fp32_matrix_07_gb300 as sg
    stream = torch.cuda.current_stream().cuda_stream
    return {"route": _own_route, "quantize": _own_quantize, "product": _own_product, "experts": _own_experts,
            "combine": _own_combine}[state["op"]](sg, state, stream)


# --------------------------------------------------------------------- inputs


def _strided(q):
    """q with rows that begin on 16 bytes, as the quantiser lays them out."""
    full = torch.zeros((q.shape[0], _up(q.shape[1], 16)), dtype=FP8, device=q.device)
    full[:, :q.shape[1]] = q
    return full[:, :q.shape[1]]


def _activations(gen, rows, cols):
    """Normal values with a few channels that are much larger, as activations have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return x * torch.exp(torch.randn(cols, generator=gen, device="cuda"))


def _room(rows, groups):
    """A length that holds `rows` rows in `groups` groups, each from a multiple of 128 on, whatever the counts."""
    return _up(rows + (BLOCK - 1) * min(rows, groups), BLOCK)


def _offsets(gen, groups, active, rows):
    """Uneven counts: `active` of the groups have at least one row each, the others none. (device offsets, counts)"""
    p = torch.zeros(groups, device="cuda")
    some = torch.randperm(groups, generator=gen, device="cuda")[:active]
    p[some] = torch.exp(0.5 * torch.randn(active, generator=gen, device="cuda"))
    counts = torch.zeros(groups, dtype=torch.long, device="cuda")
    counts[some] = 1
    if rows > active:
        more = torch.multinomial(p, rows - active, replacement=True, generator=gen)
        counts += torch.zeros_like(counts).scatter_add_(0, more, torch.ones_like(more))
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, counts.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if c["op"] == "route":
        logits = (2.0 * normal(c["T"], c["E"])).to(TYPES[c["dtype"]])
        bias = 0.05 * normal(c["E"]) if c["bias"] else None
        return dict(c, logits=logits, bias=bias, grad_w=normal(c["T"], c["k"]) if c["backward"] else None)
    if c["op"] == "quantize":
        n = c["src"] or c["rows"]
        x = _activations(gen, n, c["cols"]).to(TYPES[c["dtype"]])
        gather = torch.randint(0, n, (c["rows"],), generator=gen, device="cuda", dtype=torch.int32) if c["src"] else None
        offsets, _ = _offsets(gen, c["groups"], min(c["rows"], max(1, c["groups"] - c["groups"] // 8)), c["rows"])
        return dict(op="quantize", form=c["form"], x=x, gather=gather, offsets=offsets,
                    padded=_room(c["rows"], c["groups"]))
    if c["op"] == "product":
        A, sa = _plain_rows(_activations(gen, c["M"], c["K"]))
        w = normal(c["N"], c["K"]) / math.sqrt(c["K"])
        B, sb = _plain_rows(w) if c["form"] == "rows" else _plain_blocks(w)
        return dict(op="product", form=c["form"], A=_strided(A), sa=sa, B=_strided(B), sb=sb, out=TYPES[c["out"]])
    if c["op"] == "experts":
        offsets, counts = _offsets(gen, c["E"], c["active"], c["rows"])
        s = dict(op="experts", mode=c["mode"], offsets=offsets, cap=max(counts), out=TYPES[c["out"]])
        if c["mode"] == "rows":
            A, sa = _plain_rows(_activations(gen, c["rows"], c["K"]))
            ld = _up(c["K"], 16)
            B = torch.zeros((c["E"], c["N"], ld), dtype=FP8, device="cuda")[:, :, :c["K"]]
            sb = torch.empty((c["E"], _up(c["N"], BLOCK) // BLOCK, _up(c["K"], BLOCK) // BLOCK), device="cuda")
            for e in range(c["E"]):
                q, sb[e] = _plain_blocks(normal(c["N"], c["K"]) / math.sqrt(c["K"]))
                B[e] = q
            return dict(s, A=_strided(A), sa=sa, B=B, sb=sb)
        padded = _room(c["rows"], c["E"])
        A, sa = _plain_cols(1e-3 * normal(c["rows"], c["N"]), offsets, padded)
        B, sb = _plain_cols(_activations(gen, c["rows"], c["K"]), offsets, padded)
        return dict(s, padded=padded, A=A, sa=sa, B=B, sb=sb)
    T, k, cols = c["T"], c["k"], c["cols"]
    dtype = TYPES[c["dtype"]]
    row_of = torch.randperm(T * k, generator=gen, device="cuda").view(T, k).to(torch.int32)
    weights = torch.rand(T, k, generator=gen, device="cuda") if c["weights"] else None
    return dict(op="combine", Y=normal(T * k, cols).to(dtype), row_of=row_of, weights=weights, backward=c["backward"],
                grad_out=normal(T, cols).to(dtype) if c["backward"] else None)


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k, size = c["T"], c["E"], c["k"], SIZE[c["dtype"]]
        # logits; weights, indices, both orders; the gradient of the weights and of the logits
        b = T * E * size + T * k * 16 + 4 * (E + 1) + (T * k * 4 + T * E * size if c["backward"] else 0)
        return dict(bytes=b, flops=T * E * (10 if c["backward"] else 5))
    if c["op"] == "quantize":
        n, size = c["rows"] * c["cols"], SIZE[c["dtype"]]
        b = min(n, (c["src"] or c["rows"]) * c["cols"]) * size
        b += (1 if c["form"] == "rows" else 2) * n * (1 + 4 / (BLOCK if "rows" in c["form"] else BLOCK ** 2))
        return dict(bytes=b, flops=4 * n)
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(bytes=(M + N) * K + M * N * SIZE[c["out"]], flops=2 * M * N * K)
    if c["op"] == "experts":
        R, N, K = c["rows"], c["N"], c["K"]
        if c["mode"] == "rows":
            return dict(bytes=c["active"] * N * K + R * K + R * N * SIZE[c["out"]], flops=2 * R * N * K)
        return dict(bytes=R * (N + K) + c["E"] * N * K * SIZE[c["out"]], flops=2 * R * N * K)
    n, size = c["T"] * c["cols"], SIZE[c["dtype"]]
    b = n * (c["k"] + 1) * size + c["T"] * c["k"] * 8
    if c["backward"]:
        b += n * (c["k"] + 1) * size + c["T"] * c["k"] * 4
    return dict(bytes=b, flops=2 * n * c["k"] * (3 if c["backward"] else 1))


# ------------------------------------------------------------- 64-bit results


def _exact_route(s):
    l = s["logits"].double()
    _, indices = _plain_route(s)   # which experts: given by the keys in 32 bits; their weights by 64
    at = indices.long()
    l.requires_grad_(True)
    with torch.enable_grad():
        q = torch.special.expit(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
        w = q.gather(1, at)
        w = s["scale"] * (w / w.sum(1, keepdim=True) if s["renorm"] else w)
        got = dict(weights=w.detach(), indices=None, offsets=None, row_of=None, token_of=None)
        if s["backward"]:
            got["grad_logits"] = torch.autograd.grad(w, l, s["grad_w"].double())[0]
    return got


def _exact_scales(x, starts, ends):
    """Of each [start, end) of x's rows the largest magnitudes / 448, per column."""
    return torch.stack([x[a:b].abs().amax(0) if b > a else torch.zeros_like(x[0]) for a, b in zip(starts, ends)]) / TOP


def exact(case, seed):
    """The definition in 64 bits. What is held in 8 bits has no value that is not rounded: None there."""
    if case["op"] == "product" and case["M"] * case["N"] * case["K"] > 3e11:
        return None
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "quantize":
        x = s["x"].double()
        if s["gather"] is not None:
            x = x[s["gather"].long()]
        at = range(0, x.shape[1], BLOCK)
        rows = torch.stack([x[:, a:a + BLOCK].abs().amax(1) for a in at]).clamp(min=LEAST) / TOP
        if s["form"] == "blocks":
            both = torch.stack([rows[:, a:a + BLOCK].amax(1) for a in range(0, x.shape[0], BLOCK)])
            return dict(q=None, scales=both, q_t=None, scales_t=both.t().contiguous())
        got = dict(q=None, scales=rows)
        if s["form"] == "rows+cols":
            o = s["offsets"].tolist()
            starts = [a for lo, hi in zip(o, o[1:]) for a in range(lo, hi, BLOCK)]
            ends = [min(a + BLOCK, hi) for lo, hi in zip(o, o[1:]) for a in range(lo, hi, BLOCK)]
            rest = s["padded"] // BLOCK - len(starts)   # blocks after the last group's hold zeros
            scales = _exact_scales(x, starts + [0] * rest, ends + [0] * rest)
            got["q_t"], got["scales_t"] = None, scales.clamp(min=LEAST / TOP)
        return got
    if s["op"] == "product":
        d = torch.float64
        b = _wide_rows(s["B"], s["sb"], d) if s["form"] == "rows" else _wide_blocks(s["B"], s["sb"], d)
        return _wide_rows(s["A"], s["sa"], d) @ b.t()
    if s["op"] == "experts":
        o, d = s["offsets"].tolist(), torch.float64
        a = _wide_rows(s["A"], s["sa"], d)
        if s["mode"] == "rows":
            return torch.cat([a[lo:hi] @ _wide_blocks(s["B"][e], s["sb"][e], d).t() for e, (lo, hi) in enumerate(zip(o, o[1:]))])
        b = _wide_rows(s["B"], s["sb"], d)
        out, at = [], 0
        for lo, hi in zip(o, o[1:]):
            out.append(a[:, at:at + hi - lo] @ b[:, at:at + hi - lo].t())
            at += _up(hi - lo, BLOCK)
        return torch.stack(out)
    y = s["Y"].double()[s["row_of"].long()]
    w = s["weights"].double()[:, :, None] if s["weights"] is not None else torch.ones_like(y[:, :, :1])
    got = dict(out=torch.einsum("tkc,tko->tc", y, w))
    if s["backward"]:
        g = s["grad_out"].double()
        back = torch.empty(s["row_of"].numel(), dtype=torch.long, device="cuda")
        back[s["row_of"].long().reshape(-1)] = torch.arange(back.numel(), device="cuda")
        got["grad_y"] = g[back // y.shape[1]] * w.reshape(-1, 1)[back]
        if s["weights"] is not None:
            got["grad_w"] = torch.einsum("tc,tkc->tk", g, y)
    return got
