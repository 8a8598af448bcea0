"""Cases of the operators of dense and experts' layers in 16 bits: the root-mean-square norm with the residual's
addition, products with bias, activation and a joined matrix in their epilogue (dense and over experts), and the
gradients of all of these.

``run`` computes them in plain torch operations, or, where ``own`` is true, through the library's entry points.
16-bit operands of products have rows that begin on 16 bytes; parameters (norm weights, biases) are in 32 bits.
"""

import math

import torch

own = False

BLOCK = 128                # values that share a scale of the 8-bit form
TOP = 448.0                # largest e4m3 value
LEAST = 2.0 ** -96         # a block's largest value counts as at least this
EPS = 1e-6
FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # One token of a decode step: the residual is added and the row goes to an 8-bit product.
        dict(name="norm_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, y=False, q=True),
        # A batch of prompts: the normalised rows both for a 16-bit and for an 8-bit product.
        dict(name="norm_prompts", op="norm", rows=8191, cols=4096, dtype="bf16", residual=True, y=True, q=True),
        # Odd rows in 32 bits, the first norm of a network: nothing to add.
        dict(name="norm_odd", op="norm", rows=4097, cols=3001, dtype="f32", residual=False, y=True, q=False),
        # Its gradient in a training step, with the one that comes along the residual.
        dict(name="norm_gradient", op="norm_gradient", rows=16383, cols=2048, dtype="bf16", residual=True),
        # One decode step of a linear layer: 16 tokens.
        dict(name="linear_decode", op="linear", M=16, N=4096, K=4096, act="silu", bias=True, join="none", pre=False, out="bf16"),
        # A short batch through the gated half of a feed-forward layer: silu of this product times the other one.
        dict(name="linear_gated", op="linear", M=256, N=4096, K=4096, act="silu", bias=False, join="mul", pre=False, out="bf16"),
        # The odd rectangle, with everything that an epilogue does, in 32 bits.
        dict(name="linear_odd", op="linear", M=4097, N=3001, K=2049, act="gelu", bias=True, join="add", pre=False, out="f32"),
        # A training batch through the first product of a feed-forward layer; what the gradient needs is kept.
        dict(name="linear_train", op="linear", M=16384, N=4096, K=4096, act="gelu_tanh", bias=True, join="none", pre=True, out="bf16"),
        # The gradients of such a layer: of its sum before the activation, its bias, its input and its weights.
        dict(name="linear_gradient", op="linear_gradient", M=8191, N=4096, K=2048, act="gelu", join="none", bias=True, out="bf16"),
        # A decode step's rows over the experts they went to.
        dict(name="experts_decode", op="experts", E=64, active=48, rows=96, N=2048, K=2048, act="silu", bias=False, join="mul", pre=False, out="bf16"),
        # A prompt batch over the experts; ragged counts, some experts empty.
        dict(name="experts_prompts", op="experts", E=64, active=60, rows=16384, N=2048, K=2048, act="silu", bias=False, join="mul", pre=False, out="bf16"),
        # The gradients of the experts of a training step.
        dict(name="experts_gradient", op="experts_gradient", E=16, active=15, rows=16383, N=2048, K=2048, act="silu", join="mul", bias=True, out="bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_gradient", "linear", "linear", "linear_gradient", "experts", "experts_gradient"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "norm":
        y = rng.random() < 0.7
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 16, 4096), dtype=dtype, residual=rng.random() < 0.7,
                    y=y, q=not y or rng.random() < 0.5)
    if op == "norm_gradient":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 16, 4096), dtype=dtype, residual=rng.random() < 0.7)
    act, bias = rng.choice(ACTS), rng.random() < 0.6
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 16, 4096), K=_log(rng, 16, 4096), act=act, bias=bias,
                    join=rng.choice(["none", "add", "mul"]), pre=rng.random() < 0.4, out=dtype)
    join = rng.choice(["none", "mul"])
    if op == "linear_gradient":
        # 16-bit gradients: what the products read of them is then what is returned.
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 4096), K=_log(rng, 16, 2048), act=act, join=join,
                    bias=bias, out="bf16")
    E, rows = rng.choice([4, 8, 16, 32, 64]), _log(rng, 1, 16384)
    c = dict(op=op, E=E, active=rng.randint(1, min(E, rows)), rows=rows, N=_log(rng, 64, 2048), K=_log(rng, 64, 2048),
             act=act, join=join, bias=bias, out="bf16")
    return dict(c, pre=rng.random() < 0.4, out=dtype) if op == "experts" else c


def _up(x, m):
    return (x + m - 1) // m * m


# ---------------------------------------------------------------- plain forms


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * (1.0 / (1.0 + torch.exp(-z)))


def _slope(z, act):
    """The activation's derivative."""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * (c * (1.0 + 3.0 * 0.044715 * z * z))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s + z * s * (1.0 - s)


def _plain_rows_form(x):
    """x (rows x cols) in 8 bits with a scale per row and 128 columns: q, scales [block][row]."""
    rows, cols = x.shape
    full = x.new_zeros(rows, _up(cols, BLOCK))
    full[:, :cols] = x
    b = full.view(rows, -1, BLOCK)
    most = b.abs().amax(2, keepdim=True).clamp(min=LEAST)
    q = (b * (TOP / most)).clamp(-TOP, TOP).to(FP8)
    return q.view(rows, -1)[:, :cols], (most / TOP)[:, :, 0].t().contiguous()


def _plain_norm(s):
    x = s["x"].float()
    if s["r"] is not None:
        x = x + s["r"].float()
    y = x * (1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)) * s["w"]
    got = {}
    if s["r"] is not None:
        got["sum"] = x.to(s["x"].dtype)
    if s["y"]:
        got["y"] = y.to(s["x"].dtype)
    if s["q"]:
        got["q"], got["scales"] = _plain_rows_form(y)
    return got


def _plain_norm_gradient(s):
    x, g = s["x"].float(), s["g"].float()
    i = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    h, gw = x * i, g * s["w"]
    d = i * (gw - h * (gw * h).mean(1, keepdim=True))
    if s["gs"] is not None:
        d = d + s["gs"].float()
    return dict(grad_x=d.to(s["x"].dtype), grad_w=(g * h).sum(0))


def _finish(s, z, D):
    """What an epilogue makes of the product z (with its bias) and the joined matrix."""
    y = _act(z, s["act"])
    if s["join"] == "add":
        y = y + D
    elif s["join"] == "mul":
        y = y * D
    return y


def _outputs(s, z, D):
    got = dict(C=_finish(s, z, D).to(s["out"]))
    if s["pre"]:
        got["pre"] = z.to(s["out"])
    return got


def _float(t):
    return None if t is None else t.float()


def _plain_linear(s):
    z = s["A"].float() @ s["B"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    return _outputs(s, z, _float(s["D"]))


def _plain_epilogue_gradient(s):
    """The gradients of an epilogue: of its sum before the activation (in 32 bits), and of the joined factor."""
    g, z = s["g"].float(), s["z"].float()
    dz = g * _slope(z, s["act"])
    if s["join"] != "mul":
        return dz, None
    return dz * s["D"].float(), (g * _act(z, s["act"])).to(s["out"])


def _plain_linear_gradient(s):
    dz, dD = _plain_epilogue_gradient(s)
    got = dict(grad_z=dz.to(s["out"]))
    if dD is not None:
        got["grad_D"] = dD
    if s["bias"]:
        got["grad_bias"] = dz.sum(0)
    # The products read the gradient as it is returned.
    dz = got["grad_z"].float()
    got["grad_x"] = (dz @ s["B"].float()).to(s["out"])
    got["grad_w"] = (dz.t() @ s["A"].float()).to(s["out"])
    return got


def _padded_groups(s):
    """(E x cap places of the groups' members, which of them are some)."""
    start, counts = s["offsets"][:-1].long(), s["offsets"][1:].long() - s["offsets"][:-1].long()
    at = torch.arange(s["cap"], device=counts.device)
    there = at[None, :] < counts[:, None]
    return torch.where(there, start[:, None] + at[None, :], 0), there


def _plain_experts(s):
    at, there = _padded_groups(s)
    z = torch.bmm(s["A"].float()[at], s["B"].float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"][:, None, :]
    return _outputs(s, z[there], _float(s["D"]))


def _plain_experts_gradient(s):
    at, there = _padded_groups(s)
    dz, dD = _plain_epilogue_gradient(s)
    got = dict(grad_z=dz.to(s["out"]))
    if dD is not None:
        got["grad_D"] = dD
    some = there[:, :, None]
    if s["bias"]:
        got["grad_bias"] = (dz[at] * some).sum(1)
    # The products read the gradient as it is returned.
    d = got["grad_z"].float()[at] * some
    got["grad_x"] = torch.bmm(d, s["B"].float())[there].to(s["out"])
    got["grad_w"] = torch.bmm(d.transpose(1, 2), s["A"].float()[at] * some).to(s["out"])
    return got


# ------------------------------------------------------- the library's calls


def _ok(sg, code):
    if code != sg.SGEMM_OK:
        raise sg.SgemmError(code, "perf")


def _type(sg, dtype):
    return sg.SGEMM_F32 if dtype == torch.float32 else sg.SGEMM_BF16


def _new(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _rows16(rows, cols, dtype):
    """An uninitialised matrix whose rows begin on 16 bytes."""
    return _new((rows, _up(cols, 16 // dtype.itemsize)), dtype)[:, :cols]


def _at(t):
    return 0 if t is None else t.data_ptr()


def _ld(t):
    return 0 if t is None else t.stride(0)


def _act_id(sg, act):
    return {"none": sg.SGEMM_ACT_NONE, "relu": sg.SGEMM_ACT_RELU, "gelu": sg.SGEMM_ACT_GELU,
            "gelu_tanh": sg.SGEMM_ACT_GELU_TANH, "silu": sg.SGEMM_ACT_SILU}[act]


def _join_id(sg, join):
    return {"none": sg.SGEMM_JOIN_NONE, "add": sg.SGEMM_JOIN_ADD, "mul": sg.SGEMM_JOIN_MUL}[join]


def _own_norm(sg, s, st):
    x, r = s["x"], s["r"]
    rows, cols = x.shape
    got = {}
    if r is not None:
        got["sum"] = _new((rows, cols), x.dtype)
    if s["y"]:
        got["y"] = _new((rows, cols), x.dtype)
    q = None
    if s["q"]:
        q, got["scales"] = _new((rows, _up(cols, 16)), FP8), _new((_up(cols, BLOCK) // BLOCK, rows), torch.float32)
        got["q"] = q[:, :cols]
    _ok(sg, sg.sgemm_rms_norm(rows, cols, _type(sg, x.dtype), x.data_ptr(), x.stride(0), _at(r), _ld(r),
                              s["w"].data_ptr(), EPS, _at(got.get("sum")), cols, _at(got.get("y")), cols,
                              _at(q), _ld(q), _at(got.get("scales")), rows, st))
    return got


def _own_norm_gradient(sg, s, st):
    x, g, gs = s["x"], s["g"], s["gs"]
    rows, cols = x.shape
    d, dw = _new((rows, cols), x.dtype), _new(cols, torch.float32)
    _ok(sg, sg.sgemm_rms_norm_backward(rows, cols, _type(sg, x.dtype), g.data_ptr(), g.stride(0), x.data_ptr(),
                                       x.stride(0), s["w"].data_ptr(), EPS, _at(gs), _ld(gs), d.data_ptr(), cols,
                                       dw.data_ptr(), st))
    return dict(grad_x=d, grad_w=dw)


def _own_linear(sg, s, st):
    A, B, D = s["A"], s["B"], s["D"]
    (M, K), N = A.shape, B.shape[0]
    got = dict(C=_new((M, N), s["out"]))
    if s["pre"]:
        got["pre"] = _new((M, N), s["out"])
    _ok(sg, sg.sgemm_bf16(0, 1, M, N, K, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0), _at(s["bias"]),
                          _act_id(sg, s["act"]), _at(got.get("pre")), N, _join_id(sg, s["join"]), _at(D), _ld(D),
                          got["C"].data_ptr(), _type(sg, s["out"]), N, st))
    return got


def _own_epilogue_gradient(sg, s, st, groups, offsets):
    """The gradients of an epilogue: of its sum before the activation, of the joined factor, and of the bias."""
    g, z, D = s["g"], s["z"], s["D"]
    rows, cols = g.shape
    dz = _rows16(rows, cols, s["out"])
    dD = _new((rows, cols), s["out"]) if s["join"] == "mul" else None
    db = _new((groups, cols), torch.float32) if s["bias"] else None
    _ok(sg, sg.sgemm_epilogue_backward(rows, cols, _type(sg, g.dtype), g.data_ptr(), g.stride(0), z.data_ptr(),
                                       z.stride(0), _act_id(sg, s["act"]), _join_id(sg, s["join"]), _at(D), _ld(D),
                                       groups, _at(offsets), dz.data_ptr(), dz.stride(0), _at(dD), cols, _at(db), cols,
                                       st))
    got = dict(grad_z=dz)
    if dD is not None:
        got["grad_D"] = dD
    if db is not None:
        got["grad_bias"] = db if offsets is not None else db[0]
    return got


def _own_linear_gradient(sg, s, st):
    A, B = s["A"], s["B"]
    (M, K), N, kind = A.shape, B.shape[0], _type(sg, s["out"])
    got = _own_epilogue_gradient(sg, s, st, 1, None)
    dz, dx, dw = got["grad_z"], _new((M, K), s["out"]), _new((N, K), s["out"])
    _ok(sg, sg.sgemm_bf16(0, 0, M, K, N, dz.data_ptr(), dz.stride(0), B.data_ptr(), B.stride(0), 0, sg.SGEMM_ACT_NONE,
                          0, 0, sg.SGEMM_JOIN_NONE, 0, 0, dx.data_ptr(), kind, K, st))
    _ok(sg, sg.sgemm_bf16(1, 0, N, K, M, dz.data_ptr(), dz.stride(0), A.data_ptr(), A.stride(0), 0, sg.SGEMM_ACT_NONE,
                          0, 0, sg.SGEMM_JOIN_NONE, 0, 0, dw.data_ptr(), kind, K, st))
    return dict(got, grad_x=dx, grad_w=dw)


def _own_experts(sg, s, st):
    A, B, D, bias = s["A"], s["B"], s["D"], s["bias"]
    (R, K), (E, N, _) = A.shape, B.shape
    got = dict(C=_new((R, N), s["out"]))
    if s["pre"]:
        got["pre"] = _new((R, N), s["out"])
    _ok(sg, sg.sgemm_bf16_grouped(1, E, s["offsets"].data_ptr(), R, N, K, A.data_ptr(), A.stride(0), B.data_ptr(),
                                  B.stride(1), B.stride(0), _at(bias), N, _act_id(sg, s["act"]), _at(got.get("pre")), N,
                                  _join_id(sg, s["join"]), _at(D), _ld(D), got["C"].data_ptr(), _type(sg, s["out"]), N,
                                  st))
    return got


def _own_experts_gradient(sg, s, st):
    A, B, offsets = s["A"], s["B"], s["offsets"]
    (R, K), (E, N, _), kind = A.shape, B.shape, _type(sg, s["out"])
    got = _own_epilogue_gradient(sg, s, st, E, offsets)
    dz, dx, dw = got["grad_z"], _new((R, K), s["out"]), _new((E, N, K), s["out"])
    _ok(sg, sg.sgemm_bf16_grouped(0, E, offsets.data_ptr(), R, K, N, dz.data_ptr(), dz.stride(0), B.data_ptr(),
                                  B.stride(1), B.stride(0), 0, 0, sg.SGEMM_ACT_NONE, 0, 0, sg.SGEMM_JOIN_NONE, 0, 0,
                                  dx.data_ptr(), kind, K, st))
    _ok(sg, sg.sgemm_bf16_grouped_k(E, offsets.data_ptr(), R, N, K, dz.data_ptr(), dz.stride(0), A.data_ptr(),
                                    A.stride(0), 0, dw.data_ptr(), kind, K, N * K, st))
    return dict(got, grad_x=dx, grad_w=dw)


def run(state):
    op = state["op"]
    if not own:
        return {"norm": _plain_norm, "norm_gradient": _plain_norm_gradient, "linear": _plain_linear,
                "linear_gradient": _plain_linear_gradient, "experts": _plain_experts,
                "experts_gradient": _plain_experts_gradient}[op](state)
    import dense_fp32_matrix_07_gb300 as sg
    stream = torch.cuda.current_stream().cuda_stream
    return {"norm": _own_norm, "norm_gradient": _own_norm_gradient, "linear": _own_linear,
            "linear_gradient": _own_linear_gradient, "experts": _own_experts,
            "experts_gradient": _own_experts_gradient}[op](sg, state, stream)


# --------------------------------------------------------------------- inputs


def _activations(gen, rows, cols):
    """Normal values with a few channels that are much larger, as activations have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return x * torch.exp(torch.randn(cols, generator=gen, device="cuda"))


def _strided(x):
    """x (..., cols) in bfloat16 with rows that begin on 16 bytes."""
    full = torch.zeros((*x.shape[:-1], _up(x.shape[-1], 8)), dtype=torch.bfloat16, device=x.device)
    full[..., :x.shape[-1]] = x
    return full[..., :x.shape[-1]]


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

    if c["op"] in ("norm", "norm_gradient"):
        dtype, rows, cols = TYPES[c["dtype"]], c["rows"], c["cols"]
        s = dict(op=c["op"], x=_activations(gen, rows, cols).to(dtype), w=1.0 + 0.1 * normal(cols))
        more = normal(rows, cols).to(dtype) if c["residual"] else None
        if c["op"] == "norm":
            return dict(s, r=more, y=c["y"], q=c["q"])
        return dict(s, gs=more, g=normal(rows, cols).to(dtype))
    rows = c["rows"] if "rows" in c else c["M"]
    N, K, out = c["N"], c["K"], TYPES[c["out"]]
    s = dict(op=c["op"], act=c["act"], join=c["join"], out=out, A=_strided(_activations(gen, rows, K) / 2.0))
    w = () if "M" in c else (c["E"],)
    s["B"] = _strided(normal(*w, N, K) / math.sqrt(K))
    s["D"] = normal(rows, N).to(out) if c["join"] != "none" else None
    if "E" in c:
        s["offsets"], counts = _offsets(gen, c["E"], c["active"], rows)
        s["cap"] = max(counts)
    if c["op"] in ("linear", "experts"):
        return dict(s, bias=0.1 * normal(*w, N) if c["bias"] else None, pre=c["pre"])
    return dict(s, bias=c["bias"], g=normal(rows, N).to(out), z=(1.5 * normal(rows, N)).to(out))


def work(case):
    c = case
    if c["op"] in ("norm", "norm_gradient"):
        n, size = c["rows"] * c["cols"], SIZE[c["dtype"]]
        if c["op"] == "norm":
            b = n * size * (1 + 2 * c["residual"] + c["y"]) + (n * (1 + 4 / BLOCK) if c["q"] else 0) + 4 * c["cols"]
            return dict(bytes=b, flops=6 * n)
        return dict(bytes=n * size * (3 + c["residual"]) + 8 * c["cols"], flops=10 * n)
    rows = c["rows"] if "rows" in c else c["M"]
    N, K, size = c["N"], c["K"], SIZE[c["out"]]
    n, active, E = rows * N, c.get("active", 1), c.get("E", 1)
    if c["op"] in ("linear", "experts"):
        b = 2 * (rows + active * N) * K + n * size * (1 + c["pre"] + (c["join"] != "none")) + 4 * active * N * c["bias"]
        return dict(bytes=b, flops=2 * n * K)
    mul = c["join"] == "mul"
    b = n * size * (3 + 2 * mul) + 4 * E * N * c["bias"]               # g, z, the gradient of z; D and its gradient; bias
    b += 2 * (rows + active * N) * K + size * (rows + E * N) * K       # x and the weights, and their gradients
    return dict(bytes=b, flops=4 * n * K)


# ------------------------------------------------------------- 64-bit results


def _exact_act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return z * torch.special.expit(z) if act == "silu" else z


def _exact_epilogue(s, z):
    y = _exact_act(z, s["act"])
    if s["join"] != "none":
        y = y + s["D"].double() if s["join"] == "add" else y * s["D"].double()
    return dict(C=y, pre=z) if s["pre"] else dict(C=y)


def _exact_epilogue_gradient(s):
    z = s["z"].double().requires_grad_(True)
    with torch.enable_grad():
        y = _exact_act(z, s["act"])
        up = s["g"].double() * (s["D"].double() if s["join"] == "mul" else 1.0)
        got = dict(grad_z=torch.autograd.grad(y, z, up)[0])
    if s["join"] == "mul":
        got["grad_D"] = s["g"].double() * y.detach()
    return got


def exact(case, seed):
    """The definition in 64 bits. What is held in 8 bits has no value that is not rounded: None there."""
    s = prepare(case, seed)
    if s["op"] == "norm":
        x = s["x"].double() + (0.0 if s["r"] is None else s["r"].double())
        y = x / (x.square().sum(1, keepdim=True) / x.shape[1] + EPS).sqrt() * s["w"].double()
        got = dict(sum=x) if s["r"] is not None else {}
        if s["y"]:
            got["y"] = y
        if s["q"]:
            most = torch.stack([p.abs().amax(1) for p in torch.split(y, BLOCK, 1)])
            got["q"], got["scales"] = None, most.clamp(min=LEAST) / TOP
        return got
    if s["op"] == "norm_gradient":
        x, w = s["x"].double().requires_grad_(True), s["w"].double().requires_grad_(True)
        with torch.enable_grad():
            y = x / (x.square().sum(1, keepdim=True) / x.shape[1] + EPS).sqrt() * w
            dx, dw = torch.autograd.grad(y, (x, w), s["g"].double())
        return dict(grad_x=dx if s["gs"] is None else dx + s["gs"].double(), grad_w=dw)
    A, B = s["A"].double(), s["B"]
    if s["op"] == "linear":
        z = torch.einsum("mk,nk->mn", A, B.double())
        return _exact_epilogue(s, z if s["bias"] is None else z + s["bias"].double())
    if s["op"] == "linear_gradient":
        got = _exact_epilogue_gradient(s)
        if s["bias"]:
            got["grad_bias"] = got["grad_z"].sum(0)
        return dict(got, grad_x=torch.einsum("mn,nk->mk", got["grad_z"], B.double()),
                    grad_w=torch.einsum("mn,mk->nk", got["grad_z"], A))
    o = s["offsets"].tolist()
    parts = [(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(o, o[1:]))]
    if s["op"] == "experts":
        z = torch.cat([A[p] @ B[e].double().t() + (0.0 if s["bias"] is None else s["bias"][e].double()) for e, p in parts])
        return _exact_epilogue(s, z)
    got = _exact_epilogue_gradient(s)
    dz = got["grad_z"]
    if s["bias"]:
        got["grad_bias"] = torch.stack([dz[p].sum(0) for _, p in parts])
    return dict(got, grad_x=torch.cat([dz[p] @ B[e].double() for e, p in parts]),
                grad_w=torch.stack([dz[p].t() @ A[p] for _, p in parts]))
