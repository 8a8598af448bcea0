"""GPU parity of the operators of layers in 16 bits (16-bit products with an
epilogue, its gradient, the root-mean-square norm) against plain restatements
in 64 bits (layers_ref), at the sizes, masks, strides and alignments where they
can go wrong. Each bound is derived where it is computed."""

import itertools

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
import layers_ref as ref
from test_experts_gpu import Guarded, finish, ok, stream

pytestmark = pytest.mark.gpu

F32, BF16 = sg.SGEMM_F32, sg.SGEMM_BF16
TYPES = {F32: torch.float32, BF16: torch.bfloat16}
NAN = float("nan")
SMS = 152


def up(n, m):
    return (n + m - 1) // m * m


def operand(x, more=0):
    """x (..., rows, cols) in bfloat16 with rows on 16 bytes and NaN between them: (buffer, leading dimension)."""
    ld = up(x.shape[-1], 8) + more
    buf = torch.full((*x.shape[:-1], ld), NAN, dtype=torch.bfloat16, device="cuda")
    buf[..., :x.shape[-1]] = x
    return buf, ld


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def gen(*numbers):
    return torch.Generator(device="cuda").manual_seed(sum(n * 31 ** i for i, n in enumerate(numbers)) % 2 ** 31)


def matrix(rows, cols, dtype, aligned):
    """An output that is accessed 16 bytes at a time, or one that cannot be."""
    return Guarded(rows, cols, up(cols, 8) + 8, dtype) if aligned else Guarded(rows, cols, cols + 3, dtype, shift=1)


def ptr(m):
    return m.ptr if m is not None else 0


def ld(m):
    return m.ld if m is not None else 0


class Case:
    """Operands, bias and joined matrix of a dense product, and what it should give."""

    def __init__(self, M, N, K, op_a, op_b, ctype, act=0, join=0, bias=False, pre=False, aligned=True, integers=False):
        g = gen(M, N, K, act, join)
        self.dims, self.ops, self.ctype, self.act, self.join = (M, N, K), (op_a, op_b), ctype, act, join
        dtype = TYPES[ctype]
        if integers:
            a = torch.randint(-3, 4, (M, K), generator=g, device="cuda").double()
            b = torch.randint(-3, 4, (K, N), generator=g, device="cuda").double()
        else:
            a = normal(g, M, K).bfloat16().double()
            b = (normal(g, K, N) / max(1, K) ** 0.5).bfloat16().double()
        self.A, self.lda = operand((a.t() if op_a else a).bfloat16(), 8)
        self.B, self.ldb = operand((b.t() if op_b else b).bfloat16())
        self.bias = torch.randint(-3, 4, (N,), generator=g, device="cuda").float() if bias else None
        self.C = matrix(M, N, dtype, aligned)
        self.pre = matrix(M, N, dtype, aligned) if pre else None
        self.D = None
        if join:
            d = torch.randint(-3, 4, (M, N), generator=g, device="cuda").to(dtype)
            self.D = matrix(M, N, dtype, aligned).put(d)
        self.z, S = ref.product(a, b)
        if bias:
            self.z, S = self.z + self.bias.double(), S + self.bias.abs().double()
        self.error = ref.sum_error(S, K)
        self.exact = integers

    def run(self, D=None):
        (M, N, K), (op_a, op_b) = self.dims, self.ops
        D = D or self.D
        ok(sg.sgemm_bf16(op_a, op_b, M, N, K, self.A.data_ptr(), self.lda, self.B.data_ptr(), self.ldb,
                         self.bias.data_ptr() if self.bias is not None else 0, self.act, ptr(self.pre), ld(self.pre),
                         self.join, ptr(D), ld(D), self.C.ptr, self.ctype, self.C.ld, stream()))
        finish()
        return self

    def check(self):
        dtype = TYPES[self.ctype]
        D = self.D.view().double() if self.D is not None else None
        want, bound, pre_bound = ref.epilogue(self.z, self.error, ref.ACTS[self.act], ref.JOINS[self.join], D, dtype)
        got = self.C.view()
        if self.exact and self.act < 2:      # whole numbers, added up exactly, rounded once
            assert torch.equal(got, want.to(dtype))
        ref.close(got, want, bound, "C")
        assert self.C.outside_untouched()
        if self.pre is not None:
            ref.close(self.pre.view(), self.z, pre_bound, "pre")
            assert self.pre.outside_untouched()


# ------------------------------------------------------------- dense products

# Around every tile edge (16 to 256 columns, 128 and 256 lanes), ends of K inside 16 and 64, K in 512s, split K, waves.
SHAPES = [(1, 1, 1), (1, 129, 16), (3, 257, 127), (16, 128, 129), (17, 4096, 1024), (33, 640, 513), (64, 1024, 2048),
          (65, 384, 256), (127, 130, 385), (128, 256, 128), (129, 255, 300), (300, 511, 1000), (1000, 777, 640),
          (2500, 1200, 272), (8, 7000, 4096), (3000, 17, 400), (5121, 1025, 1296), (2000, 60, 64), (64, 64, 6000)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ops", [(0, 1), (0, 0), (1, 0), (1, 1)], ids=lambda o: "op%d%d" % o)
@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
def test_product_of_integers_is_exact(cuda_device, shape, ops, ctype):
    Case(*shape, *ops, ctype, integers=True, aligned=shape[0] % 2 == 0).run().check()


@pytest.mark.parametrize("shape", [(1, 129, 16), (33, 640, 513), (129, 255, 300), (1000, 777, 640), (3000, 17, 400),
                                   (1500, 1030, 1100)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", range(5), ids=ref.ACTS)
@pytest.mark.parametrize("join", range(3), ids=ref.JOINS)
@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
def test_epilogue(cuda_device, shape, act, join, ctype):
    for aligned, bias, pre in ((True, True, True), (False, True, True), (True, False, join == 1), (False, act == 2, False)):
        Case(*shape, 0, 1, ctype, act=act, join=join, bias=bias, pre=pre, aligned=aligned).run().check()


def plan_of(M, N, K):
    rc, *plan = sg.sgemm_bf16_plan(sg.SGEMM_BF16_DENSE, 1, M, N, K, SMS)
    assert rc == sg.SGEMM_OK
    return tuple(plan[:4])


# One shape for each kernel shape that the rule gives: columns, pair, swapped, split.
@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
def test_every_kernel_shape(cuda_device, ctype):
    seen = {}
    for M, N, K in itertools.product((5, 30, 60, 100, 200, 500, 900, 1500, 5000), (20, 100, 300, 1100, 4100), (100, 1030, 5000)):
        if M * N * K <= 6e9:
            seen.setdefault(plan_of(M, N, K), (M, N, K))
    kinds = {(c, p) for c, p, _, _ in seen}
    assert kinds == {(16, 0), (32, 0), (64, 0), (128, 0), (128, 1), (256, 1)}, kinds
    assert {s for *_, s in seen} == {1, 2, 4, 8} and {w for _, _, w, _ in seen} == {0, 1}
    for shape in seen.values():
        Case(*shape, 0, 1, ctype, act=4, join=1, bias=True, pre=True, integers=True).run().check()


@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [10, 900])
def test_no_k_gives_the_epilogue_of_the_bias(cuda_device, ctype, M):
    for act, join, bias in ((0, 0, False), (4, 2, True), (2, 1, True)):
        Case(M, 300, 0, 0, 1, ctype, act=act, join=join, bias=bias, pre=True).run().check()


@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(20, 500, 1024), (700, 600, 300)], ids=["split", "tiles"])
@pytest.mark.parametrize("join", [1, 2])
def test_joined_matrix_in_the_place_of_c(cuda_device, ctype, shape, join):
    c = Case(*shape, 0, 1, ctype, act=4, join=join, bias=True)
    c.C.put(c.D.view())
    c.run(D=c.C).check()


def test_infinities_and_nan_stay_in_their_rows_and_columns(cuda_device):
    c = Case(300, 400, 200, 0, 1, F32, bias=True, act=1)
    c.A[7, 3], c.A[9, 199], c.B[11, 5] = NAN, float("inf"), NAN
    c.run()
    got, want = c.C.view(), c.z.clamp(min=0)
    assert bool(torch.isnan(got[7]).all()) and bool(torch.isnan(got[:, 11]).all())
    rows = [r for r in range(300) if r not in (7, 9)]
    cols = [n for n in range(400) if n != 11]
    ref.close(got[rows][:, cols], want[rows][:, cols], c.error[rows][:, cols] * 1.01 + 1e-6)
    assert bool((~torch.isfinite(got[9]) | (got[9] == 0)).all())


# ----------------------------------------------------------- groups of rows


def offsets_of(counts, first=0):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[0] = first
    off[1:] = first + torch.tensor(counts).cumsum(0)
    return off.tolist(), off.cuda()


COUNTS = [[5], [0, 3, 0, 1], [1] * 40, [17, 0, 33, 64, 15, 0], [200, 0, 1, 130, 256, 65], [700, 3, 513, 0, 300, 128], [0, 0]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("op_b", [1, 0])
@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
def test_groups_of_rows(cuda_device, counts, op_b, ctype):
    dtype = TYPES[ctype]
    E, first, behind = len(counts), 2, 5
    R = first + sum(counts) + behind
    for N, K, act, join, bias, aligned in ((136, 72, 0, 0, False, True), (301, 200, 4, 2, True, False), (520, 648, 2, 1, True, True)):
        g = gen(R, N, K, E)
        o, off = offsets_of(counts, first)
        a, b = normal(g, R, K).bfloat16(), (normal(g, E, K, N) / K ** 0.5).bfloat16()
        a[:first], a[R - behind:] = NAN, NAN           # rows of no group
        A, lda = operand(a)
        B, ldb = operand(b.transpose(1, 2) if op_b else b)
        bi = normal(g, E, N + 1) if bias else None
        D = matrix(R, N, dtype, aligned).put(normal(g, R, N).to(dtype)) if join else None
        C, pre = matrix(R, N, dtype, aligned), matrix(R, N, dtype, aligned)
        ok(sg.sgemm_bf16_grouped(op_b, E, off.data_ptr(), R, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, B.stride(0),
                                 bi.data_ptr() if bias else 0, N + 1, act, pre.ptr, pre.ld, join, ptr(D), ld(D), C.ptr, ctype,
                                 C.ld, stream()))
        finish()
        for e in range(E):
            rows = slice(o[e], o[e + 1])
            z, S = ref.product(a[rows].double(), b[e].double())
            if bias:
                z, S = z + bi[e, :N].double(), S + bi[e, :N].abs().double()
            want, bound, pre_bound = ref.epilogue(z, ref.sum_error(S, K), ref.ACTS[act], ref.JOINS[join],
                                                  D.view()[rows].double() if join else None, dtype)
            ref.close(C.view()[rows], want, bound, ("C", e, N))
            ref.close(pre.view()[rows], z, pre_bound, ("pre", e, N))
        for m in (C, pre):
            assert m.outside_untouched()
            assert bool((m.view()[:first] == m.fill).all()) and bool((m.view()[R - behind:] == m.fill).all())


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_groups_rows_as_k(cuda_device, counts, ctype, accumulate):
    dtype = TYPES[ctype]
    E, first, behind = len(counts), 3, 4
    R = first + sum(counts) + behind
    for M, N, aligned in ((8, 24, True), (130, 72, False), (264, 520, True), (777, 300, True)):
        g = gen(R, M, N, E)
        o, off = offsets_of(counts, first)
        a, b = normal(g, R, M).bfloat16(), normal(g, R, N).bfloat16()
        # What a group holds stays its own: NaN and infinities in the rows of none and in a whole group.
        a[:first], b[R - behind:] = NAN, float("inf")
        bad = [e for e in range(E) if counts[e]][1:2]
        for e in bad:
            a[o[e]:o[e + 1]] = NAN
            b[o[e]:o[e + 1]] = float("inf")
        A, lda = operand(a)
        B, ldb = operand(b)
        rows_c = E * M + E           # a row between the groups' matrices
        C = matrix(rows_c, N, dtype, aligned)
        stride = (M + 1) * C.ld
        old = normal(g, rows_c, N).to(dtype)
        C.put(old)
        C.start = C.flat.clone()
        ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), R, M, N, A.data_ptr(), lda, B.data_ptr(), ldb, accumulate, C.ptr, ctype,
                                   C.ld, stride, stream()))
        finish()
        for e in range(E):
            rows = slice(o[e], o[e + 1])
            got, was = C.view()[e * (M + 1):e * (M + 1) + M], old[e * (M + 1):e * (M + 1) + M].double()
            if e in bad:
                assert bool(torch.isnan(got).all())
                continue
            z, S = ref.product(a[rows].double().t(), b[rows].double())
            want, bound, _ = ref.epilogue(z, ref.sum_error(S, counts[e]), "none", "add" if accumulate else "none", was, dtype)
            ref.close(got, want, bound, ("C", e, M, N))
            assert torch.equal(C.view()[e * (M + 1) + M], old[e * (M + 1) + M])
        assert C.outside_untouched()


@pytest.mark.parametrize("values", [[0, 500, 100, 400, 50], [-5, 10, 10 ** 9, 300, 7], [900, 900, 900, 900, 900],
                                    [2 ** 31 - 1] * 5, [5, 4, 3, 2, 1]], ids=lambda v: "-".join(map(str, v)))
def test_offsets_that_are_no_partition_stay_in_bounds(cuda_device, values):
    """Each group's rows are held to the matrices; what rows of several groups hold is not defined, the rest is not written."""
    R, N, K, E = 320, 200, 136, 4
    off = torch.tensor(values, dtype=torch.int32).cuda()
    A, lda = operand(torch.ones(R, K, device="cuda").bfloat16())
    B, ldb = operand(torch.ones(E, N, K, device="cuda").bfloat16())
    C = Guarded(R, N, N, torch.float32)
    ok(sg.sgemm_bf16_grouped(1, E, off.data_ptr(), R, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, B.stride(0), 0, 0, 0, 0, 0, 0,
                             0, 0, C.ptr, F32, C.ld, stream()))
    finish()
    assert C.outside_untouched() and bool(((C.view() == K) | (C.view() == C.fill)).all())
    G, ldg = operand(torch.ones(R, N, device="cuda").bfloat16())
    W = Guarded(E * N, K, K, torch.float32)
    ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), R, N, K, G.data_ptr(), ldg, A.data_ptr(), lda, 0, W.ptr, F32, K, N * K, stream()))
    finish()
    assert W.outside_untouched()
    for e in range(E):
        lo = min(max(values[e], 0), R)
        hi = min(max(values[e + 1], lo), R)
        assert bool((W.view()[e * N:(e + 1) * N] == hi - lo).all())
    dz, db = Guarded(R, N, N, torch.float32), Guarded(E, N, N, torch.float32)
    g = torch.ones(R, N, device="cuda")
    ok(sg.sgemm_epilogue_backward(R, N, F32, g.data_ptr(), N, 0, 0, 0, 0, 0, 0, E, off.data_ptr(), dz.ptr, N, 0, 0, db.ptr, N,
                                  stream()))
    finish()
    assert dz.outside_untouched() and db.outside_untouched()


# --------------------------------------------------- gradient of the epilogue


def slope_error(z):
    """The slopes in FP32: as the activations' own error, with a slope's slope of at most 1.13 and terms of at most
    1 + |z|: 48 * 2^-24 (1 + |z|)."""
    return 48.0 * 2.0 ** -24 * (1.0 + z.abs())


@pytest.mark.parametrize("act", range(5), ids=ref.ACTS)
@pytest.mark.parametrize("join", range(3), ids=ref.JOINS)
@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
def test_epilogue_backward(cuda_device, act, join, type):
    dtype, half = TYPES[type], ref.half_step(TYPES[type])
    for counts, cols, aligned in ((None, 1, True), (None, 300, False), ([64, 0, 65, 1], 264, True), ([7, 500, 0, 129], 301, False),
                                  (None, 1000, True)):
        g = gen(act, join, cols)
        first, behind = (2, 3) if counts else (0, 0)
        R = first + sum(counts) + behind if counts else 517
        o, off = offsets_of(counts, first) if counts else ([0, R], None)
        E = len(o) - 1
        put = lambda x: matrix(R, cols, dtype, aligned).put(x.to(dtype))  # noqa: E731
        go, z, D = put(normal(g, R, cols)), put(3.0 * normal(g, R, cols)), put(normal(g, R, cols))
        z.view()[R // 2, 0] = 0.0
        dz, dD, db = matrix(R, cols, dtype, aligned), matrix(R, cols, dtype, aligned), Guarded(E, cols, cols + 5, torch.float32)
        mul = join == 2
        ok(sg.sgemm_epilogue_backward(R, cols, type, go.ptr, go.ld, z.ptr, z.ld, act, join, ptr(D) if join else 0, D.ld, E,
                                      off.data_ptr() if counts else 0, dz.ptr, dz.ld, dD.ptr if mul else 0, dD.ld, db.ptr,
                                      db.ld, stream()))
        finish()
        x, G, d = z.view().double(), go.view().double(), D.view().double() if mul else torch.ones(R, cols, device="cuda").double()
        want, e = G * ref.slope(x, ref.ACTS[act]) * d, (G * d).abs() * (slope_error(x) if act else 0.0) + 2.0 ** -126
        e = e + 2 * 2.0 ** -24 * want.abs() if act or mul else e        # two products
        rows = slice(o[0], o[-1])
        ref.close(dz.view()[rows], want[rows], (e + half * (want.abs() + e))[rows], "dz")
        if mul:
            y = G * ref.act(x, ref.ACTS[act])
            e_y = G.abs() * ref.ACT_ERROR * x.abs() + 2.0 ** -24 * y.abs() + 2.0 ** -126
            ref.close(dD.view()[rows], y[rows], (e_y + half * (y.abs() + e_y))[rows], "dD")
            assert dD.outside_untouched()
        for i in range(E):
            r = slice(o[i], o[i + 1])
            n = o[i + 1] - o[i]
            ref.close(db.view()[i], want[r].sum(0), e[r].sum(0) + n * 2.0 ** -24 * want[r].abs().sum(0) + 2.0 ** -126, ("db", i))
        for m in (dz, db):
            assert m.outside_untouched()
        if counts:
            for m in (dz, dD):
                assert bool((m.view()[:first] == m.fill).all()) and bool((m.view()[R - behind:] == m.fill).all())


def test_epilogue_backward_parts_on_request(cuda_device):
    R, cols = 100, 72
    g, z, D = (torch.randn(R, cols, device="cuda") for _ in range(3))
    def run(act, join, want_z, want_D, want_b, pre=True):
        out = [torch.full((R, cols), 5.0, device="cuda"), torch.full((R, cols), 5.0, device="cuda"), torch.full((cols,), 5.0, device="cuda")]
        p = [o.data_ptr() if w else 0 for o, w in zip(out, (want_z, want_D, want_b))]
        ok(sg.sgemm_epilogue_backward(R, cols, F32, g.data_ptr(), cols, z.data_ptr() if pre else 0, cols, act, join, D.data_ptr(), cols,
                                      1, 0, p[0], cols, p[1], cols, p[2], cols, stream()))
        finish()
        return out
    whole = run(4, 2, True, True, True)
    for wants in itertools.product((False, True), repeat=3):
        for got, w, all_ in zip(run(4, 2, *wants), wants, whole):
            assert torch.equal(got, all_) if w else bool((got == 5.0).all())
    got = run(0, 1, True, False, True, pre=False)         # nothing of z is read
    assert torch.equal(got[0], g)
    # No rows: a bias gradient of zeros.
    db = torch.full((3, cols), 5.0, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok(sg.sgemm_epilogue_backward(0, cols, F32, 0, cols, 0, cols, 4, 0, 0, 0, 3, off.data_ptr(), 0, 0, 0, 0, db.data_ptr(), cols, stream()))
    finish()
    assert bool((db == 0).all())


@pytest.mark.parametrize("act", range(1, 5), ids=ref.ACTS[1:])
def test_epilogue_backward_against_differences(cuda_device, act):
    """(f(z + h) - f(z - h)) / 2h of the product's own epilogue, over FP32 sums that are exact: rounding gives 2 * 2^-24
    |f| ACT_ERROR-like terms over 2 h, the difference h^2 / 6 times a third derivative of at most 4."""
    n, h = 256, 2.0 ** -5
    z = torch.linspace(-4, 4, n, device="cuda").bfloat16()
    z = torch.where(z.abs() < 2 * h, torch.full_like(z, 1.0), z)          # relu has no derivative at 0
    eye = torch.eye(n, device="cuda").bfloat16()
    def f(bias):
        C = torch.empty(1, n, device="cuda")
        ok(sg.sgemm_bf16(0, 1, 1, n, n, z.data_ptr(), n, eye.data_ptr(), n, bias.data_ptr(), act, 0, 0, 0, 0, 0, C.data_ptr(), F32, n, stream()))
        return C[0].double()
    up_, down = torch.full((n,), h, device="cuda"), torch.full((n,), -h, device="cuda")
    want = (f(up_) - f(down)) / (2 * h)
    g, dz, z32 = torch.ones(1, n, device="cuda"), torch.empty(1, n, device="cuda"), z.float()
    ok(sg.sgemm_epilogue_backward(1, n, F32, g.data_ptr(), n, z32.data_ptr(), n, act, 0, 0, 0, 1, 0, dz.data_ptr(), n, 0, 0, 0, 0, stream()))
    finish()
    bound = h * h / 6 * 4 + 2 * (ref.ACT_ERROR * 4.1) / (2 * h) + 1e-6
    assert bool(((dz[0].double() - want).abs() <= bound).all())


# --------------------------------------------------------------------- norm

NORMS = [(1, 1), (3, 7), (1, 4096), (5, 127), (9, 256), (17, 257), (33, 1000), (8, 1024), (20, 1025), (7, 2048), (11, 3001), (6, 4100),
         (3, 8192), (2, 8200), (2, 16384), (300, 520)]


def norm_error(s, y, cols):
    """The sum of squares: cols additions in any order and the squares, (cols + 1) 2^-24 relative, halved by the root; its
    reciprocal 2^-22, the mean and eps 2 * 2^-24, two products; s itself is one addition (2^-24)."""
    return y.abs() * ((cols + 1) * 2.0 ** -25 + 2.0 ** -22 + 6 * 2.0 ** -24)


@pytest.mark.parametrize("shape", NORMS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("aligned", [True, False])
def test_rms_norm(cuda_device, shape, type, aligned):
    (rows, cols), dtype, half, eps = shape, TYPES[type], ref.half_step(TYPES[type]), 1e-6
    g = gen(rows, cols, type)
    for residual, weight, outs in ((True, True, "syq"), (False, True, "y"), (True, False, "q"), (False, False, "yq"), (True, True, "sq")):
        x = matrix(rows, cols, dtype, aligned).put((normal(g, rows, cols) * torch.exp(normal(g, cols))).to(dtype))
        r = matrix(rows, cols, dtype, aligned).put(normal(g, rows, cols).to(dtype)) if residual else None
        w = normal(g, cols + 1)[1:] if weight else None              # on 4 bytes
        s_out = matrix(rows, cols, dtype, aligned) if "s" in outs else None
        y_out = matrix(rows, cols, dtype, aligned) if "y" in outs else None
        q = Guarded(rows, cols, up(cols, 16) + 16, torch.float8_e4m3fn) if "q" in outs else None
        scales = Guarded(-(-cols // 128), rows, rows + 2, torch.float32) if q else None
        ok(sg.sgemm_rms_norm(rows, cols, type, x.ptr, x.ld, ptr(r), ld(r), w.data_ptr() if weight else 0, eps, ptr(s_out), ld(s_out),
                             ptr(y_out), ld(y_out), ptr(q), ld(q), ptr(scales), ld(scales), stream()))
        finish()
        s = x.view().double() + (r.view().double() if residual else 0.0)
        y = ref.rms_norm(s, w.double() if weight else None, eps)
        # Cancellation in x + residual is a rounding of s, which y follows.
        e = norm_error(s, y, cols)
        if s_out:
            assert s_out.outside_untouched()
            ref.close(s_out.view(), s, (half + 2.0 ** -24) * s.abs(), "sum")
        if y_out:
            assert y_out.outside_untouched()
            ref.close(y_out.view(), y, e + half * (y.abs() + e) + 2.0 ** -126, "y")
        if q:
            assert q.outside_untouched(8) and scales.outside_untouched()
            for b in range(-(-cols // 128)):
                c = slice(128 * b, min(cols, 128 * b + 128))
                most, rel = y[:, c].abs().amax(1), norm_error(s, torch.ones_like(y), cols).amax(1)
                a = most.clamp(min=2.0 ** -96)
                ref.close(scales.view()[b], a / 448.0, a / 448.0 * (rel + 2.0 ** -24), "scales")
                # A value over its scale is rounded to 4 bits (2^-4; below 2^-6 to multiples of 2^-9); the scale that
                # it was multiplied by and the one that it is held with differ by three roundings.
                got = q.view()[:, c].double() * scales.view()[b].double()[:, None]
                bound = (2.0 ** -4 + 4 * 2.0 ** -24) * (y[:, c].abs() + e[:, c]) + (a / 448.0)[:, None] * 2.0 ** -10 + e[:, c]
                ref.close(got, y[:, c], bound, "q")


@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cols", [300, 2048, 4099])
def test_rms_norm_in_place(cuda_device, type, cols):
    """The sum in the residual's place, y in x's."""
    dtype, rows = TYPES[type], 50
    g = gen(cols)
    x, r, w = normal(g, rows, cols).to(dtype), normal(g, rows, cols).to(dtype), normal(g, cols)
    args = lambda x, r, s, y: (rows, cols, type, x.data_ptr(), cols, r.data_ptr(), cols, w.data_ptr(), 1e-5, s.data_ptr(), cols,  # noqa: E731
                               y.data_ptr(), cols, 0, 0, 0, 0, stream())
    s, y = torch.empty_like(x), torch.empty_like(x)
    ok(sg.sgemm_rms_norm(*args(x, r, s, y)))
    x2, r2 = x.clone(), r.clone()
    ok(sg.sgemm_rms_norm(*args(x2, r2, r2, x2)))
    finish()
    assert torch.equal(s, r2) and torch.equal(y, x2)
    d, d2, gs = torch.empty_like(x), y.clone(), normal(g, rows, cols).to(dtype)
    back = lambda gy, gs, d: sg.sgemm_rms_norm_backward(rows, cols, type, gy.data_ptr(), cols, s.data_ptr(), cols, w.data_ptr(), 1e-5,  # noqa: E731
                                                        gs.data_ptr(), cols, d.data_ptr(), cols, 0, stream())
    ok(back(y, gs, d))
    ok(back(d2, gs, d2))
    d3 = gs.clone()
    ok(back(y, d3, d3))
    finish()
    assert torch.equal(d, d2) and torch.equal(d, d3)


def test_rms_norm_of_zeros_infinities_and_nan(cuda_device):
    cols = 384
    x = torch.ones(5, cols, device="cuda")
    x[0], x[1, 7], x[2, 9], x[3] = 0.0, NAN, float("inf"), 0.0
    y = torch.empty_like(x)
    q, scales = torch.zeros(5, cols, dtype=torch.uint8, device="cuda"), torch.zeros(3, 5, device="cuda")
    ok(sg.sgemm_rms_norm(5, cols, F32, x.data_ptr(), cols, 0, 0, 0, 1e-6, 0, 0, y.data_ptr(), cols, q.data_ptr(), cols, scales.data_ptr(),
                         5, stream()))
    finish()
    assert bool((y[0] == 0).all()) and bool((q[0] == 0).all()) and bool((scales[:, 0] == 2.0 ** -96 / 448).all())
    assert bool(torch.isnan(y[1]).all()) and bool((q[1] & 0x7F == 0x7F).all())
    # 1 / sqrt(inf) = 0: zeros, and NaN where the infinity was.
    assert bool(torch.isnan(y[2, 9])) and bool((y[2, :9] == 0).all()) and bool((y[2, 10:] == 0).all())
    assert bool(torch.isnan(scales[0, 2])) and bool((scales[1:, 2] == 2.0 ** -96 / 448).all())
    assert bool((y[4] - 1).abs().max() < 1e-5)


@pytest.mark.parametrize("shape", NORMS + [(2000, 300), (1300, 2048)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("type", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("aligned", [True, False])
def test_rms_norm_backward(cuda_device, shape, type, aligned):
    (rows, cols), dtype, half, eps = shape, TYPES[type], ref.half_step(TYPES[type]), 1e-6
    g = gen(rows, cols, type)
    for stream_grad, weight, want_w in ((True, True, True), (False, False, True), (True, True, False)):
        put = lambda v: matrix(rows, cols, dtype, aligned).put(v.to(dtype))  # noqa: E731
        s, gy = put(normal(g, rows, cols) * torch.exp(normal(g, cols))), put(normal(g, rows, cols))
        gs = put(normal(g, rows, cols)) if stream_grad else None
        w = normal(g, cols) if weight else None
        d, dw = matrix(rows, cols, dtype, aligned), Guarded(1, cols, cols, torch.float32)
        ok(sg.sgemm_rms_norm_backward(rows, cols, type, gy.ptr, gy.ld, s.ptr, s.ld, w.data_ptr() if weight else 0, eps, ptr(gs), ld(gs),
                                      d.ptr, d.ld, dw.ptr if want_w else 0, stream()))
        finish()
        S, G, W = s.view().double(), gy.view().double(), w.double() if weight else None
        want, want_dw = ref.rms_norm_backward(G, S, W, eps, gs.view().double() if stream_grad else None)
        # h and g w have relative errors r; their mean's is cols 2^-24 more, of the sum of magnitudes.
        r = (cols + 1) * 2.0 ** -25 + 2.0 ** -22 + 6 * 2.0 ** -24
        i = 1.0 / torch.sqrt((S * S).mean(1, keepdim=True) + eps)
        h, gw = S * i, G * (W if weight else 1.0)
        mean = (gw * h).abs().mean(1, keepdim=True)
        e = i * (gw.abs() + h.abs() * mean) * (4 * r + (cols + 4) * 2.0 ** -24)
        if stream_grad:
            e = e + 2.0 ** -24 * (want.abs() + e)
        ref.close(d.view(), want, e + half * (want.abs() + e) + 2.0 ** -126, "d")
        assert d.outside_untouched() and dw.outside_untouched()
        if want_w:
            ref.close(dw.view()[0], want_dw, (G * h).abs().sum(0) * (r + (rows + 2) * 2.0 ** -24) + 2.0 ** -126, "dw")


def test_rms_norm_backward_against_differences(cuda_device):
    """Directional differences of the forward pass in FP32: with a step t the error is t^2 times a third derivative (of
    order 1 for rows of unit size) and the rounding of the two sums, 2^-20 / t; t = 2^-7 keeps both below 2e-3."""
    rows, cols, t = 16, 200, 2.0 ** -7
    g = gen(5)
    x, v, gy, w = normal(g, rows, cols), normal(g, rows, cols), normal(g, rows, cols), normal(g, cols)
    def f(x):
        y = torch.empty_like(x)
        ok(sg.sgemm_rms_norm(rows, cols, F32, x.data_ptr(), cols, 0, 0, w.data_ptr(), 1e-6, 0, 0, y.data_ptr(), cols, 0, 0, 0, 0, stream()))
        return (y.double() * gy.double()).sum(1)
    d = torch.empty_like(x)
    ok(sg.sgemm_rms_norm_backward(rows, cols, F32, gy.data_ptr(), cols, x.data_ptr(), cols, w.data_ptr(), 1e-6, 0, 0, d.data_ptr(), cols,
                                  0, stream()))
    finish()
    u = v / v.norm(dim=1, keepdim=True)
    want = (f(x + t * u) - f(x - t * u)) / (2 * t)
    assert bool(((d.double() * u.double()).sum(1) - want).abs().max() <= 2e-3 * gy.norm(dim=1).max())


def test_no_rows_give_a_weight_gradient_of_zeros(cuda_device):
    dw = torch.full((70,), 5.0, device="cuda")
    ok(sg.sgemm_rms_norm_backward(0, 70, F32, 0, 70, 0, 70, 0, 1e-6, 0, 0, 0, 70, dw.data_ptr(), stream()))
    finish()
    assert bool((dw == 0).all())


# ------------------------------------------------- streams, graphs, same bits


def block(x, r, w, W1, W2, b1, bufs, st):
    """A norm, a gated product and a product that adds the residual, with the gradients of the second."""
    T, D = x.shape
    F = W1.shape[0]
    s, y, h, z, out, dh, dz, dW, db, dn, dw = bufs
    no = (0, 0)
    return [
        sg.sgemm_rms_norm(T, D, BF16, x.data_ptr(), D, r.data_ptr(), D, w.data_ptr(), 1e-6, s.data_ptr(), D, y.data_ptr(), D, 0, 0, 0, 0, st),
        sg.sgemm_bf16(0, 1, T, F, D, y.data_ptr(), D, W1.data_ptr(), D, b1.data_ptr(), 4, z.data_ptr(), F, 0, *no, h.data_ptr(), BF16, F, st),
        sg.sgemm_bf16(0, 1, T, D, F, h.data_ptr(), F, W2.data_ptr(), F, 0, 0, *no, 1, s.data_ptr(), D, out.data_ptr(), BF16, D, st),
        sg.sgemm_bf16(0, 0, T, F, D, x.data_ptr(), D, W2.data_ptr(), F, 0, 0, *no, 0, *no, dh.data_ptr(), BF16, F, st),
        sg.sgemm_epilogue_backward(T, F, BF16, dh.data_ptr(), F, z.data_ptr(), F, 4, 0, *no, 1, 0, dz.data_ptr(), F, *no, db.data_ptr(), F, st),
        sg.sgemm_bf16(1, 0, F, D, T, dz.data_ptr(), F, y.data_ptr(), D, 0, 0, *no, 0, *no, dW.data_ptr(), F32, D, st),
        sg.sgemm_rms_norm_backward(T, D, BF16, x.data_ptr(), D, s.data_ptr(), D, w.data_ptr(), 1e-6, r.data_ptr(), D, dn.data_ptr(), D,
                                   dw.data_ptr(), st),
    ]


def block_inputs(seed, T=300, D=256, F=512):
    g = gen(seed)
    x, r = normal(g, T, D).bfloat16(), normal(g, T, D).bfloat16()
    W1, W2 = (normal(g, F, D) / 16).bfloat16(), (normal(g, D, F) / 22).bfloat16()
    return x, r, normal(g, D), W1, W2, normal(g, F)


def block_outputs(T=300, D=256, F=512):
    b = lambda *s: torch.full(s, NAN, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    f = lambda *s: torch.full(s, NAN, device="cuda")  # noqa: E731
    return b(T, D), b(T, D), b(T, F), b(T, F), b(T, D), b(T, F), b(T, F), f(F, D), f(F), b(T, D), f(D)


def test_captured_concurrent_and_repeated_calls_give_the_same_bits(cuda_device):
    inputs, outs = [block_inputs(i) for i in range(3)], [block_outputs() for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):                                   # side by side
        for i, o, s in zip(inputs, outs, streams):
            assert block(*i, o, s.cuda_stream) == [sg.SGEMM_OK] * 7
    finish()
    for i, o in zip(inputs, outs):                       # alone
        alone = block_outputs()
        assert block(*i, alone, stream()) == [sg.SGEMM_OK] * 7
        finish()
        assert all(torch.equal(a, b) for a, b in zip(alone, o))
    graphs, captured = [], [block_outputs() for _ in range(2)]
    for i, o, s in zip(inputs, captured, streams):       # two graphs that share the library's pool
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            assert block(*i, o, torch.cuda.current_stream().cuda_stream) == [sg.SGEMM_OK] * 7
        graphs.append(graph)
    for _ in range(3):
        for o in captured:
            for t in o:
                t.fill_(NAN)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, want in zip(captured, outs):
            assert all(torch.equal(a, b) for a, b in zip(o, want))
    assert sg.sgemm_check_status(stream()) == sg.SGEMM_OK


def test_norm_feeds_the_8_bit_product(cuda_device):
    """The norm's 8-bit rows times weights in blocks: within the two quantisations (2^-4 each, relative) of y . w^T."""
    T, D, N = 50, 384, 256
    g = gen(1)
    x, w, W = normal(g, T, D).bfloat16(), normal(g, D), normal(g, N, D)
    q, sc = torch.empty(T, D, dtype=torch.uint8, device="cuda"), torch.empty(3, T, device="cuda")
    qw, sw = torch.empty(N, D, dtype=torch.uint8, device="cuda"), torch.empty(2, 3, device="cuda")
    C = torch.empty(T, N, device="cuda")
    ok(sg.sgemm_rms_norm(T, D, BF16, x.data_ptr(), D, 0, 0, w.data_ptr(), 1e-6, 0, 0, 0, 0, q.data_ptr(), D, sc.data_ptr(), T, stream()))
    ok(sg.sgemm_fp8_quantize_blocks(N, D, W.data_ptr(), F32, D, 0, 0, qw.data_ptr(), D, 0, sw.data_ptr(), 3, 0, 1, stream()))
    ok(sg.sgemm_fp8(sg.SGEMM_SCALE_BLOCKS, T, N, D, q.data_ptr(), D, sc.data_ptr(), T, qw.data_ptr(), D, sw.data_ptr(), 3, 0.0, C.data_ptr(),
                    F32, N, stream()))
    finish()
    y = ref.rms_norm(x.double(), w.double(), 1e-6)
    want, S = ref.product(y, W.double().t())
    half = 2.0 ** -4 + 2.0 ** -10                       # a rounding, and what the smallest values of a block lose
    ref.close(C, want, S * (2 * half + half * half + 1e-4) + y.abs().amax() * W.abs().amax() * D * 2.0 ** -9 / 100)
