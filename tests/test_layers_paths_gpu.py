"""Which kernel a call of the 16-bit products takes, and that each gives the
same whole numbers: pairs of CTAs with and without a joined matrix in 16-byte
pieces, tiles cut for the last wave, parts of a long K, groups spread evenly,
rows far apart. Small whole numbers are exact in bfloat16 and their sums in
FP32, so results are compared bit by bit (after one rounding to C's type)."""

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
from test_experts_gpu import Guarded, finish, ok, stream
from test_layers_gpu import BF16, F32, TYPES, gen, ld, matrix, offsets_of, operand, ptr, up

pytestmark = pytest.mark.gpu

NONE, ADD, MUL = sg.SGEMM_JOIN_NONE, sg.SGEMM_JOIN_ADD, sg.SGEMM_JOIN_MUL


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def plan(mode, groups, M, N, K):
    rc, cols, pair, swap, split, grid = sg.sgemm_bf16_plan(mode, groups, M, N, K, sms())
    assert rc == sg.SGEMM_OK
    return cols, pair, swap, split, grid


def whole(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").double()


def joined(z, join, d):
    return z + d if join == ADD else z * d if join == MUL else z


def dense(M, N, K, ctype, join, aligned, ops=(0, 1), in_place=False):
    g = gen(M, N, K, join)
    a, b, bias = whole(g, M, K), whole(g, K, N), whole(g, N)
    A, lda = operand((a.t() if ops[0] else a).bfloat16())
    B, ldb = operand((b.t() if ops[1] else b).bfloat16())
    dtype = TYPES[ctype]
    C, pre = matrix(M, N, dtype, aligned), matrix(M, N, dtype, aligned)
    d = whole(g, M, N).to(dtype)
    D = None if join == NONE else C.put(d) if in_place else matrix(M, N, dtype, aligned).put(d)
    if in_place:
        C.start = C.flat.clone()
    bias32 = bias.float()
    ok(sg.sgemm_bf16(*ops, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, bias32.data_ptr(), sg.SGEMM_ACT_RELU, pre.ptr, pre.ld,
                     join, ptr(D), ld(D), C.ptr, ctype, C.ld, stream()))
    finish()
    z = a @ b + bias
    assert torch.equal(pre.view(), z.to(dtype))
    assert torch.equal(C.view(), joined(z.clamp(min=0), join, d.double()).to(dtype))
    assert C.outside_untouched() and pre.outside_untouched()


@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("join", [NONE, ADD, MUL], ids=["none", "add", "mul"])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
@pytest.mark.parametrize("shape,kind", [((900, 4100, 136), (256, 1)), ((500, 4100, 136), (256, 1)), ((1030, 2061, 1700), (256, 1)),
                                        ((400, 2061, 1700), (128, 1)), ((260, 2061, 1700), (128, 1))], ids=str)
def test_pairs(cuda_device, ctype, join, aligned, shape, kind):
    assert plan(sg.SGEMM_BF16_DENSE, 1, *shape)[:2] == kind
    dense(*shape, ctype, join, aligned)
    if join != NONE:
        dense(*shape, ctype, join, aligned, in_place=True)


@pytest.mark.parametrize("ops", [(0, 1), (0, 0), (1, 0), (1, 1)], ids=lambda o: "op%d%d" % o)
@pytest.mark.parametrize("tiles", [(24, 4), (13, 7), (10, 8), (19, 8), (9, 9)], ids=str)
def test_tiles_cut_for_the_last_wave(cuda_device, ops, tiles):
    """76 pairs of SMs: 96 tiles leave 20 (two pieces each), 91 leave 15 (four), 80 leave 4 (four), 152 none, 81 five."""
    M, N = 256 * tiles[0] - 3, 256 * tiles[1] - 40
    assert plan(sg.SGEMM_BF16_DENSE, 1, M, N, 200)[:2] == (256, 1)
    dense(M, N, 200, BF16, NONE, True, ops)
    dense(M, N, 100, F32, ADD, False, ops)


@pytest.mark.parametrize("K", [768, 769, 1536, 2000, 6000])
@pytest.mark.parametrize("shape", [(20, 300), (300, 500), (900, 4100)], ids=str)
def test_parts_of_a_long_k(cuda_device, K, shape):
    dense(*shape, K, F32, ADD, True)


@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("join", [NONE, ADD, MUL], ids=["none", "add", "mul"])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
@pytest.mark.parametrize("counts", [[2600, 0, 1257, 900, 1, 33], [400] * 12, [6000, 3], [5000]], ids=lambda c: "-".join(map(str, c[:6])))
def test_groups_of_rows_by_pairs(cuda_device, ctype, join, aligned, counts):
    E, R, N, K, dtype = len(counts), sum(counts) + 5, 1100, 200, TYPES[ctype]
    assert plan(sg.SGEMM_BF16_GROUPED, E, R, N, K)[1] == 1
    g = gen(E, R, join)
    o, off = offsets_of(counts, 2)
    a, b, bias, d = whole(g, R, K), whole(g, E, N, K), whole(g, E, N), whole(g, R, N)
    a[:2], a[R - 3:] = float("nan"), float("nan")
    A, lda = operand(a.bfloat16())
    B, ldb = operand(b.bfloat16())
    C, bias32 = matrix(R, N, dtype, aligned), bias.float()
    D = None if join == NONE else matrix(R, N, dtype, aligned).put(d.to(dtype))
    ok(sg.sgemm_bf16_grouped(1, E, off.data_ptr(), R, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, B.stride(0), bias32.data_ptr(), N,
                             sg.SGEMM_ACT_RELU, 0, 0, join, ptr(D), ld(D), C.ptr, ctype, C.ld, stream()))
    finish()
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        z = (a[rows] @ b[e].t() + bias[e]).clamp(min=0)
        assert torch.equal(C.view()[rows], joined(z, join, d[rows]).to(dtype)), e
    assert C.outside_untouched() and bool((C.view()[:2] == C.fill).all()) and bool((C.view()[R - 3:] == C.fill).all())


# 152 SMs: 64 tiles of 256 x 256 per group on 76 pairs, and others around a wave; odd lengths along K.
@pytest.mark.parametrize("ctype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("E,M,N", [(9, 2048, 2048), (5, 2560, 2048), (30, 1000, 1100), (3, 2300, 2500), (140, 600, 520)], ids=str)
def test_groups_along_k_spread_evenly(cuda_device, ctype, accumulate, E, M, N):
    g = gen(E, M, N)
    counts = torch.randint(0, 90, (E,), generator=g, device="cuda").tolist()
    counts[1], counts[2] = 0, 64
    R, dtype = sum(counts) + 3, TYPES[ctype]
    o, off = offsets_of(counts, 1)
    a, b, c = whole(g, R, M), whole(g, R, N), whole(g, E, M, N).to(dtype)
    a[0], b[R - 2:] = float("nan"), float("inf")
    A, lda = operand(a.bfloat16())
    B, ldb = operand(b.bfloat16())
    C = c.clone()
    ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), R, M, N, A.data_ptr(), lda, B.data_ptr(), ldb, accumulate, C.data_ptr(), ctype, N,
                               M * N, stream()))
    finish()
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        z = a[rows].t() @ b[rows]
        assert torch.equal(C[e], (z + c[e].double() if accumulate else z).to(dtype)), e


def test_an_empty_group_added_to_stays_as_it_was(cuda_device):
    """In every bit, negative zeros and NaN among them; a single row with any leading dimension."""
    E, M, N = 3, 300, 264
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[2:] = 5
    g = gen(1)
    a, b = whole(g, 5, M).bfloat16(), whole(g, 5, N).bfloat16()
    A, lda = operand(a)
    B, ldb = operand(b)
    C = torch.full((E, M, N), -0.0, device="cuda")
    C[0, 3, 4] = float("nan")
    was = C.clone()
    ok(sg.sgemm_bf16_grouped_k(E, off.data_ptr(), 5, M, N, A.data_ptr(), lda, B.data_ptr(), ldb, 1, C.data_ptr(), F32, N, M * N, stream()))
    finish()
    for e in (0, 2):
        assert torch.equal(C[e].view(torch.int32), was[e].view(torch.int32))
    assert torch.equal(C[1].double(), a.double().t() @ b.double())
    out = torch.full((1, N), 5.0, device="cuda")
    W, ldw = operand(whole(g, N, M).bfloat16())
    ok(sg.sgemm_bf16(0, 1, 1, N, M, A.data_ptr(), 2 ** 50, W.data_ptr(), ldw, 0, 0, 0, 0, 0, 0, 0, out.data_ptr(), F32, 2 ** 50, stream()))
    finish()
    assert torch.equal(out.double(), a[:1].double() @ W[:, :M].double().t())


def far(rows, cols, apart, dtype):
    """A matrix whose rows are `apart` elements from each other (its memory is not touched in between)."""
    buf = torch.empty((rows - 1) * apart + cols, dtype=dtype, device="cuda")
    return buf, torch.as_strided(buf, (rows, cols), (apart, 1))


@pytest.mark.parametrize("M", [5, 130])
def test_offsets_past_32_bits(cuda_device, M):
    N, K = 200, 72
    apart = 2 ** 30 + 8 if M == 5 else 2 ** 25 + 8        # times rows: over 2^32 elements
    g = gen(M)
    a, b, d = whole(g, M, K), whole(g, N, K), whole(g, M, N)
    bufs, views = zip(*(far(M, c, apart, t) for c, t in ((K, torch.bfloat16), (N, torch.bfloat16), (N, torch.bfloat16), (N, torch.bfloat16))))
    A, C, pre, D = views
    A.copy_(a)
    D.copy_(d)
    B = b.bfloat16()
    ok(sg.sgemm_bf16(0, 1, M, N, K, A.data_ptr(), apart, B.data_ptr(), K, 0, sg.SGEMM_ACT_RELU, pre.data_ptr(), apart, MUL, D.data_ptr(),
                     apart, C.data_ptr(), BF16, apart, stream()))
    finish()
    z = a @ b.t()
    assert torch.equal(pre, z.bfloat16()) and torch.equal(C, (z.clamp(min=0) * d).bfloat16())
    # The gradients, and the norm, of the same rows.
    dz, dD, db = C, pre.clone(), torch.empty(N, device="cuda")
    ok(sg.sgemm_epilogue_backward(M, N, BF16, D.data_ptr(), apart, pre.data_ptr(), apart, sg.SGEMM_ACT_RELU, MUL, D.data_ptr(), apart, 1, 0,
                                  dz.data_ptr(), apart, dD.data_ptr(), N, db.data_ptr(), N, stream()))
    ok(sg.sgemm_rms_norm(M, N, BF16, D.data_ptr(), apart, 0, 0, 0, 1e-6, 0, 0, pre.data_ptr(), apart, 0, 0, 0, 0, stream()))
    finish()
    on = (z.bfloat16().double() > 0).double()
    assert torch.equal(dz, (d * d * on).bfloat16()) and torch.equal(db, (d * d * on).sum(0).float())
    want = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6)
    assert bool(((pre.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all())


def test_rows_of_the_largest_norm(cuda_device):
    """16384 columns, and one less: rows of every layout in both types, forward and backward."""
    rows = 3
    for cols in (16384, 16383):
        for type, dtype in TYPES.items():
            g = gen(cols, type)
            x, gy = (torch.randn(rows, cols, generator=g, device="cuda").to(dtype) for _ in range(2))
            w = torch.randn(cols, generator=g, device="cuda")
            results = []
            for apart, shift in ((up(cols, 8), 0), (cols, 1), (cols + 5, 3)):
                m = [torch.empty(rows * apart + 8, dtype=dtype, device="cuda")[shift:] for _ in range(4)]
                v = [t[:rows * apart].view(rows, apart)[:, :cols] for t in m]
                v[0].copy_(x)
                v[1].copy_(gy)
                dw = torch.empty(cols, device="cuda")
                ok(sg.sgemm_rms_norm(rows, cols, type, v[0].data_ptr(), apart, 0, 0, w.data_ptr(), 1e-6, 0, 0, v[2].data_ptr(), apart, 0, 0, 0,
                                     0, stream()))
                ok(sg.sgemm_rms_norm_backward(rows, cols, type, v[1].data_ptr(), apart, v[0].data_ptr(), apart, w.data_ptr(), 1e-6, 0, 0,
                                              v[3].data_ptr(), apart, dw.data_ptr(), stream()))
                finish()
                results.append((v[2].double(), v[3].double(), dw.double()))
            X, G, W = x.double(), gy.double(), w.double()
            i = 1 / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-6)
            h = X * i
            wants = (h * W, i * (G * W - h * (G * W * h).mean(1, keepdim=True)), (G * h).sum(0))
            for got in results:
                for a, b, t in zip(got, wants, (dtype, dtype, torch.float32)):
                    # A rounding to the type, and 16384 of FP32's in the sums at most.
                    assert float((a - b).norm()) <= (torch.finfo(t).eps / 2 + 16384 * 2.0 ** -24) * float(b.norm())
