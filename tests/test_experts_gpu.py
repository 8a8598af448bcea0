"""GPU parity of the operators around products over experts against plain
restatements in 64 bits (experts_ref), at the sizes, masks, strides and
alignments where they can go wrong.

Tolerances. Product: experts_ref.product_tolerance() times sum |a b|; results
in bfloat16 also half an ulp of 2^-8 (one rounding). Products of small integers
with power-of-two scales are exact. The quantiser is exact in every bit.
Router weights: an exponential (2 ulp), a sum of E terms in any order and two
divisions: (E / 2 + 8) 2^-23 relative. Combining sums: k roundings of the terms'
magnitudes; dot products of n terms: n 2^-24 times sum |a b| bounds any order.
"""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
import experts_ref as ref

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
TYPES = {sg.SGEMM_F32: torch.float32, sg.SGEMM_BF16: torch.bfloat16}
GUARD = 64


def stream():
    return torch.cuda.current_stream().cuda_stream


def ok(rc):
    assert rc == sg.SGEMM_OK, sg.sgemm_error_string(rc)


def finish():
    torch.cuda.synchronize()
    assert sg.sgemm_check_status(stream()) == sg.SGEMM_OK


class Guarded:
    """A rows x cols device matrix with leading dimension ld, `shift` elements into its buffer, filled with `fill`
    and surrounded by it."""

    def __init__(self, rows, cols, ld, dtype, shift=0, fill=77.0):
        self.rows, self.cols, self.ld, self.shift, self.fill = rows, cols, ld, shift, fill
        self.flat = torch.empty(GUARD + shift + rows * ld + GUARD, dtype=dtype, device="cuda")
        if dtype == FP8:
            self.flat.view(torch.uint8).fill_(0x77)
        else:
            self.flat.fill_(fill)
        self.start = self.flat.clone()

    @property
    def ptr(self):
        return self.flat.data_ptr() + (GUARD + self.shift) * self.flat.element_size()

    def view(self):
        at = GUARD + self.shift
        return self.flat[at:at + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols]

    def put(self, x):
        self.view().copy_(x)
        return self

    def outside_untouched(self, pad=0):
        """Everything but the matrix (and up to `pad` elements after each row) is as it was."""
        a, b = self.flat.clone(), self.start
        at = GUARD + self.shift
        keep = min(self.ld, self.cols + pad)
        a[at:at + self.rows * self.ld].view(self.rows, self.ld)[:, :keep] = \
            b[at:at + self.rows * self.ld].view(self.rows, self.ld)[:, :keep]
        if a.dtype == FP8:
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        return bool((a == b).all())


def fp8_operand(q, ld=None):
    """q (rows x K float8 CPU tensor) on the device with rows of ld bytes; NaN bytes between and after them."""
    rows, K = q.shape
    ld = ref.up(K, 16) if ld is None else ld
    buf = torch.full((rows * ld + 256,), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:rows * ld].view(rows, ld)[:, :K] = q.view(torch.uint8).cuda()
    return buf, ld


def scales_operand(s, ld=None):
    """s (float32 CPU matrix) on the device with NaN in the padding."""
    rows, cols = s.shape
    ld = cols if ld is None else ld
    buf = torch.full((rows * ld,), float("nan"), device="cuda")
    buf.view(rows, ld)[:, :cols] = s.cuda()
    return buf, ld


def check_product(C, want, S, nk, bf16, old=None):
    C = C.double().cpu()
    tol = ref.product_tolerance(nk) * S + 1e-300
    if bf16:
        tol = tol + want.abs() * 2.0 ** -8
    bad = (C - want).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), C[bad][0].item(), want[bad][0].item())


# ------------------------------------------------------------------ products

# M, N, K around every tile edge (16, 32, 64, 128 columns, 128 and 256 rows), K tails, split K, several waves.
SHAPES = [(1, 1, 1), (1, 129, 16), (3, 257, 127), (16, 128, 129), (17, 4096, 1024), (33, 640, 513), (64, 1024, 2048),
          (65, 384, 256), (127, 130, 385), (128, 256, 128), (129, 255, 300), (300, 511, 1000), (1000, 777, 640),
          (2500, 1200, 272), (8, 7000, 4096), (3000, 1700, 400), (5121, 1025, 1296)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("form", [sg.SGEMM_SCALE_BLOCKS, sg.SGEMM_SCALE_ROWS], ids=["blocks", "rows"])
@pytest.mark.parametrize("ctype", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
def test_product(cuda_device, shape, form, ctype):
    M, N, K = shape
    g = torch.Generator().manual_seed(M * 31 + N * 7 + K)
    nk = -(-K // 128)
    qa, sa = ref.quantize_rows_fast(torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g)))
    qb, sb = ref.quantize_rows_fast(torch.randn(N, K, generator=g))
    a = ref.wide_rows(qa, sa.t())
    if form == sg.SGEMM_SCALE_BLOCKS:
        sb = torch.rand(-(-N // 128), nk, generator=g) + 0.1
        b = ref.wide_blocks(qb, sb)
    else:
        b = ref.wide_rows(qb, sb.t())
        sb = sb.t().contiguous()
    want, S = ref.product(a, b)
    dA, lda = fp8_operand(qa)
    dB, ldb = fp8_operand(qb, ref.up(K, 16) + 16)
    dsa, ld_sa = scales_operand(sa.t().contiguous(), M + 3)
    dsb, ld_sb = scales_operand(sb, sb.shape[1] + 1)
    # An odd leading dimension and base: the scalar stores; 16-byte rows: the vector ones.
    for ldc, shift in ((N + 5, 1), (ref.up(N, 8), 0)):
        C = Guarded(M, N, ldc, TYPES[ctype], shift, fill=float("nan"))
        C.flat.view(torch.uint8).fill_(0x55)
        C.start = C.flat.clone()
        ok(sg.sgemm_fp8(form, M, N, K, dA.data_ptr(), lda, dsa.data_ptr(), ld_sa, dB.data_ptr(), ldb, dsb.data_ptr(),
                        ld_sb, 0.0, C.ptr, ctype, ldc, stream()))
        finish()
        check_product(C.view(), want, S, nk, ctype == sg.SGEMM_BF16)
        assert C.outside_untouched()


@pytest.mark.parametrize("M", [1, 20, 40, 100, 130, 1100, 5100])
@pytest.mark.parametrize("form", [sg.SGEMM_SCALE_BLOCKS, sg.SGEMM_SCALE_ROWS], ids=["blocks", "rows"])
def test_integer_products_are_exact(cuda_device, M, form):
    N, K = 777, 1300
    g = torch.Generator().manual_seed(M)
    qa = torch.randint(-8, 9, (M, K), generator=g).float().to(FP8)
    qb = torch.randint(-8, 9, (N, K), generator=g).float().to(FP8)
    nk = -(-K // 128)
    sa = 2.0 ** torch.randint(0, 2, (nk, M), generator=g).float()
    sb = 2.0 ** torch.randint(0, 2, (nk, N) if form == sg.SGEMM_SCALE_ROWS else (-(-N // 128), nk), generator=g).float()
    b = ref.wide_rows(qb, sb) if form == sg.SGEMM_SCALE_ROWS else ref.wide_blocks(qb, sb)
    want, _ = ref.product(ref.wide_rows(qa, sa), b)   # below 64 * 4 * 1300 < 2^24
    dA, lda = fp8_operand(qa)
    dB, ldb = fp8_operand(qb)
    dsa, dsb = sa.cuda(), sb.cuda()
    C = torch.full((M, N), float("nan"), device="cuda")
    old = torch.randint(-9, 10, (M, N), generator=g).float()
    for beta in (0.0, 2.0):
        if beta:
            C.copy_(old)
        ok(sg.sgemm_fp8(form, M, N, K, dA.data_ptr(), lda, dsa.data_ptr(), M, dB.data_ptr(), ldb, dsb.data_ptr(),
                        sb.shape[1], beta, C.data_ptr(), sg.SGEMM_F32, N, stream()))
        finish()
        assert torch.equal(C.cpu().double(), want + beta * old.double())


def test_product_of_nothing_scales_c(cuda_device):
    for M in (5, 200):
        C = torch.full((M, 40), 3.0, device="cuda")
        ok(sg.sgemm_fp8(0, M, 40, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.5, C.data_ptr(), sg.SGEMM_F32, 40, stream()))
        finish()
        assert bool((C == 1.5).all())
        ok(sg.sgemm_fp8(0, M, 40, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0.0, C.data_ptr(), sg.SGEMM_F32, 40, stream()))
        finish()
        assert bool((C == 0).all())


def test_nan_stays_in_its_rows_and_columns(cuda_device):
    for M in (20, 300):
        N, K = 300, 384
        g = torch.Generator().manual_seed(1)
        qa, sa = ref.quantize_rows_fast(torch.randn(M, K, generator=g))
        qb, _ = ref.quantize_rows_fast(torch.randn(N, K, generator=g))
        sb = torch.ones(3, 3)
        qa.view(torch.uint8)[7, 200] = 0x7F
        sa[11, 2] = float("inf")
        qb.view(torch.uint8)[5, 3] = 0x7F
        dA, lda = fp8_operand(qa)
        dB, ldb = fp8_operand(qb)
        C = torch.zeros(M, N, device="cuda")
        ok(sg.sgemm_fp8(0, M, N, K, dA.data_ptr(), lda, sa.t().contiguous().cuda().data_ptr(), M, dB.data_ptr(), ldb,
                        sb.cuda().data_ptr(), 3, 0.0, C.data_ptr(), sg.SGEMM_F32, N, stream()))
        finish()
        c = C.cpu()
        assert bool(c[7].isnan().all()) and bool(c[:, 5].isnan().all()) and not bool(c[11].isfinite().any())
        rest = c.clone()
        rest[7], rest[11], rest[:, 5] = 0, 0, 0
        assert bool(rest.isfinite().all())


# ---------------------------------------------------------- grouped products

COUNTS = {
    "decode": [1, 0, 3, 2, 0, 0, 1, 5],
    "edges": [16, 17, 15, 0, 1, 32, 33, 64],
    "one_heavy": [0, 0, 500, 0],
    "ragged": [127, 129, 0, 300, 1, 128],
    "none": [0, 0, 0],
    "many": [3, 0, 1, 2] * 100,
    "prompts": [700, 0, 257, 1300, 256, 3],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("ctype", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("NK", [(200, 144), (512, 700), (2200, 272)], ids=["200x144", "512x700", "2200x272"])
def test_grouped(cuda_device, name, ctype, NK):
    (N, K), counts = NK, COUNTS[name]
    E, R = len(counts), sum(counts) + 5               # five rows that no group has
    g = torch.Generator().manual_seed(len(name))
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    qa, sa = ref.quantize_rows_fast(torch.randn(R, K, generator=g))
    qb = torch.randn(E, N, K, generator=g).clamp(-6, 6).to(FP8)
    nk, nb = -(-K // 128), -(-N // 128)
    sb = torch.rand(E, nb, nk, generator=g) + 0.2
    ld = ref.up(K, 16)
    dB = torch.full((E, N, ld), 0x7F, dtype=torch.uint8, device="cuda")
    dB[:, :, :K] = qb.view(torch.uint8).cuda()
    dA, lda = fp8_operand(qa)
    dsa, dsb = sa.t().contiguous().cuda(), sb.cuda()
    C = Guarded(R, N, N + 3, TYPES[ctype])
    ok(sg.sgemm_fp8_grouped(E, off.cuda().data_ptr(), R, N, K, dA.data_ptr(), lda, dsa.data_ptr(), R, dB.data_ptr(), ld,
                            N * ld, dsb.data_ptr(), nk, nb * nk, 0.0, C.ptr, ctype, N + 3, stream()))
    finish()
    a = ref.wide_rows(qa, sa.t())
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            want, S = ref.product(a[lo:hi], ref.wide_blocks(qb[e], sb[e]))
            check_product(C.view()[lo:hi], want, S, nk, ctype == sg.SGEMM_BF16)
    assert bool((C.view()[int(off[-1]):] == 77.0).all()), "rows of no group were written"
    assert C.outside_untouched()


@pytest.mark.parametrize("name", ["decode", "ragged", "one_heavy", "none", "prompts"])
@pytest.mark.parametrize("MN", [(130, 100), (384, 512), (1000, 1100)], ids=["130x100", "384x512", "1000x1100"])
def test_grouped_k(cuda_device, name, MN):
    """The weight gradients, from the tokens on: the quantiser's layout and the product together."""
    (M, N), counts = MN, COUNTS[name]
    E, R = len(counts), sum(counts)
    g = torch.Generator().manual_seed(M)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    padded = ref.up(R + 127 * min(R, E), 128)
    # Integers of magnitude 448 at most in every block: scale 1, no rounding, exact sums.
    def tokens(cols):
        x = torch.randint(-3, 4, (R, cols), generator=g).float()
        return x
    dy, x = tokens(M), tokens(N)
    out = {}
    for key, t, cols in (("a", dy, M), ("b", x, N)):
        q = torch.zeros(cols, max(padded, 16), dtype=FP8, device="cuda")
        s = torch.zeros(max(padded, 128) // 128, cols, device="cuda")
        ok(sg.sgemm_fp8_quantize_cols(R, cols, t.cuda().data_ptr(), sg.SGEMM_F32, cols, 0, R, E, off.data_ptr(), padded,
                                      q.data_ptr(), max(padded, 16), s.data_ptr(), cols, stream()))
        out[key] = (q, s)
    C = torch.full((E, M, N), 5.0, device="cuda")
    ld = max(padded, 16)
    for beta in (0.0, 1.0):
        ok(sg.sgemm_fp8_grouped_k(E, off.data_ptr(), padded, M, N, out["a"][0].data_ptr(), ld, out["a"][1].data_ptr(), M,
                                  out["b"][0].data_ptr(), ld, out["b"][1].data_ptr(), N, beta, C.data_ptr(),
                                  sg.SGEMM_F32, N, M * N, stream()))
        finish()
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            a, b = dy[lo:hi].t().double(), x[lo:hi].t().double()
            want, S = a @ b.t(), a.abs() @ b.abs().t()
            # Each value is off by at most 2^-4 of itself (e4m3 keeps 4 significant bits), both by 2^-3 + 2^-8.
            err = (C[e].cpu().double() - want * (1 + beta)).abs()
            assert bool((err <= (1 + beta) * (0.13 * S + 1e-6)).all()), (e, float(err.max()))
            qa = ref.wide_rows(out["a"][0].cpu().view(torch.uint8).view(FP8), out["a"][1].cpu())
            qb = ref.wide_rows(out["b"][0].cpu().view(torch.uint8).view(FP8), out["b"][1].cpu())
            k0 = sum(ref.up(c, 128) for c in counts[:e])
            ka, kb = qa[:, k0:k0 + hi - lo], qb[:, k0:k0 + hi - lo]
            want, S = ka @ kb.t(), ka.abs() @ kb.abs().t()
            check_product(C[e], want * (1 + beta), S * (1 + beta) + 1e-30, padded // 128 + 2, False)


def small_integers(rows, cols, generator):
    return torch.randint(-3, 4, (rows, cols), generator=generator, device="cuda").float().to(FP8)


def powers_of_two(rows, cols, generator):
    return 2.0 ** torch.randint(0, 2, (rows, cols), generator=generator, device="cuda").float()


def spread(s, cols, rows=1):
    """Scales of blocks of `rows` x 128 values, one per value of `cols` columns."""
    return s.repeat_interleave(128, 1)[:, :cols].repeat_interleave(rows, 0).double()


@pytest.mark.parametrize("counts", [[5, 0, 160, 31, 33, 300, 1, 700], [32, 64, 0, 95, 129, 1, 1300], [700, 900]], ids=str)
@pytest.mark.parametrize("N", [256, 328, 1000])
@pytest.mark.parametrize("ctype", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
def test_groups_that_end_inside_pieces_of_an_aligned_c(cuda_device, counts, N, ctype):
    """Integers (sums below 9 * 4 * 200 < 2^24): exact, or rounded once."""
    E, K, R = len(counts), 200, sum(counts) + 40
    g = torch.Generator(device="cuda").manual_seed(N + E)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    nk, nb = 2, -(-N // 128)
    A, B = small_integers(R, 208, g), small_integers(E * N, 208, g)
    sa, sb = powers_of_two(nk, R, g), powers_of_two(E * nb, nk, g)
    C = Guarded(R, N, ref.up(N, 8) + 8, TYPES[ctype])
    ok(sg.sgemm_fp8_grouped(E, off.data_ptr(), R, N, K, A.data_ptr(), 208, sa.data_ptr(), R, B.data_ptr(), 208, N * 208,
                            sb.data_ptr(), nk, nb * nk, 0.0, C.ptr, ctype, C.ld, stream()))
    finish()
    a = A[:, :K].double() * spread(sa.t(), K)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        b = B[e * N:(e + 1) * N, :K].double() * spread(sb[e * nb:(e + 1) * nb], K, 128)[:N]
        assert torch.equal(C.view()[lo:hi], (a[lo:hi] @ b.t()).to(TYPES[ctype]))
    assert bool((C.view()[int(off[-1]):] == 77.0).all()), "rows of no group were written"
    assert C.outside_untouched()


@pytest.mark.parametrize("form", [sg.SGEMM_SCALE_BLOCKS, sg.SGEMM_SCALE_ROWS], ids=["blocks", "rows"])
@pytest.mark.parametrize("shape", [(20000, 1500, 130), (40, 65000, 250)], ids=lambda s: "x".join(map(str, s)))
def test_many_tiles_per_cta(cuda_device, shape, form):
    M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(M)
    nk, nb, ld = -(-K // 128), -(-N // 128), ref.up(K, 16)
    A, B = small_integers(M, ld, g), small_integers(N, ld, g)
    sa = powers_of_two(nk, M, g)
    sb = powers_of_two(nb, nk, g) if form == sg.SGEMM_SCALE_BLOCKS else powers_of_two(nk, N, g)
    b = spread(sb, K, 128)[:N] if form == sg.SGEMM_SCALE_BLOCKS else spread(sb.t(), K)
    C = Guarded(M, N, ref.up(N, 8), torch.float32)
    ok(sg.sgemm_fp8(form, M, N, K, A.data_ptr(), ld, sa.data_ptr(), M, B.data_ptr(), ld, sb.data_ptr(), sb.shape[1], 0.0,
                    C.ptr, sg.SGEMM_F32, C.ld, stream()))
    finish()
    want = (A[:, :K].double() * spread(sa.t(), K)) @ (B[:, :K].double() * b).t()
    assert torch.equal(C.view().double(), want)
    assert C.outside_untouched()


@pytest.mark.parametrize("MN", [(512, 512), (300, 1030)], ids=["512x512", "300x1030"])
def test_many_groups_of_k_most_of_them_short_or_empty(cuda_device, MN):
    """Several tiles per CTA, runs of them without a single K block."""
    M, N = MN
    g = torch.Generator(device="cuda").manual_seed(M)
    counts = [(0, 0, 0, 0, 0, 200, 1, 0, 128, 0, 0, 129, 0, 0, 0, 0)[e % 16] for e in range(112)]
    E, R = len(counts), sum(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    padded = ref.up(R + 127 * min(R, E), 128)
    A, B = (torch.zeros(rows, padded, dtype=FP8, device="cuda") for rows in (M, N))
    begin, at = [], 0
    for n in counts:
        begin.append(at)
        A[:, at:at + n] = small_integers(M, n, g)
        B[:, at:at + n] = small_integers(N, n, g)
        at += ref.up(n, 128)
    sa, sb = powers_of_two(padded // 128, M, g), powers_of_two(padded // 128, N, g)
    C = Guarded(E * M, N, ref.up(N, 4), torch.float32)
    ok(sg.sgemm_fp8_grouped_k(E, off.data_ptr(), padded, M, N, A.data_ptr(), padded, sa.data_ptr(), M, B.data_ptr(),
                              padded, sb.data_ptr(), N, 0.0, C.ptr, sg.SGEMM_F32, C.ld, M * C.ld, stream()))
    finish()
    a, b = (q.double() * spread(s.t(), padded) for q, s in ((A, sa), (B, sb)))
    for e, (at, n) in enumerate(zip(begin, counts)):
        assert torch.equal(C.view()[e * M:(e + 1) * M].double(), a[:, at:at + n] @ b[:, at:at + n].t()), e
    assert C.outside_untouched()


def test_group_offsets_out_of_range_stay_in_bounds(cuda_device):
    """Offsets that are no partition are held to the rows there are."""
    R, N, K, E = 40, 128, 128, 4
    qa = torch.ones(R, K).to(FP8)
    dA, lda = fp8_operand(qa)
    dB = torch.ones(E, N, K, device="cuda").to(FP8)
    one = torch.ones(E * R, device="cuda")
    C = Guarded(R, N, N, torch.float32)
    off = torch.tensor([-7, 10, 25, 1000, 90], dtype=torch.int32, device="cuda")
    ok(sg.sgemm_fp8_grouped(E, off.data_ptr(), R, N, K, dA.data_ptr(), lda, one.data_ptr(), R, dB.data_ptr(), K, N * K,
                            one.data_ptr(), 1, 1, 0.0, C.ptr, sg.SGEMM_F32, N, stream()))
    finish()
    assert bool((C.view() == 128.0).all()) and C.outside_untouched()


# ---------------------------------------------------------------- quantisers

def special(x):
    """Blocks with zeros, denormals, the type's largest values, one large value."""
    x[0] = 0.0
    if x.shape[0] > 3:
        x[1] = 1e-40
        x[2, :: 3] = 3.0e38
        x[3, -1] = 1e30
    return x


def same_bits(q, want):
    a, b = q.cpu().view(torch.uint8), want.view(torch.uint8)
    return bool(((a == b) | ((a & 0x7F == 0) & (b & 0x7F == 0))).all())


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 127), (16, 128), (17, 129), (40, 700), (129, 1024)])
@pytest.mark.parametrize("type_", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gathered", [False, True], ids=["plain", "gathered"])
def test_quantize_rows(cuda_device, rows, cols, type_, gathered):
    g = torch.Generator().manual_seed(rows + cols)
    n = 23 if gathered else rows
    x = special(torch.randn(n, cols, generator=g) * 10).to(TYPES[type_])
    pick = torch.randint(-1, n + 1, (rows,), generator=g, dtype=torch.int32) if gathered else None
    for ld, shift in ((cols + 3, 1), (ref.up(cols, 8), 0)):
        src = Guarded(n, cols, ld, TYPES[type_], shift).put(x)
        q = Guarded(rows, cols, ref.up(cols, 16), FP8)
        s = Guarded(-(-cols // 128), rows, rows + 2, torch.float32)
        dpick = pick.cuda() if gathered else None
        ok(sg.sgemm_fp8_quantize_rows(rows, cols, src.ptr, type_, ld, dpick.data_ptr() if gathered else 0, n, q.ptr, q.ld,
                                      s.ptr, s.ld, stream()))
        finish()
        xx = x.float()
        if gathered:
            inside = (pick >= 0) & (pick < n)
            xx = torch.where(inside[:, None], xx[pick.clamp(0, n - 1).long()], torch.zeros(()))
        wq, ws = ref.quantize(xx, 1)
        assert same_bits(q.view(), wq) and torch.equal(s.view().cpu(), ws.t())
        assert q.outside_untouched(pad=15) and s.outside_untouched() and src.outside_untouched()


@pytest.mark.parametrize("rows,cols,counts", [(1, 1, None), (130, 65, None), (128, 128, None), (300, 200, [300]),
                                              (300, 200, [0, 130, 128, 0, 1, 41]), (7, 140, [1, 1, 0, 5]),
                                              (0, 64, [0, 0]), (50, 64, [20, 10])])
@pytest.mark.parametrize("type_", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gathered", [False, True], ids=["plain", "gathered"])
def test_quantize_both(cuda_device, rows, cols, counts, type_, gathered):
    g = torch.Generator().manual_seed(rows + cols)
    n = 11 if gathered and rows else rows
    x = torch.randn(n, cols, generator=g)
    x = (special(x) if n else x).to(TYPES[type_])
    pick = torch.randint(0, max(n, 1), (rows,), generator=g, dtype=torch.int32)
    groups = counts if counts is not None else [rows]
    off = torch.tensor(np.concatenate([[0], np.cumsum(groups)]), dtype=torch.int32).cuda() if counts else None
    padded = ref.up(rows + 127 * min(rows, len(groups)), 128) + 128
    ld = cols + (1 if type_ == sg.SGEMM_F32 else 0)
    src = Guarded(n, cols, ld, TYPES[type_]).put(x)
    q, s = Guarded(rows, cols, ref.up(cols, 16), FP8), Guarded(-(-cols // 128), rows, rows, torch.float32)
    qt, st = Guarded(cols, padded, padded + 16, FP8), Guarded(padded // 128, cols, cols + 1, torch.float32)
    dpick = pick.cuda()
    ok(sg.sgemm_fp8_quantize_both(rows, cols, src.ptr, type_, ld, dpick.data_ptr() if gathered else 0, n, len(groups),
                                  off.data_ptr() if counts else 0, padded, q.ptr, q.ld, s.ptr, s.ld, qt.ptr, qt.ld,
                                  st.ptr, st.ld, stream()))
    finish()
    xx = x.float()[pick.long()] if gathered and rows else x.float()
    full = torch.zeros(padded, cols)
    at, src_at, covered = 0, 0, sum(groups)
    for c in groups:
        full[at:at + c] = xx[src_at:src_at + c]
        at, src_at = at + ref.up(c, 128), src_at + c
    wq, ws = ref.quantize(full, 0)
    assert same_bits(qt.view(), wq.t().contiguous()) and torch.equal(st.view().cpu(), ws)
    if covered:
        wq, ws = ref.quantize(xx[:covered], 1)
        assert same_bits(q.view()[:covered], wq) and torch.equal(s.view().cpu()[:, :covered], ws.t())
    assert q.outside_untouched(pad=15) and qt.outside_untouched() and st.outside_untouched()


@pytest.mark.parametrize("rows,cols,batch", [(1, 1, 1), (128, 128, 1), (129, 300, 2), (257, 100, 3), (64, 513, 1)])
@pytest.mark.parametrize("transpose", [0, 1])
@pytest.mark.parametrize("type_", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
def test_quantize_blocks(cuda_device, rows, cols, batch, transpose, type_):
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(batch, rows, cols, generator=g).to(TYPES[type_])
    qr, qc = (cols, rows) if transpose else (rows, cols)
    ldq, sr, sc = ref.up(qc, 16), -(-qr // 128), -(-qc // 128)
    src = x.cuda()
    q = torch.zeros(batch, qr, ldq, dtype=torch.uint8, device="cuda")
    s = torch.zeros(batch, sr, sc, device="cuda")
    ok(sg.sgemm_fp8_quantize_blocks(rows, cols, src.data_ptr(), type_, cols, rows * cols, transpose, q.data_ptr(), ldq,
                                    qr * ldq, s.data_ptr(), sc, sr * sc, batch, stream()))
    finish()
    for b in range(batch):
        wq, ws = ref.quantize(x[b].float().t().contiguous() if transpose else x[b].float(), None)
        assert same_bits(q[b, :, :qc].contiguous().view(FP8), wq) and torch.equal(s[b].cpu(), ws)


def test_quantize_keeps_nan_and_infinity_in_their_blocks(cuda_device):
    x = torch.randn(200, 300)
    x[3, 5], x[150, 200] = float("nan"), float("inf")
    src = x.cuda()
    q, s = torch.zeros(200, 304, dtype=FP8, device="cuda"), torch.zeros(3, 200, device="cuda")
    qt, st = torch.zeros(300, 256, dtype=FP8, device="cuda"), torch.zeros(2, 300, device="cuda")
    ok(sg.sgemm_fp8_quantize_both(200, 300, src.data_ptr(), 0, 300, 0, 200, 1, 0, 256, q.data_ptr(), 304, s.data_ptr(), 200,
                                  qt.data_ptr(), 256, st.data_ptr(), 300, stream()))
    finish()
    s, st, q = s.cpu(), st.cpu(), q.cpu().float()
    assert s[0, 3].isnan() and s[1, 150].isinf() and int((~s.isfinite()).sum()) == 2
    assert st[0, 5].isnan() and st[1, 200].isinf() and int((~st.isfinite()).sum()) == 2
    assert bool(q[3, :128].isnan().all()) and q[150, 200].isnan() and int(q[:, :300].isnan().sum()) == 129


# ------------------------------------------------------------------- routing

def grid_logits(T, E, seed):
    """Logits whose scores are far apart for FP32: a shuffled grid per token."""
    rng = np.random.RandomState(seed)
    return np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float64) * (6.0 / E) - 3.0


ROUTES = [  # E, k, kind, bias, groups, kept, two, renorm, scale
    (8, 2, "softmax", False, 1, 1, False, True, 1.0), (64, 6, "sigmoid", True, 8, 4, True, True, 2.5),
    (64, 6, "sigmoid", False, 8, 3, False, False, 1.0), (60, 4, "softmax", False, 1, 1, False, False, 1.0),
    (128, 8, "softmax", True, 1, 1, False, True, 1.0), (160, 6, "softmax", False, 8, 3, False, False, 16.0),
    (256, 8, "sigmoid", True, 8, 4, True, True, 2.5), (1024, 32, "softmax", False, 32, 5, True, True, 1.0),
    (1, 1, "softmax", False, 1, 1, False, True, 1.0), (33, 32, "sigmoid", False, 3, 2, True, True, 1.0),
    (512, 10, "sigmoid", True, 1, 1, False, False, 1.0),
]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("T", [1, 67])
def test_route_and_its_gradient(cuda_device, case, T):
    E, k, kind, with_bias, groups, kept, two, renorm, scale = case
    L = grid_logits(T, E, E + T).astype(np.float32).astype(np.float64)
    if T > 10:
        L[3] = -np.inf                    # a token with no expert
        L[4, 1:] = -np.inf                # one with a single expert
        L[5, : E // 2] = np.nan
    bias = (np.random.RandomState(1).permutation(E) * 0.37 / E).astype(np.float32) if with_bias else None
    W, I = ref.route(np.where(np.isnan(L), -np.inf, L), bias, kind, groups, kept, two, k, renorm, scale)
    dl = Guarded(T, E, E + 1, torch.float32).put(torch.tensor(L))
    db = torch.tensor(bias).cuda() if with_bias else None
    w, ix = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    kinds = {"softmax": sg.SGEMM_SCORE_SOFTMAX, "sigmoid": sg.SGEMM_SCORE_SIGMOID}
    ok(sg.sgemm_route(T, E, dl.ptr, sg.SGEMM_F32, E + 1, db.data_ptr() if with_bias else 0, kinds[kind], groups, kept,
                      int(two), k, int(renorm), scale, w.data_ptr(), ix.data_ptr(), stream()))
    finish()
    assert np.array_equal(ix.cpu().numpy(), I)
    tol = (E / 2 + 8) * 2.0 ** -23
    assert np.all(np.abs(w.cpu().numpy() - W) <= tol * np.abs(W) + 1e-38)
    # The gradient, against the definition differentiated in 64 bits.
    gw = np.random.RandomState(2).randn(T, k).astype(np.float32)
    G = np.zeros((T, E))
    for t in range(T):
        at = I[t][I[t] >= 0]
        if len(at) == 0:
            continue
        x = torch.tensor(np.where(np.isnan(L[t]), -np.inf, L[t]), requires_grad=True)
        s = torch.special.expit(x) if kind == "sigmoid" else torch.softmax(x, 0)
        v = s[torch.tensor(at)]
        v = scale * (v / v.sum() if renorm else v)
        (v * torch.tensor(gw[t][I[t] >= 0].astype(np.float64))).sum().backward()
        G[t] = np.nan_to_num(x.grad.numpy())
    d = Guarded(T, E, E + 2, torch.float32)
    dgw = torch.tensor(gw).cuda()
    ok(sg.sgemm_route_backward(T, E, dl.ptr, sg.SGEMM_F32, E + 1, kinds[kind], k, int(renorm), scale, ix.data_ptr(),
                               dgw.data_ptr(), d.ptr, E + 2, stream()))
    finish()
    # Each entry is a weight times a difference of gradients and their mean: the bound on the weights, on the
    # magnitudes before the difference.
    big = np.abs(gw).max() * scale * 2
    assert np.all(np.abs(d.view().cpu().numpy() - G) <= tol * big + 1e-38)
    assert d.outside_untouched()


def test_route_gradient_against_differences(cuda_device):
    """Central differences of the kernel's own weights, at a step where rounding and curvature are both small:
    h = 2^-6, error of the difference about h^2 / 6 * |w'''| + 2^-23 / h, below 2e-4 of the gradient's scale."""
    T, E, k = 1, 16, 4
    for kind in (sg.SGEMM_SCORE_SOFTMAX, sg.SGEMM_SCORE_SIGMOID):
        for renorm in (0, 1):
            l0 = grid_logits(1, E, 3).astype(np.float32) * 2
            gw = np.random.RandomState(5).randn(1, k).astype(np.float32)

            def weights(l):
                dl = torch.tensor(l).cuda()
                w, ix = torch.empty(1, k, device="cuda"), torch.empty(1, k, dtype=torch.int32, device="cuda")
                ok(sg.sgemm_route(T, E, dl.data_ptr(), 0, E, 0, kind, 1, 1, 0, k, renorm, 1.0, w.data_ptr(), ix.data_ptr(),
                                  stream()))
                finish()
                return w.cpu().numpy().astype(np.float64), ix

            _, ix = weights(l0)
            dl, dg, out = torch.tensor(l0).cuda(), torch.tensor(gw).cuda(), torch.empty(1, E, device="cuda")
            ok(sg.sgemm_route_backward(T, E, dl.data_ptr(), 0, E, kind, k, renorm, 1.0, ix.data_ptr(), dg.data_ptr(),
                                       out.data_ptr(), E, stream()))
            finish()
            h = 2.0 ** -6
            for e in range(E):
                up, down = l0.copy(), l0.copy()
                up[0, e] += h
                down[0, e] -= h
                diff = ((weights(up)[0] - weights(down)[0]) * gw).sum() / (2 * h)
                assert abs(diff - out[0, e].item()) <= 2e-4 * max(1.0, np.abs(gw).max()), (kind, renorm, e)


def test_route_breaks_ties_towards_the_lowest_expert(cuda_device):
    T, E, k = 40, 100, 8
    rng = np.random.RandomState(0)
    L = rng.randint(-2, 3, (T, E)).astype(np.float32)
    L[0], L[1] = 0.0, -0.0
    L[1, ::2] = 0.0                                   # +0 and -0 are one value
    for dtype, t in ((sg.SGEMM_F32, torch.float32), (sg.SGEMM_BF16, torch.bfloat16)):
        _, I = ref.route(L.astype(np.float64), None, "softmax", 1, 1, False, k, True, 1.0)
        dl = torch.tensor(L).to(t).cuda()
        w, ix = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
        ok(sg.sgemm_route(T, E, dl.data_ptr(), dtype, E, 0, 0, 1, 1, 0, k, 1, 1.0, w.data_ptr(), ix.data_ptr(), stream()))
        finish()
        assert np.array_equal(ix.cpu().numpy(), I)


def test_route_with_infinite_logits(cuda_device):
    L = np.zeros((2, 8), np.float32)
    L[0, 3] = np.inf
    L[1, 2] = L[1, 6] = np.inf
    dl = torch.tensor(L).cuda()
    w, ix = torch.empty(2, 2, device="cuda"), torch.empty(2, 2, dtype=torch.int32, device="cuda")
    ok(sg.sgemm_route(2, 8, dl.data_ptr(), 0, 8, 0, 0, 1, 1, 0, 2, 1, 1.0, w.data_ptr(), ix.data_ptr(), stream()))
    finish()
    assert ix.cpu().tolist() == [[3, 0], [2, 6]] and w.cpu().tolist() == [[1.0, 0.0], [0.5, 0.5]]


@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (7, 6, 64), (100, 8, 256), (2047, 8, 60), (2049, 8, 1024),
                                   (5000, 7, 128), (70000, 8, 16), (4096, 1, 33), (4097, 1, 33), (16384, 8, 256),
                                   (16385, 8, 64),
                                   (16384, 1, 9), (16385, 1, 9)])
def test_dispatch(cuda_device, T, k, E):
    rng = np.random.RandomState(T + E)
    idx = rng.randint(-1, E + 1, (T, k)) if T % 2 else np.minimum(rng.geometric(0.05, (T, k)) - 1, E - 1)
    O, R, K = ref.dispatch(idx, E)
    di = torch.tensor(idx, dtype=torch.int32).cuda()
    off = torch.full((E + 1,), 99, dtype=torch.int32, device="cuda")
    row = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    tok = torch.full((T * k,), 99, dtype=torch.int32, device="cuda")
    ok(sg.sgemm_dispatch(T, k, E, di.data_ptr(), off.data_ptr(), row.data_ptr(), tok.data_ptr(), stream()))
    finish()
    assert np.array_equal(off.cpu().numpy(), O) and np.array_equal(row.cpu().numpy(), R)
    assert np.array_equal(tok.cpu().numpy(), K)


def test_dispatch_reports_a_failed_allocation(cuda_device):
    T, k, E = 20000, 7, 128                          # more pairs than a cluster holds: counts in scratch
    di = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    out = [torch.full((n,), 99, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k)]
    ok(sg.sgemm_test_fail_next_allocs(1))
    assert sg.sgemm_dispatch(T, k, E, di.data_ptr(), *[o.data_ptr() for o in out], stream()) == sg.SGEMM_ERR_ALLOC
    torch.cuda.synchronize()
    assert all(bool((o == 99).all()) for o in out)
    ok(sg.sgemm_dispatch(T, k, E, di.data_ptr(), *[o.data_ptr() for o in out], stream()))
    finish()
    assert int(out[0][1]) == T * k


# ----------------------------------------------------------------- combining

@pytest.mark.parametrize("T,k,cols", [(1, 1, 1), (5, 3, 130), (16, 6, 2048), (33, 8, 4100), (3, 32, 520)])
@pytest.mark.parametrize("type_", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("weighted", [True, False], ids=["weighted", "ones"])
@pytest.mark.parametrize("ragged", [True, False], ids=["odd_strides", "aligned"])
def test_combine_and_its_gradients(cuda_device, T, k, cols, type_, weighted, ragged):
    g = torch.Generator().manual_seed(T * k + cols)
    R = T * k + 2
    dt = TYPES[type_]
    eps = 2.0 ** -8 if type_ == sg.SGEMM_BF16 else 0.0     # the one rounding of the result
    Y = torch.randn(R, cols, generator=g).to(dt)
    go = torch.randn(T, cols, generator=g).to(dt)
    row = torch.randperm(R, generator=g)[:T * k].view(T, k).to(torch.int32)
    if T > 2:
        row[1, 0], row[2, k - 1] = -1, R                # no row
        row[0] = -1 if k < 8 else row[0]
    w = torch.randn(T, k, generator=g) if weighted else None
    there = ((row >= 0) & (row < R)).double()
    picked = Y.double()[row.clamp(0, R - 1).long()] * there[:, :, None]
    ww = w.double() if weighted else torch.ones(T, k).double()
    pad = 3 if ragged else ref.up(cols, 8) - cols
    dY = Guarded(R, cols, cols + pad, dt, 1 if ragged else 0).put(Y)
    dgo = Guarded(T, cols, cols + pad, dt).put(go)
    out = Guarded(T, cols, cols + pad, dt, 1 if ragged else 0)
    drow, dw = row.cuda(), w.cuda() if weighted else None
    wp = dw.data_ptr() if weighted else 0
    ok(sg.sgemm_combine(T, k, cols, R, dY.ptr, type_, dY.ld, drow.data_ptr(), wp, out.ptr, out.ld, stream()))
    gy, gw = Guarded(R, cols, cols + pad, dt), torch.full((T, k), 9.0, device="cuda")
    ok(sg.sgemm_combine_backward(T, k, cols, R, dgo.ptr, type_, dgo.ld, dY.ptr, dY.ld, drow.data_ptr(), wp, gy.ptr, gy.ld,
                                 gw.data_ptr(), stream()))
    finish()
    terms = picked * ww[:, :, None]
    want = terms.sum(1)
    assert bool(((out.view().cpu().double() - want).abs() <= (k + 1) * 2.0 ** -24 * terms.abs().sum(1) + eps * want.abs() + 1e-38).all())
    want_gw = (go.double()[:, None, :] * picked).sum(2)
    bound = (go.double()[:, None, :] * picked).abs().sum(2)
    assert bool(((gw.cpu().double() - want_gw).abs() <= cols * 2.0 ** -24 * bound + 1e-38).all())
    got, named = gy.view().cpu().double(), torch.zeros(R, dtype=torch.bool)
    for t in range(T):
        for j in range(k):
            r = int(row[t, j])
            if 0 <= r < R:
                x = ww[t, j] * go[t].double()
                assert bool(((got[r] - x).abs() <= (eps + 2.0 ** -24) * x.abs() + 1e-38).all())
                named[r] = True
    assert bool((gy.view().cpu()[~named] == 77.0).all()), "rows that no pair names were written"
    assert out.outside_untouched() and gy.outside_untouched() and dY.outside_untouched()


def test_combine_weight_gradient_against_differences(cuda_device):
    """out is linear in the weights, so a difference of two weights' outputs is exact up to rounding: with
    L = <grad, out>, (L(w + 1) - L(w)) is grad_w to cols 2^-22 of sum |grad| |Y|."""
    T, k, cols = 4, 3, 96
    g = torch.Generator().manual_seed(0)
    Y, go, w = torch.randn(12, cols, generator=g), torch.randn(T, cols, generator=g), torch.randn(T, k, generator=g)
    row = torch.randperm(12, generator=g).view(T, k).to(torch.int32).cuda()
    dY, dgo = Y.cuda(), go.cuda()

    def out_of(w):
        dw, out = w.cuda(), torch.empty(T, cols, device="cuda")
        ok(sg.sgemm_combine(T, k, cols, 12, dY.data_ptr(), 0, cols, row.data_ptr(), dw.data_ptr(), out.data_ptr(), cols,
                            stream()))
        finish()
        return out.cpu().double()

    gw, dw = torch.empty(T, k, device="cuda"), w.cuda()
    ok(sg.sgemm_combine_backward(T, k, cols, 12, dgo.data_ptr(), 0, cols, dY.data_ptr(), cols, row.data_ptr(),
                                 dw.data_ptr(), 0, cols, gw.data_ptr(), stream()))
    finish()
    base = out_of(w)
    for j in range(k):
        w1 = w.clone()
        w1[:, j] += 1.0
        diff = ((out_of(w1) - base) * go.double()).sum(1)
        bound = (go.double().abs() * (base.abs() + Y.double().abs().max())).sum(1) * 2.0 ** -20
        assert bool(((gw[:, j].cpu().double() - diff).abs() <= bound).all())


# ------------------------------------------------- streams, graphs, long rows

def test_another_stream_and_graph_capture(cuda_device):
    """The chain of a layer's calls on a side stream, captured once and replayed on new inputs."""
    T, E, k, D, F = 24, 8, 2, 256, 384
    g = torch.Generator().manual_seed(3)
    W = torch.randn(E, F, D, generator=g).cuda()
    x, logits = torch.zeros(T, D, device="cuda"), torch.zeros(T, E, device="cuda")
    qw, sw = torch.empty(E, F, D, dtype=FP8, device="cuda"), torch.empty(E, F // 128, D // 128, device="cuda")
    w, ix = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    off, row = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    tok = torch.empty(T * k, dtype=torch.int32, device="cuda")
    qa, sa = torch.empty(T * k, D, dtype=FP8, device="cuda"), torch.empty(D // 128, T * k, device="cuda")
    y, out = torch.empty(T * k, F, device="cuda"), torch.empty(T, F, device="cuda")

    def step(st):
        ok(sg.sgemm_route(T, E, logits.data_ptr(), 0, E, 0, 0, 1, 1, 0, k, 1, 1.0, w.data_ptr(), ix.data_ptr(), st))
        ok(sg.sgemm_dispatch(T, k, E, ix.data_ptr(), off.data_ptr(), row.data_ptr(), tok.data_ptr(), st))
        ok(sg.sgemm_fp8_quantize_rows(T * k, D, x.data_ptr(), 0, D, tok.data_ptr(), T, qa.data_ptr(), D, sa.data_ptr(),
                                      T * k, st))
        ok(sg.sgemm_fp8_grouped(E, off.data_ptr(), T * k, F, D, qa.data_ptr(), D, sa.data_ptr(), T * k, qw.data_ptr(), D,
                                F * D, sw.data_ptr(), D // 128, F // 128 * (D // 128), 0.0, y.data_ptr(), 0, F, st))
        ok(sg.sgemm_combine(T, k, F, T * k, y.data_ptr(), 0, F, row.data_ptr(), w.data_ptr(), out.data_ptr(), F, st))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ok(sg.sgemm_fp8_quantize_blocks(F, D, W.data_ptr(), 0, D, F * D, 0, qw.data_ptr(), D, F * D, sw.data_ptr(),
                                        D // 128, F // 128 * (D // 128), E, side.cuda_stream))
        step(side.cuda_stream)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(torch.cuda.current_stream().cuda_stream)
    for seed in (1, 2):
        h = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, D, generator=h))
        logits.copy_(torch.randn(T, E, generator=h))
        torch.cuda.synchronize()
        graph.replay()
        finish()
        p, at = torch.softmax(logits.cpu().double(), 1).topk(k, 1)
        p = p / p.sum(1, keepdim=True)
        want = torch.zeros(T, F).double()
        for t in range(T):
            for j in range(k):
                want[t] += p[t, j] * (W[at[t, j]].cpu().double() @ x[t].cpu().double())
        # Two 8-bit operands: each value within 2^-4 of itself, the products of a dot product independent.
        scale = want.norm() / want.numel() ** 0.5
        assert float((out.cpu().double() - want).abs().max()) <= 0.3 * float(scale)
        assert float((out.cpu().double() - want).norm() / want.norm()) <= 2.0 ** -4


def test_offsets_past_32_bits(cuda_device):
    """Rows of C, of A and of the quantiser's input that lie more than 2^31 elements apart."""
    M, N, K, ld = 300, 64, 128, 1 << 23
    qa = torch.ones(M, K).to(FP8)
    dB = torch.ones(N, K, device="cuda").to(FP8)
    A = torch.empty(M * ld, dtype=torch.uint8, device="cuda")
    A.view(M, ld)[:, :K] = qa.view(torch.uint8).cuda()
    one = torch.ones(M, device="cuda")
    C = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    ok(sg.sgemm_fp8(0, M, N, K, A.data_ptr(), ld, one.data_ptr(), M, dB.data_ptr(), K, one.data_ptr(), 1, 0.0, C.data_ptr(),
                    sg.SGEMM_BF16, ld, stream()))
    finish()
    assert bool((C.view(M, ld)[:, :N] == 128.0).all())
    src = C.view(M, ld)
    src[:, :200] = 2.0
    q, s = torch.zeros(M, 208, dtype=FP8, device="cuda"), torch.zeros(2, M, device="cuda")
    ok(sg.sgemm_fp8_quantize_rows(M, 200, C.data_ptr(), sg.SGEMM_BF16, ld, 0, M, q.data_ptr(), 208, s.data_ptr(), M, stream()))
    finish()
    assert bool((q[:, :200].float() == 448.0).all()) and bool((s == 2.0 / 448.0).all())
