"""Paths of the experts' operators that the sizes, strides and types of
test_experts_gpu.py do not reach."""

import threading

import pytest
import torch

import dense_fp32_matrix_07_gb300 as sg
import experts_ref as ref

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
TYPES = {sg.SGEMM_F32: torch.float32, sg.SGEMM_BF16: torch.bfloat16}


def stream():
    return torch.cuda.current_stream().cuda_stream


def ok(rc):
    assert rc == sg.SGEMM_OK, sg.sgemm_error_string(rc)


def finish():
    torch.cuda.synchronize()
    assert sg.sgemm_check_status(stream()) == sg.SGEMM_OK


# ---------------------------------------------------------------- quantisers

@pytest.mark.parametrize("form", ["rows", "both", "blocks", "blocks transposed"])
def test_scales_right_behind_the_values(cuda_device, form):
    """One buffer: 8-bit values, and the scales from where the last row's stores end. Exact in every bit."""
    rows, cols = 9, 130
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(0))
    src = x.cuda()
    turned = form == "blocks transposed"
    qr, qc, ld = (cols, rows, 16) if turned else (rows, cols, 144)
    end = (qr - 1) * ld + (16 if turned else 136)
    shape = (2, rows) if form in ("rows", "both") else (-(-qr // 128), -(-qc // 128))
    buf = torch.zeros(end + 4 * shape[0] * shape[1], dtype=torch.uint8, device="cuda")
    q, s = buf.data_ptr(), buf.data_ptr() + end
    if form == "rows":
        ok(sg.sgemm_fp8_quantize_rows(rows, cols, src.data_ptr(), sg.SGEMM_F32, cols, 0, rows, q, ld, s, rows, stream()))
    elif form == "both":
        qt, st = torch.zeros(cols, 128, dtype=FP8, device="cuda"), torch.zeros(1, cols, device="cuda")
        ok(sg.sgemm_fp8_quantize_both(rows, cols, src.data_ptr(), sg.SGEMM_F32, cols, 0, rows, 1, 0, 128, q, ld, s, rows,
                                      qt.data_ptr(), 128, st.data_ptr(), cols, stream()))
    else:
        ok(sg.sgemm_fp8_quantize_blocks(rows, cols, src.data_ptr(), sg.SGEMM_F32, cols, 0, int(turned), q, ld, 0, s,
                                        shape[1], 0, 1, stream()))
    finish()
    wq, ws = ref.quantize(x.t().contiguous() if turned else x, 1 if form in ("rows", "both") else None)
    got = torch.zeros(qr * ld, dtype=torch.uint8)
    got[:end] = buf.cpu()[:end]
    assert torch.equal(got.view(qr, ld)[:, :qc].contiguous().view(FP8).float(), wq.float())
    scales = buf[end:].cpu().view(torch.float32).view(shape)
    assert torch.equal(scales, ws.t() if form in ("rows", "both") else ws)


# ------------------------------------------------------------------ products
#
# Small integers in e4m3 and scales that are powers of two: every sum is an
# integer below 2^24, so an FP32 result is exact, and a bfloat16 result that
# one rounded once. beta = 0.5 and old values that are even keep that.

def integers(*shape, g, most=3):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").float()


def twos(*shape, g):
    return 2.0 ** torch.randint(0, 2, shape, generator=g, device="cuda").float()


def over_rows(s, cols):
    """Scales [K block][row] as one per value of rows x cols."""
    return s.t().repeat_interleave(128, 1)[:, :cols].double()


def over_blocks(s, rows, cols):
    return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols].double()


class Placed:
    """rows x cols old values of C, `shift` elements into a buffer, with leading dimension ld and `fill` around them."""

    def __init__(self, rows, cols, ld, dtype, shift, g):
        n = shift + rows * ld + 32
        self.flat = torch.full((n,), 77.0, dtype=dtype, device="cuda")
        self.rows, self.cols, self.ld, self.shift = rows, cols, ld, shift
        self.old = 2 * integers(rows, cols, g=g, most=9)
        self.view().copy_(self.old)
        self.start = self.flat.clone()

    @property
    def ptr(self):
        return self.flat.data_ptr() + self.shift * self.flat.element_size()

    def view(self):
        return self.flat[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols]

    def check(self, want, rows=None):
        """`want` (64-bit) in `rows` (all by default), everything else as before."""
        rows = slice(None) if rows is None else rows
        assert torch.equal(self.view()[rows], want.to(self.flat.dtype))
        self.view()[rows] = self.old[rows].to(self.flat.dtype)
        assert torch.equal(self.flat, self.start)


# M, N, K: split tiles with B on the lanes, whole ones (many weight tiles), 128 columns, 256 columns; odd ones.
BETA_SHAPES = [(20, 777, 1300), (9, 40000, 129), (130, 520, 300), (1100, 5200, 140), (2000, 1024, 384)]


@pytest.mark.parametrize("shape", BETA_SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("form", [sg.SGEMM_SCALE_BLOCKS, sg.SGEMM_SCALE_ROWS], ids=["blocks", "rows"])
@pytest.mark.parametrize("ctype", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
def test_product_added_to_c(cuda_device, shape, form, ctype, aligned):
    M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    nk, nb, ld = -(-K // 128), -(-N // 128), ref.up(K, 16)
    A, B = integers(M, ld, g=g).to(FP8), integers(N, ld, g=g).to(FP8)
    sa = twos(nk, M, g=g)
    sb = twos(nb, nk, g=g) if form == sg.SGEMM_SCALE_BLOCKS else twos(nk, N, g=g)
    b = over_blocks(sb, N, K) if form == sg.SGEMM_SCALE_BLOCKS else over_rows(sb, K)
    want = (A[:, :K].double() * over_rows(sa, K)) @ (B[:, :K].double() * b).t()
    C = Placed(M, N, ref.up(N, 8) + (0 if aligned else 3), TYPES[ctype], 0 if aligned else 1, g)
    ok(sg.sgemm_fp8(form, M, N, K, A.data_ptr(), ld, sa.data_ptr(), M, B.data_ptr(), ld, sb.data_ptr(), sb.shape[1], 0.5,
                    C.ptr, ctype, C.ld, stream()))
    finish()
    C.check(want + 0.5 * C.old.double())


@pytest.mark.parametrize("counts", [[1, 0, 3, 2, 0, 7, 5], [5, 0, 160, 31, 33, 300, 1, 700]], ids=["few", "many"])
@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("ctype", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
def test_grouped_added_to_c_with_strides_between_the_weights(cuda_device, counts, beta, ctype, aligned):
    E, N, K, R = len(counts), 328, 200, sum(counts) + 9
    g = torch.Generator(device="cuda").manual_seed(E)
    off = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    nk, nb, ld = 2, 3, 208
    stride_b, ld_sb, stride_sb = N * ld + 48, nk + 1, nb * (nk + 1) + 2
    A = integers(R, ld, g=g).to(FP8)
    B = torch.full((E * stride_b,), 0x7F, dtype=torch.uint8, device="cuda").view(FP8)      # NaN between the matrices
    sb = torch.full((E * stride_sb,), float("nan"), device="cuda")
    sa, weights = twos(nk, R, g=g), []
    for e in range(E):
        q, s = integers(N, K, g=g).to(FP8), twos(nb, nk, g=g)
        B[e * stride_b:e * stride_b + N * ld].view(N, ld)[:, :K] = q
        sb[e * stride_sb:e * stride_sb + nb * ld_sb].view(nb, ld_sb)[:, :nk] = s
        weights.append(q.double() * over_blocks(s, N, K))
    C = Placed(R, N, ref.up(N, 8) + (0 if aligned else 3), TYPES[ctype], 0 if aligned else 1, g)
    ok(sg.sgemm_fp8_grouped(E, off.data_ptr(), R, N, K, A.data_ptr(), ld, sa.data_ptr(), R, B.data_ptr(), ld, stride_b,
                            sb.data_ptr(), ld_sb, stride_sb, beta, C.ptr, ctype, C.ld, stream()))
    finish()
    a = A[:, :K].double() * over_rows(sa, K)
    o = off.tolist()
    want = torch.cat([a[lo:hi] @ w.t() for w, lo, hi in zip(weights, o, o[1:])])
    C.check(want + beta * C.old[:o[-1]].double(), slice(0, o[-1]))


@pytest.mark.parametrize("MN", [(130, 100), (512, 384), (300, 1032)], ids=["130x100", "512x384", "300x1032"])
@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("ctype", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
def test_weight_gradients_from_the_tokens_on_are_exact(cuda_device, MN, beta, ctype, aligned):
    """Quantiser and product together. Integers to 7, and a 7 in each column of each group's blocks: the values are held
    as 64 times themselves, the scales are 1 / 64, and every sum is an integer below 49 * 1300 < 2^24."""
    M, N = MN
    counts = [127, 129, 0, 300, 1, 128, 0, 520]
    E, R = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(M)
    off = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    o = off.tolist()
    firsts = [r for lo, hi in zip(o, o[1:]) for r in range(lo, hi, 128)]
    padded = ref.up(R + 127 * min(R, E), 128)
    held = []
    for cols in (M, N):
        x = integers(R, cols, g=g, most=7)
        x[firsts] = 7.0 * (1 - 2 * torch.randint(0, 2, (len(firsts), cols), generator=g, device="cuda").float())
        q, s = torch.zeros(cols, padded, dtype=FP8, device="cuda"), torch.zeros(padded // 128, cols, device="cuda")
        ok(sg.sgemm_fp8_quantize_cols(R, cols, x.data_ptr(), sg.SGEMM_F32, cols, 0, R, E, off.data_ptr(), padded,
                                      q.data_ptr(), padded, s.data_ptr(), cols, stream()))
        held.append((x, q, s))
    (dy, qa, sa), (x, qb, sb) = held
    rows = M + 3                                       # of C from one group to the next
    C = Placed(E * rows, N, ref.up(N, 8) + (0 if aligned else 3), TYPES[ctype], 0 if aligned else 1, g)
    ok(sg.sgemm_fp8_grouped_k(E, off.data_ptr(), padded, M, N, qa.data_ptr(), padded, sa.data_ptr(), M, qb.data_ptr(),
                              padded, sb.data_ptr(), N, beta, C.ptr, ctype, C.ld, rows * C.ld, stream()))
    finish()
    want = torch.cat([dy[lo:hi].double().t() @ x[lo:hi].double() for lo, hi in zip(o, o[1:])])
    at = torch.cat([torch.arange(e * rows, e * rows + M) for e in range(E)]).cuda()
    C.check(want + beta * C.old[at].double(), at)


# ------------------------------------------------------------------- routing

KINDS = {"softmax": sg.SGEMM_SCORE_SOFTMAX, "sigmoid": sg.SGEMM_SCORE_SIGMOID}
ROUTES = [  # E, k, kind, bias, groups, kept, two, renorm
    (8, 2, "softmax", False, 1, 1, False, True), (32, 5, "sigmoid", True, 4, 2, True, True),
    (64, 6, "softmax", False, 8, 3, False, False), (128, 8, "sigmoid", False, 1, 1, False, True),
    (256, 8, "sigmoid", True, 8, 4, True, True), (256, 6, "softmax", False, 8, 3, False, False),
    (512, 10, "sigmoid", False, 16, 5, False, False), (512, 9, "softmax", True, 1, 1, False, True),
    (1024, 32, "softmax", False, 32, 5, False, True), (1024, 7, "sigmoid", True, 32, 9, True, False),
]


def routed(values, ld, ld_g, type_, case, bias, g, shift=0):
    """Weights, choice and gradient of the library, with rows of the logits ld and of the gradient ld_g apart."""
    E, k, kind, _, groups, kept, two, renorm = case
    T, dt = values.shape[0], TYPES[type_]
    l = torch.full((T * ld + shift,), float("nan"), dtype=dt, device="cuda")
    l[shift:].view(T, ld)[:, :E] = values
    d = torch.full((T * ld_g + shift,), 77.0, dtype=dt, device="cuda")
    w, ix = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    at, out = (t.data_ptr() + shift * t.element_size() for t in (l, d))
    ok(sg.sgemm_route(T, E, at, type_, ld, bias.data_ptr() if bias is not None else 0, KINDS[kind], groups, kept, int(two),
                      k, int(renorm), 2.5, w.data_ptr(), ix.data_ptr(), stream()))
    ok(sg.sgemm_route_backward(T, E, at, type_, ld, KINDS[kind], k, int(renorm), 2.5, ix.data_ptr(), g.data_ptr(), out,
                               ld_g, stream()))
    finish()
    d = d[shift:].view(T, ld_g)
    assert bool((d[:, E:] == 77.0).all())
    return w, ix, d[:, :E]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("type_", [sg.SGEMM_F32, sg.SGEMM_BF16], ids=["f32", "bf16"])
def test_route_with_rows_on_and_off_16_bytes(cuda_device, case, type_):
    """Wide loads and stores and single ones give the same bits; indices, weights and gradients follow the definition.

    Logits on a grid of bfloat16 values, with many equal ones: keys that are logits are compared exactly. Where keys are
    sums in FP32, which of two nearly equal ones is larger is the kernel's to say, and weights and gradients are
    compared for its choice. Tolerances as in test_experts_gpu.py: (E / 2 + 8) 2^-23 relative for weights, that of
    2 scale max |g| for gradients, and a bfloat16 gradient's one rounding."""
    E, k, kind, with_bias, groups, kept, two, renorm = case
    T = 53
    rng = torch.Generator().manual_seed(E + k)
    values = (torch.randn(T, E, generator=rng) * 2).bfloat16().float()
    values[3] = -float("inf")
    values[4, 1:] = -float("inf")
    values[5, :E // 2] = float("nan")
    values[6] = torch.finfo(torch.bfloat16).min
    bias = (torch.randn(E, generator=rng) * 0.1).cuda() if with_bias else None
    g = torch.randn(T, k, generator=rng)
    wide = routed(values.cuda(), E, E, type_, case, bias, g.cuda())
    for ld, ld_g, shift in ((E + 1, E + 3, 0), (E + 8, E + 8, 1)):
        single = routed(values.cuda(), ld, ld_g, type_, case, bias, g.cuda(), shift)
        assert torch.equal(wide[0], single[0]) and torch.equal(wide[1], single[1])
        assert torch.equal(wide[2].view(torch.uint8), single[2].contiguous().view(torch.uint8))
    w, ix, d = (t.cpu() for t in wide)
    L = torch.where(values.isnan(), -float("inf"), values).double()
    if not (with_bias or two):
        _, want_ix = ref.route(L.numpy(), None, kind, groups, kept, two, k, renorm, 2.5)
        assert torch.equal(ix, torch.tensor(want_ix, dtype=torch.int32))
    tol = (E / 2 + 8) * 2.0 ** -23
    for t in range(T):
        at = ix[t][ix[t] >= 0].long()
        assert len(set(at.tolist())) == len(at) and bool((w[t][ix[t] < 0] == 0).all())
        x = L[t].clone().requires_grad_(True)
        if len(at) == 0:
            assert not bool(d[t].any())
            continue
        s = torch.log_softmax(x, 0) if kind == "softmax" else torch.nn.functional.logsigmoid(x)
        v = 2.5 * (torch.softmax(s[at], 0) if renorm else torch.exp(s[at]))
        assert bool(((w[t][ix[t] >= 0].double() - v.detach()).abs() <= tol * v.detach() + 1e-38).all()), t
        grad, = torch.autograd.grad((v * g[t][ix[t] >= 0].double()).sum(), x)
        grad = grad.nan_to_num()
        bound = tol * 2 * 2.5 * float(g.abs().max()) + (grad.abs() * 2.0 ** -8 if type_ == sg.SGEMM_BF16 else 0.0)
        assert bool(((d[t].double() - grad).abs() <= bound + 1e-38).all()), t


# ------------------------------------------------------------------- threads

def test_concurrent_calls_on_separate_streams(cuda_device):
    """Each thread's chain, on a stream of its own, gives the bits that it gives alone."""
    def chain(seed, T, E, k, D, F):
        g = torch.Generator(device="cuda").manual_seed(seed)
        R = T * k
        logits, x = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, D, generator=g, device="cuda")
        W = torch.randn(E, F, D, generator=g, device="cuda")
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
        w, ix, off = new(T, k), new(T, k, dtype=torch.int32), new(E + 1, dtype=torch.int32)
        row, tok = new(T, k, dtype=torch.int32), new(R, dtype=torch.int32)
        q, s, y, out = new(R, D, dtype=FP8), new(D // 128, R), new(R, F), new(T, F)
        qw, sw = new(E, F, D, dtype=FP8), new(E, F // 128, D // 128)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()

        def run():
            st = side.cuda_stream
            codes = [
                sg.sgemm_route(T, E, logits.data_ptr(), 0, E, 0, 0, 1, 1, 0, k, 1, 1.0, w.data_ptr(), ix.data_ptr(), st),
                sg.sgemm_dispatch(T, k, E, ix.data_ptr(), off.data_ptr(), row.data_ptr(), tok.data_ptr(), st),
                sg.sgemm_fp8_quantize_rows(R, D, x.data_ptr(), 0, D, tok.data_ptr(), T, q.data_ptr(), D, s.data_ptr(), R, st),
                sg.sgemm_fp8_quantize_blocks(F, D, W.data_ptr(), 0, D, F * D, 0, qw.data_ptr(), D, F * D, sw.data_ptr(),
                                             D // 128, F // 128 * (D // 128), E, st),
                sg.sgemm_fp8_grouped(E, off.data_ptr(), R, F, D, q.data_ptr(), D, s.data_ptr(), R, qw.data_ptr(), D, F * D,
                                     sw.data_ptr(), D // 128, F // 128 * (D // 128), 0.0, y.data_ptr(), 0, F, st),
                sg.sgemm_combine(T, k, F, R, y.data_ptr(), 0, F, row.data_ptr(), w.data_ptr(), out.data_ptr(), F, st)]
            with torch.cuda.stream(side):
                copies = [t.clone() for t in (w, ix, off, row, tok, out)]
            side.synchronize()
            return codes, copies
        return run

    # The second's pairs take scratch for their counts.
    chains = [chain(1, 24, 8, 2, 256, 384), chain(2, 20000, 16, 7, 128, 256), chain(3, 3000, 64, 4, 256, 128),
              chain(4, 1, 8, 8, 128, 128)]
    alone = [run() for run in chains]
    torch.cuda.synchronize()
    results, errors = [[] for _ in chains], []

    def worker(i):
        try:
            for _ in range(8):
                results[i].append(chains[i]())
        except Exception as e:        # surfaced by the assertion below
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(chains))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    finish()
    assert not errors, errors
    for (codes, want), got in zip(alone, results):
        assert codes == [sg.SGEMM_OK] * 6
        for c, outs in got:
            assert c == codes and all(torch.equal(a, b) for a, b in zip(outs, want))
