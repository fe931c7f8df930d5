"""Products grouped by expert against the formula in 64 bits, group by group:
sizes around every tile and step, empty experts, both layouts of the weights,
types, pitches, NaN beside what counts, rows of no expert.

Tolerance: K fp32 additions in any order, each off by at most one step (2^-23)
of a partial sum no larger than sum |a b|, and half a step of the output's
rounding.  Integer operands whose sums stay below 2^24 have to be exact."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

from operator_refs import BF16, F32, HALF_STEP, TORCH, Buffer, pad

pytestmark = pytest.mark.gpu
STEP32 = 2.0 ** -23


def ints(seed, rows, cols, most=4):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, (rows, cols), generator=g).float()


def normal(seed, rows, cols):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed))


def ends_of(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


class Weights:
    """`groups` matrices rows x cols with a pitch, a stride and guard bytes (NaN) around each."""

    def __init__(self, groups, rows, cols, dtype, fill=None):
        self.groups, self.rows, self.cols = groups, rows, cols
        self.buf = Buffer(groups * (rows + 1), cols, dtype)      # a guard row after every matrix
        self.ld, self.stride = self.buf.ld, (rows + 1) * self.buf.ld
        self.t = self.buf.t.view(groups, rows + 1, self.ld)
        if fill is not None:
            self.t[:, :rows, :cols] = fill.to(dtype).cuda()

    @property
    def ptr(self):
        return self.buf.ptr

    def get(self):
        return self.t[:, :self.rows, :self.cols]

    def guards_ok(self):
        b = self.buf.raw.view(-1, self.ld * self.buf.esize)
        own = self.t[:, :self.rows, :self.cols]
        keep = own.clone()
        own.view(torch.int16 if self.buf.esize == 2 else torch.int32).fill_(-1)
        ok = bool((b == 0xFF).all())
        own.copy_(keep)
        return ok


def run_rows(sizes, N, K, layout, c_type, make, spare=0, seed=0):
    """C, the reference and sum |a b| of a grouped product; rows of no expert are checked here."""
    E, M = len(sizes), int(sum(sizes)) + spare
    a = make(seed, M, K)
    w = make(seed + 1, E * N, K).view(E, N, K)
    A = Buffer(M, K, torch.bfloat16, fill=a)
    B = Weights(E, N, K, torch.bfloat16, w) if layout == G.KMAJOR else \
        Weights(E, K, N, torch.bfloat16, w.transpose(1, 2))
    C = Buffer(M, N, TORCH[c_type])
    ends = ends_of(sizes)
    G.gemm_bf16_grouped(A.ptr, B.ptr, ends, C.ptr, E, M, N, K, A.ld, B.ld, B.stride, C.ld, c_type, layout)
    G.gemm_check_device_status()
    assert C.guards_ok()
    used = M - spare
    assert bool((C.t[used:].contiguous().view(torch.uint8) == 0xFF).all()), "rows of no expert"
    ad, wd = A.t[:, :K].double(), w.bfloat16().double().cuda()
    ref, mag, lo = [], [], 0
    for e, n in enumerate(sizes):
        ref.append(ad[lo:lo + n] @ wd[e].t())
        mag.append(ad[lo:lo + n].abs() @ wd[e].abs().t())
        lo += n
    return C.t[:used, :N].double(), torch.cat(ref), torch.cat(mag)


def check(got, ref, mag, length, c_type):
    tol = length * STEP32 * mag + HALF_STEP[c_type] * ref.abs() + 1e-37
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"


SIZES = [
    [1], [0], [3, 0, 0, 5], [0, 0, 7], [15, 16, 17], [31, 32, 33, 0, 1], [63, 64, 65], [127, 128, 129], [255, 256, 257],
    [300, 1, 0, 511, 513], [1000], [0] * 40 + [2] + [0] * 23, [1] * 100,
]


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}groups_{sum(s)}rows")
def test_rows_exact(sizes, layout):
    for c_type, N, K, spare in ((F32, 264, 136, 0), (BF16, 129, 65, 5)):
        got, ref, mag = run_rows(sizes, N, K, layout, c_type, ints, spare)
        want = ref if c_type == F32 else ref.bfloat16().double()
        assert torch.equal(got, want)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 8), (8, 7), (31, 63), (128, 64), (130, 66), (257, 200), (600, 520)])
def test_rows_odd_sizes(N, K, layout):
    for sizes in ([2, 0, 9], [70, 300, 0, 33]):
        for c_type in (F32, BF16):
            check(*run_rows(sizes, N, K, layout, c_type, normal, 3, N + K), K, c_type)


def test_rows_long_reduction_and_many_tiles():
    check(*run_rows([700, 0, 1300, 48], 2048, 4096, G.KMAJOR, F32, normal), 4096, F32)
    check(*run_rows([700, 0, 1300, 48], 2050, 1000, G.MNMAJOR, BF16, normal), 1000, BF16)
    check(*run_rows([5, 0, 1, 64], 4096, 4096, G.KMAJOR, BF16, normal), 4096, BF16)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("sizes", [[255, 256, 257, 0, 700], [300, 1, 0, 511, 513], [1500], [31, 33, 0, 1000, 97, 129]])
def test_rows_of_many_tiles(sizes, layout):
    """Sizes for which CTA pairs are chosen."""
    check(*run_rows(sizes, 4196, 1000, layout, F32, normal, 3), 1000, F32)
    check(*run_rows(sizes, 4101, 1090, layout, BF16, normal, 0, 4), 1090, BF16)
    got, ref, _ = run_rows(sizes, 5000, 1064, layout, F32, ints, 1)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("M", [1, 3, 16, 33, 64])
@pytest.mark.parametrize("N,K", [(130, 8192), (257, 4100), (1000, 4096), (2049, 2050), (4100, 1030)])
def test_few_rows_with_k_split_over_clusters(M, N, K, layout):
    for c_type in (F32, BF16):
        check(*run_rows([M], N, K, layout, c_type, normal, 1, M), K, c_type)
    got, ref, _ = run_rows([0, M, 0, 0], N, K, layout, F32, ints)
    assert torch.equal(got, ref)


def test_rows_without_reduction():
    for sizes in ([3, 0, 70], [500, 1]):
        M, N = sum(sizes) + 4, 40
        C = Buffer(M, N, torch.float32)
        G.gemm_bf16_grouped(None, None, ends_of(sizes), C.ptr, len(sizes), M, N, 0, 0, 0, 0, C.ld, F32)
        G.gemm_check_device_status()
        assert bool((C.t[:M - 4, :N] == 0).all()) and C.guards_ok()
        assert bool((C.t[M - 4:].contiguous().view(torch.uint8) == 0xFF).all())


@pytest.mark.parametrize("sizes", [[20, 30, 0, 40], [200, 300, 0, 400]])
@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
def test_nan_stays_with_its_expert(sizes, layout):
    """NaN and infinities in one expert's weights, in an expert without rows and
    in rows of no expert reach no other expert's rows; a NaN row only itself."""
    E, N, K = len(sizes), 136, 72
    M = sum(sizes) + 8
    a, w = normal(1, M, K), normal(2, E * N, K).view(E, N, K)
    w[0, 5, 3], w[2] = float("nan"), float("inf")
    a[M - 8:] = float("nan")
    a[sizes[0] + 2, 9] = float("nan")
    A = Buffer(M, K, torch.bfloat16, fill=a)
    B = Weights(E, N, K, torch.bfloat16, w) if layout == G.KMAJOR else \
        Weights(E, K, N, torch.bfloat16, w.transpose(1, 2))
    C = Buffer(M, N, torch.float32)
    G.gemm_bf16_grouped(A.ptr, B.ptr, ends_of(sizes), C.ptr, E, M, N, K, A.ld, B.ld, B.stride, C.ld, F32, layout)
    G.gemm_check_device_status()
    bad = torch.zeros(M - 8, N, dtype=torch.bool)
    bad[:sizes[0], 5] = True
    bad[sizes[0] + 2] = True
    assert torch.equal(torch.isnan(C.get()[:M - 8]), bad)


def run_grad(sizes, N, K, layout, d_type, make, spare=0, seed=0, beta=0.0, old=None):
    E, M = len(sizes), int(sum(sizes)) + spare
    a, d = make(seed, M, K), make(seed + 1, M, N)
    a[M - spare:], d[M - spare:] = float("nan"), float("nan")
    A, D = Buffer(M, K, torch.bfloat16, fill=a), Buffer(M, N, torch.bfloat16, fill=d)
    high, wide = (N, K) if layout == G.KMAJOR else (K, N)
    W = Weights(E, high, wide, TORCH[d_type], old)
    G.gemm_bf16_grouped_wgrad(D.ptr, A.ptr, ends_of(sizes), W.ptr, E, M, N, K, D.ld, A.ld, W.ld, W.stride, d_type, layout,
                              beta)
    G.gemm_check_device_status()
    assert W.guards_ok()
    ad, dd = A.t[:, :K].double(), D.t[:, :N].double()
    ref, mag, lo = [], [], 0
    for n in sizes:
        x, y = ad[lo:lo + n], dd[lo:lo + n]
        if layout == G.KMAJOR:
            x, y = y, x
        ref.append(x.t() @ y)
        mag.append(x.abs().t() @ y.abs())
        lo += n
    return W.get().double(), torch.stack(ref), torch.stack(mag)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("sizes", SIZES + [[1, 2, 3, 4, 5, 6, 7, 8], [49, 64, 79, 80, 81]],
                         ids=lambda s: f"{len(s)}groups_{sum(s)}rows")
def test_gradient_exact(sizes, layout):
    for d_type, N, K, spare in ((F32, 136, 264, 0), (BF16, 65, 129, 5)):
        got, ref, mag = run_grad(sizes, N, K, layout, d_type, ints, spare)
        want = ref if d_type == F32 else ref.bfloat16().double()
        assert torch.equal(got, want)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 8), (8, 7), (63, 31), (64, 128), (66, 130), (200, 257), (520, 600)])
def test_gradient_odd_sizes(N, K, layout):
    for sizes in ([2, 0, 9], [70, 300, 0, 33]):
        for d_type in (F32, BF16):
            check(*run_grad(sizes, N, K, layout, d_type, normal, 3, N + K), max(sizes), d_type)


def test_gradient_long_reduction_and_many_tiles():
    check(*run_grad([5000, 0, 1301], 1024, 700, G.KMAJOR, F32, normal), 5000, F32)
    check(*run_grad([77] * 30 + [0] * 5, 700, 520, G.MNMAJOR, BF16, normal), 77, BF16)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("sizes", [[255, 256, 257, 0, 700], [300, 1, 0, 511, 513], [31, 33, 0, 1000, 97, 129]])
def test_gradient_of_many_tiles(sizes, layout):
    """Sizes for which CTA pairs are chosen."""
    check(*run_grad(sizes, 4196, 2100, layout, F32, normal, 3), max(sizes), F32)
    check(*run_grad(sizes, 3001, 4101, layout, BF16, normal, 0, 4), max(sizes), BF16)
    old = ints(9, len(sizes) * 4000, 2500).view(len(sizes), 4000, 2500)
    if layout == G.KMAJOR:
        got, ref, _ = run_grad(sizes, 4000, 2500, layout, F32, ints, 1, 2, 1.0, old)
        assert torch.equal(got, ref + old.double().cuda())


@pytest.mark.parametrize("d_type", [F32, BF16])
@pytest.mark.parametrize("beta", [1.0, 0.5])
def test_gradient_is_added(d_type, beta):
    sizes, N, K = [40, 0, 131], 65, 137
    old = normal(9, 3 * N, K).view(3, N, K).to(TORCH[d_type]).float()
    got, ref, mag = run_grad(sizes, N, K, G.KMAJOR, d_type, normal, 2, 5, beta, old)
    ref = ref + beta * old.double().cuda()
    check(got, ref, mag + old.abs().double().cuda(), max(sizes) + 1, d_type)
    assert torch.equal(got[1], (beta * old[1].double()).cuda())          # exact: no product, beta a power of two


def test_gradient_without_rows():
    W = Weights(3, 20, 24, torch.float32, torch.full((3, 20, 24), 2.0))
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    G.gemm_bf16_grouped_wgrad(None, None, ends, W.ptr, 3, 0, 20, 24, 0, 0, W.ld, W.stride, F32, G.KMAJOR, 1.0)
    assert bool((W.get() == 2.0).all())
    G.gemm_bf16_grouped_wgrad(None, None, ends, W.ptr, 3, 0, 20, 24, 0, 0, W.ld, W.stride, F32)
    G.gemm_check_device_status()
    assert bool((W.get() == 0.0).all()) and W.guards_ok()


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("N,K", [(72, 136), (4200, 4200)])       # single CTAs, pairs
def test_gradient_nan_stays_with_its_expert(N, K, layout):
    sizes = [37, 0, 50, 13, 90]
    M = sum(sizes)
    a, d = normal(1, M, K), normal(2, M, N)
    a[87:100] = float("nan")            # all of expert 3's rows
    d[87:100] = float("inf")
    A, D = Buffer(M, K, torch.bfloat16, fill=a), Buffer(M, N, torch.bfloat16, fill=d)
    high, wide = (N, K) if layout == G.KMAJOR else (K, N)
    W = Weights(5, high, wide, torch.float32)
    G.gemm_bf16_grouped_wgrad(D.ptr, A.ptr, ends_of(sizes), W.ptr, 5, M, N, K, D.ld, A.ld, W.ld, W.stride, F32, layout)
    G.gemm_check_device_status()
    bad = torch.isnan(W.get())
    assert bool(bad[3].all()) and not bool(bad[[0, 1, 2, 4]].any())


@pytest.mark.parametrize("ends", [[1 << 30, 50, 60], [-5, 10, 1000], [30, 10, 40], [-(1 << 31), -1, 0], [40, 0, 40],
                                  [40, 0, 40] * 20, [5, 3, 9, 8, 8, 100, 7]])
def test_ends_are_made_to_rise_within_the_buffer(ends):
    """An end past M counts as M, below 0 as 0, below an earlier one as that one."""
    M, N, K, E = 40, 24, 16, len(ends)
    fixed = np.maximum.accumulate(np.clip(ends, 0, M))
    sizes = np.diff(np.concatenate([[0], fixed])).tolist()
    a, w, d = ints(1, M, K), ints(2, E * N, K), ints(3, M, N)
    A, D = Buffer(M, K, torch.bfloat16, fill=a), Buffer(M, N, torch.bfloat16, fill=d)
    B, C, W = Weights(E, N, K, torch.bfloat16, w.view(E, N, K)), Buffer(M, N, torch.float32), Weights(E, N, K, torch.float32)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    G.gemm_bf16_grouped(A.ptr, B.ptr, e, C.ptr, E, M, N, K, A.ld, B.ld, B.stride, C.ld)
    G.gemm_bf16_grouped_wgrad(D.ptr, A.ptr, e, W.ptr, E, M, N, K, D.ld, A.ld, W.ld, W.stride)
    G.gemm_check_device_status()
    assert C.guards_ok() and W.guards_ok()
    lo = 0
    for i, n in enumerate(sizes):
        assert torch.equal(C.get()[lo:lo + n], a[lo:lo + n] @ w.view(E, N, K)[i].t())
        assert torch.equal(W.get()[i].cpu(), d[lo:lo + n].t() @ a[lo:lo + n])
        lo += n
    assert bool((C.t[lo:].contiguous().view(torch.uint8) == 0xFF).all())


def test_same_bits_every_time():
    sizes = [100, 3, 0, 400]
    for run in (lambda: run_rows(sizes, 300, 500, G.KMAJOR, F32, normal)[0],
                lambda: run_grad(sizes, 300, 500, G.MNMAJOR, F32, normal)[0]):
        first = run()
        for _ in range(3):
            assert torch.equal(run(), first)


def test_offsets_past_32_bits():
    """Rows of C, of A and matrices of dB that lie more than 2^32 bytes from the first."""
    M, N, K, ld = 70000, 64, 64, 1 << 15
    sizes = [69000, 0, 1000]
    C = torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")
    a, w = ints(1, M, K).bfloat16().cuda(), ints(2, 3 * N, K).bfloat16().cuda()
    G.gemm_bf16_grouped(a, w, ends_of(sizes), C, 3, M, N, K, K, K, N * K, ld, BF16)
    G.gemm_check_device_status()
    w = w.view(3, N, K)
    assert torch.equal(C[:69000, :N].float(), (a[:69000].float() @ w[0].float().t()).bfloat16().float())
    assert torch.equal(C[69000:, :N].float(), (a[69000:].float() @ w[2].float().t()).bfloat16().float())
    assert not bool(C[:, N:].any())
    stride = 1 << 30
    dB = torch.zeros(3 * stride, dtype=torch.float32, device="cuda")
    G.gemm_bf16_grouped_wgrad(C, a, ends_of(sizes), dB, 3, M, N, K, ld, K, K, stride)
    G.gemm_check_device_status()
    want = C[69000:, :N].double().t() @ a[69000:].double()
    got = dB[2 * stride:2 * stride + N * K].view(N, K).double()
    mag = C[69000:, :N].double().abs().t() @ a[69000:].double().abs()
    check(got, want, mag, 1000, F32)
    assert not bool(dB[stride:2 * stride].any())
