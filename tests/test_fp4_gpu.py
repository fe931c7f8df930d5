"""4-bit floating point against its definition in 64 bits: the quantiser's codes
and scales bit for bit, and products of arbitrary codes and scales.

The quantiser rounds 6 g, s g and the quotients to fp32 before it rounds them to
E4M3 and E2M1; the reference does the same from 64-bit values (a quotient of two
fp32 numbers in 64 bits, rounded to fp32, is the rounded quotient: 53 >= 2 * 24 +
2).  Products: exact terms, K fp32 additions in any order, each off by at most
one step (2^-23) of a partial sum no larger than sum |a b|; then times ga gb (two
roundings to fp32: at most one more step) and half a step of the output."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

from operator_refs import BF16, F32, HALF_STEP, TORCH, Buffer

pytestmark = pytest.mark.gpu
MX, NV = G.FP4_MX, G.FP4_NV
BLOCK = {MX: 32, NV: 16}
STEP32 = 2.0 ** -23
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def scale_values(byte, form):
    if form == MX:
        return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return torch.from_numpy(byte.astype(np.uint8)).view(torch.float8_e4m3fn).double().numpy()


def untile(sf, rows, K, form):
    """[rows, blocks] scale bytes, by the documented index, and the whole rows' padded bytes."""
    blocks = K // BLOCK[form]
    T = -(-blocks // 4)
    i, b = np.arange(rows)[:, None], np.arange(4 * T)[None, :]
    full = sf[512 * (i // 128 * T + b // 4) + 16 * (i % 32) + 4 * (i % 128 // 32) + b % 4]
    return full[:, :blocks], full[:, blocks:]


def tile(scales, form, pad=0):
    rows, blocks = scales.shape
    T = -(-blocks // 4)
    out = np.full(512 * -(-rows // 128) * T, 0xFF, np.uint8)        # rows past the last: NaN
    full = np.full((rows, 4 * T), pad, np.uint8)
    full[:, :blocks] = scales
    i, b = np.arange(rows)[:, None], np.arange(4 * T)[None, :]
    out[512 * (i // 128 * T + b // 4) + 16 * (i % 32) + 4 * (i % 128 // 32) + b % 4] = full
    return out


def nearest_code(q):
    """E2M1 codes of q: the nearest value, ties to the even code."""
    a = np.abs(q)[..., None]
    d = np.abs(np.minimum(a, 6.0) - VALUES[:8])
    low = d.min(-1, keepdims=True)
    tied = d == low
    even = tied & (np.arange(8) % 2 == 0)
    code = np.where(tied.sum(-1) > 1, even.argmax(-1), tied.argmax(-1))
    return (code + 8 * np.signbit(q)).astype(np.uint8)


def reference_quantise(x, g, form):
    """x: fp64 of fp32 values, finite.  Codes [rows, K] and scale bytes [rows, blocks]."""
    b = x.reshape(x.shape[0], -1, BLOCK[form])
    top = np.abs(b).max(2)
    def f32(v):
        with np.errstate(over="ignore"):
            return v.astype(np.float32).astype(np.float64)

    if form == MX:
        byte = np.searchsorted(6.0 * 2.0 ** np.arange(-127, 128, dtype=np.float64), top, side="left")
        q = b * 2.0 ** (127.0 - byte)[:, :, None]
    else:
        t = f32(top / f32(np.float64(6.0) * g))
        s = torch.from_numpy(np.clip(t, 2.0 ** -9, 448).astype(np.float32)).to(torch.float8_e4m3fn)
        byte = s.view(torch.uint8).numpy()
        q = b / f32(s.double().numpy() * g)[:, :, None]
        q = f32(np.clip(q, -1e30, 1e30))
    return nearest_code(q).reshape(x.shape), byte.astype(np.uint8)


def quantise(x, form, x_type, layout, g):
    """Runs the quantiser on the fp32 tensor x (M x K); returns codes, scale bytes, padding bytes, and x as stored."""
    M, K = x.shape
    X = Buffer(M, K, TORCH[x_type], fill=x) if layout == G.KMAJOR else Buffer(K, M, TORCH[x_type], fill=x.t())
    Q = Buffer(M, K // 2, torch.uint8)
    n = G.gemm_fp4_scale_bytes(M, K, form)
    sf = torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.tensor([g], device="cuda") if g is not None else None
    G.gemm_fp4_quantize(X.ptr, scale, Q.ptr, sf, M, K, X.ld, Q.ld, form, x_type, layout)
    torch.cuda.synchronize()
    assert Q.guards_ok()
    q = Q.get().numpy()
    codes = np.stack((q & 15, q >> 4), 2).reshape(M, K)
    scales, pads = untile(sf.cpu().numpy(), M, K, form)
    stored = X.get() if layout == G.KMAJOR else X.get().t()
    return codes, scales, pads, stored.double().numpy()


FORMS = [(MX, None), (NV, None), (NV, 0.0081), (NV, 1.0)]


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("form,g", FORMS)
def test_quantiser_matches_its_definition(form, g, x_type, layout):
    for M, K in ((1, 32), (1, 8192), (3, 64), (31, 96), (33, 160), (64, 128), (65, 288), (130, 1056), (257, 2080), (2000, 512)):
        gen = torch.Generator().manual_seed(M + K)
        x = torch.randn(M, K, generator=gen) * torch.exp(2 * torch.randn(M, 1, generator=gen))
        x[M // 2, :32] = 0.0
        codes, scales, pads, stored = quantise(x, form, x_type, layout, g)
        want, byte = reference_quantise(stored, np.float64(np.float32(1.0 if g is None else g)), form)
        assert np.array_equal(scales, byte), (M, K)
        assert np.array_equal(codes, want), (M, K)
        assert not pads.any(), "bytes past a row's last block"


@pytest.mark.parametrize("form", [MX, NV])
def test_quantiser_at_ties_and_borders(form):
    """Values on and beside every border between codes, for scales that are powers
    of two and others; maxima on and beside 6 * 2^e; tiny and huge values."""
    rows = []
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for unit in (1.0, 1.125, 1.75, 2.0 ** -20, 2.0 ** 30 * 1.5):
        t = np.concatenate([border, np.nextafter(border.astype(np.float32), np.float32(0)).astype(np.float64),
                            np.nextafter(border.astype(np.float32), np.float32(9)).astype(np.float64)]) * unit
        t = np.concatenate([t, -t])
        for lo in range(0, 48, 15):
            part = t[lo:lo + 15]
            part = np.concatenate([part, np.zeros(15 - len(part)), [6.0 * unit]])
            rows.append(np.concatenate([part, part]))
    for top in (6.0, 6.03125, 5.96875, 6.375, 448 * 6, 500 * 6, 3e38, 1e-38, 1e-42, 0.0117, 0.005):
        rows.append(np.full(32, top) * np.linspace(-1, 1, 32))
    for unit in (float(np.nextafter(np.float32(0.25), np.float32(0))), 1e-20, 1e20):      # ties of those g as well
        for s in (1.0, 1.125, 1.875):
            t = np.concatenate([border[:7], -border[:7], [6.0, 0.0]]) * unit * s
            rows.append(np.concatenate([t, t]))
    x = torch.from_numpy(np.array(rows)).float()
    ones = float(np.nextafter(np.float32(0.25), np.float32(0)))      # a mantissa of ones, as s g has it for s a power of two
    sixth = float(np.float32(np.nextafter(np.float32(1), np.float32(0)) / 6))
    assert np.float32(6) * np.float32(sixth) == np.nextafter(np.float32(1), np.float32(0))
    for x_type in (F32, BF16):
        for g in ((None,) if form == MX else (None, 0.37, ones, sixth, 1e-20, 1e20)):
            codes, scales, _, stored = quantise(x, form, x_type, G.KMAJOR, g)
            want, byte = reference_quantise(stored, np.float64(np.float32(1.0 if g is None else g)), form)
            assert np.array_equal(scales, byte)
            # as values: 8 and 0 are both zero (a quotient below fp32's normal range may lose its sign)
            assert np.array_equal(VALUES[codes], VALUES[want])


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("form", [MX, NV])
def test_quantiser_marks_blocks_that_are_not_finite(form, x_type, layout):
    x = torch.ones(5, 128)
    x[0, 3], x[1, 40], x[2, 127], x[4, 64] = float("nan"), float("inf"), -float("inf"), -float("nan")
    codes, scales, _, stored = quantise(x, form, x_type, layout, None)
    bad = ~np.isfinite(stored).reshape(5, -1, BLOCK[form]).all(2)
    assert np.array_equal(scales == (0xFF if form == MX else 0x7F), bad)
    clean = np.where(np.isfinite(stored), stored, 0.0)
    want, byte = reference_quantise(clean, 1.0, form)
    assert np.array_equal(scales[~bad], byte[~bad])
    keep = ~np.repeat(bad, BLOCK[form], 1)
    assert np.array_equal(codes[keep], want[keep])


def operand(seed, rows, K, form, spread=6):
    """Random codes and scales: [rows, K] codes, [rows, blocks] bytes."""
    r = np.random.RandomState(seed)
    codes = r.randint(0, 16, (rows, K)).astype(np.uint8)
    mid = 127 if form == MX else 56
    return codes, r.randint(mid - spread, mid + spread + 1, (rows, K // BLOCK[form])).astype(np.uint8)


def values(codes, scales, form):
    return torch.from_numpy(VALUES[codes] * np.repeat(scale_values(scales, form), BLOCK[form], 1)).cuda()


def put(codes):
    rows, K = codes.shape
    packed = torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4)
    return Buffer(rows, K // 2, torch.uint8, fill=packed)


def product(M, N, K, form, c_type, a, b, g=(None, None), pad=0):
    A, B, C = put(a[0]), put(b[0]), Buffer(M, N, TORCH[c_type])
    sa, sb = (torch.from_numpy(tile(s, form, pad)).cuda() for s in (a[1], b[1]))
    ga, gb = (torch.tensor([v], device="cuda") if v is not None else None for v in g)
    G.gemm_fp4(A.ptr, sa, ga, B.ptr, sb, gb, C.ptr, M, N, K, A.ld, B.ld, C.ld, form, c_type)
    G.gemm_check_device_status()
    assert C.guards_ok()
    return C.t[:, :N].double()


def check_product(M, N, K, form, c_type, seed=0, g=(None, None)):
    a, b = operand(seed, M, K, form), operand(seed + 1, N, K, form)
    got = product(M, N, K, form, c_type, a, b, g)
    x, y = values(*a, form), values(*b, form)
    scale = np.float64(np.float32(1.0 if g[0] is None else g[0])) * np.float64(np.float32(1.0 if g[1] is None else g[1]))
    ref, mag = x @ y.t() * scale, x.abs() @ y.abs().t() * abs(scale)
    bad = ~((got - ref).abs() <= (K + 1) * STEP32 * mag + HALF_STEP[c_type] * ref.abs() + 1e-37)
    assert not bool(bad.any()), f"{int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"


ROWS = [1, 2, 8, 15, 16, 17, 31, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257, 300, 513]


@pytest.mark.parametrize("form", [MX, NV])
@pytest.mark.parametrize("M", ROWS)
def test_product_rows(M, form):
    check_product(M, 264, 512, form, F32, M)
    check_product(M, 129, 2080, form, BF16, M)


@pytest.mark.parametrize("form", [MX, NV])
@pytest.mark.parametrize("N,K", [(1, 32), (2, 64), (7, 96), (31, 128), (33, 160), (127, 224), (130, 256), (257, 288), (600, 3200)])
def test_product_odd_sizes(N, K, form):
    for M in (3, 70, 260):
        for c_type in (F32, BF16):
            check_product(M, N, K, form, c_type, N + K)


@pytest.mark.parametrize("form", [MX, NV])
def test_product_large(form):
    check_product(1, 8192, 8192, form, BF16)
    check_product(64, 4096, 4096, form, F32)
    check_product(16, 4200, 8192, form, F32)
    check_product(2500, 2300, 2016, form, F32)
    check_product(4096, 4096, 1024, form, BF16)
    check_product(300, 20000, 512, form, BF16)


def test_product_under_scales_of_the_matrices():
    for M in (5, 100, 5000):
        check_product(M, 520, 544, NV, F32, 1, (0.0081, 0.0021))
        check_product(M, 520, 544, NV, BF16, 1, (None, 3.7))


@pytest.mark.parametrize("form", [MX, NV])
@pytest.mark.parametrize("M", [4, 90, 5000])
def test_nan_scale_makes_its_row_nan(form, M):
    N, K = 260, 576
    a, b = operand(1, M, K, form), operand(2, N, K, form)
    a[1][M // 2, 1] = b[1][77, 3] = 0xFF if form == MX else 0x7F
    got = product(M, N, K, form, F32, a, b)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[M // 2] = True
    want[:, 77] = True
    assert torch.equal(torch.isnan(got), want)


def test_product_exact_integers():
    """Whole codes and scales of one: every partial sum is exact."""
    for form, one in ((MX, 127), (NV, 56)):
        for M, N, K in ((1, 300, 4096), (37, 130, 1056), (128, 128, 256), (700, 500, 4128), (3000, 3000, 544)):
            r = np.random.RandomState(M)
            a, b = (r.choice([0, 2, 4, 5, 6, 7, 10, 12, 13], (n, K)).astype(np.uint8) for n in (M, N))
            s = lambda n: np.full((n, K // BLOCK[form]), one, np.uint8)
            got = product(M, N, K, form, F32, (a, s(M)), (b, s(N)))
            x, y = (torch.from_numpy(VALUES[v]).cuda() for v in (a, b))
            assert torch.equal(got, x @ y.t())


def test_product_without_reduction():
    C = Buffer(5, 40, torch.bfloat16)
    G.gemm_fp4(None, None, None, None, None, None, C.ptr, 5, 40, 0, 0, 0, C.ld, MX, BF16)
    assert bool((C.get() == 0).all()) and C.guards_ok()


@pytest.mark.parametrize("form", [MX, NV])
def test_same_bits_every_time(form):
    for M in (1, 64, 150, 3000):
        a, b = operand(1, M, 2048, form), operand(2, 700, 2048, form)
        first = product(M, 700, 2048, form, F32, a, b)
        for _ in range(3):
            assert torch.equal(product(M, 700, 2048, form, F32, a, b), first)
