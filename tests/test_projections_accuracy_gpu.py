"""How far the sums of the grouped and the 4-bit products are from those in 64
bits, closely enough to notice a missing term or sums that are not taken out of
the tensor core.

An MMA adds its K products (16 of bf16, 64 of 4 bits) to the accumulator and cuts
the sum to fp32, towards zero: at most one step, 2^-23 of it, and 0.58 steps in the
mean square.  With an fp32 result the grouped products take a segment's sum (512,
32 MMAs) out and add it in fp32 to nearest, n / 512 = S additions of half a step at
most.

Positive operands: after i of m equal MMAs the sum is i / m of the last, so m cuts
take off at most (m + 1) / 2 steps of it: 16.5 steps with segments, however many,
and S 2^-24 for the additions.
Operands of either sign: after i MMAs the sum is about sqrt(i / m) of the last, m
cuts take 0.58 2 m / 3 steps where none is undone by another.  Segments' errors
are independent of one another, so those of S of them add up as the segments'
sums do and leave the quotient that one has, 0.58 2 32 / 3 = 12.4 steps; the additions'
errors, 2^-24 sqrt(j / S) each, add up in the same way to at most 2^-24 sqrt(S).
A sum of 4096 that stayed in the tensor core would be 3 to 9 times further off."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

from operator_refs import F32

pytestmark = pytest.mark.gpu
MX, NV = G.FP4_MX, G.FP4_NV
STEP = 2.0 ** -23
SEGMENT = 512


def make(seed, rows, cols, positive):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.rand(rows, cols, generator=g, device="cuda") + 0.5 if positive else \
        torch.randn(rows, cols, generator=g, device="cuda")
    return x.bfloat16()


def check(got, ref, positive, cuts, parts):
    """cuts: MMAs of a sum that the tensor core keeps; parts: such sums added up."""
    d = got.double() - ref
    if positive:
        off = float((d / ref).mean())
        assert abs(off) <= (cuts + 1) / 2 * STEP + parts * STEP / 2, off
    else:
        off = float(d.norm() / ref.norm())
        assert off <= 0.58 * 2 / 3 * cuts * STEP + parts ** 0.5 * STEP / 2, off


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("sizes,N,K", [
    ([3], 256, 4096), ([33], 520, 4096), ([2, 0, 5], 256, 2048), ([1], 264, 1024),      # K split over clusters
    ([3], 256, 4160), ([1], 264, 8192), ([60, 0, 4], 520, 5000),                        # 64-row tiles, unsplit
    ([300, 0, 500, 77], 1032, 4096), ([700, 1300], 4104, 4096), ([129], 264, 20000)])
def test_rows(sizes, N, K, layout, positive):
    M, E = sum(sizes), len(sizes)
    a, w = make(1, M, K, positive), make(2, E * N, K, positive).view(E, N, K)
    b = w if layout == G.KMAJOR else w.transpose(1, 2).contiguous()
    c = torch.empty(M, N, device="cuda")
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    G.gemm_bf16_grouped(a, b, ends, c, E, M, N, K, K, K if layout == G.KMAJOR else N, N * K, N, F32, layout)
    G.gemm_check_device_status()
    ref = torch.cat([x.double() @ w[e].double().t() for e, x in enumerate(a.split(sizes))])
    check(c, ref, positive, SEGMENT // 16, -(-K // SEGMENT))


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("rows,N,K", [(4096, 264, 520), (16384, 264, 520), (5001, 264, 520), (4096, 2056, 2568), (16384, 2056, 2568)])
def test_gradient(rows, N, K, layout, positive):
    """One expert with `rows`, beside smaller ones."""
    sizes = [77, rows, 0, 1000]
    M = sum(sizes)
    d, a = make(3, M, N, positive), make(4, M, K, positive)
    high, wide = (N, K) if layout == G.KMAJOR else (K, N)
    db = torch.empty(4, high, wide, device="cuda")
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    G.gemm_bf16_grouped_wgrad(d, a, ends, db, 4, M, N, K, N, K, wide, high * wide, F32, layout)
    G.gemm_check_device_status()
    for e, (x, y) in enumerate(zip(d.split(sizes), a.split(sizes))):
        ref = x.double().t() @ y.double()
        ref = ref if layout == G.KMAJOR else ref.t()
        if sizes[e] == 0:
            assert not bool(db[e].any())
        else:
            check(db[e], ref, positive, min(SEGMENT, sizes[e]) // 16 + 1, -(-sizes[e] // SEGMENT))


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("form", [MX, NV])
@pytest.mark.parametrize("M,N,K", [(1, 520, 8192), (60, 520, 8192), (200, 520, 8192), (1100, 2056, 8192), (300, 2056, 2048)])
@pytest.mark.parametrize("spread", [0, 3, 12])
def test_4_bits(M, N, K, form, spread, positive):
    """Scales over 2 * spread steps of their type: octaves for MX, eighths for NV
    (three octaves at most).  Widely spread ones make single blocks as large as
    the rest together, at any place: each cut is then of a sum no larger than
    that of the magnitudes."""
    block = 32 if form == MX else 16
    r = np.random.RandomState(M + K + spread)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")

    def operand(rows):
        codes = torch.from_numpy(r.randint(1, 8 if positive else 16, (rows, K))).cuda()
        mid = 127 if form == MX else 64
        scales = torch.from_numpy(r.randint(mid - spread, mid + spread + 1, (rows, K // block))).to(torch.uint8).cuda()
        s = torch.exp2(scales.double() - 127) if form == MX else scales.view(torch.float8_e4m3fn).double()
        T = -(-(K // block) // 4)
        full = torch.zeros(-(-rows // 128) * 128, 4 * T, dtype=torch.uint8, device="cuda")
        full[:rows, :K // block] = scales
        tiled = full.view(-1, 4, 32, T, 4).permute(0, 3, 2, 1, 4).reshape(-1)
        packed = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)
        return packed, tiled, values[codes] * s.repeat_interleave(block, 1)

    (qa, sa, x), (qb, sb, y) = operand(M), operand(N)
    c = torch.empty(M, N, device="cuda")
    G.gemm_fp4(qa, sa, None, qb, sb, None, c, M, N, K, K // 2, K // 2, N, form, F32)
    G.gemm_check_device_status()
    ref, cuts = x @ y.t(), K // 64
    if spread == 0:
        # codes under one scale: multiples of a quarter, below 2^24 of them, so exact
        assert torch.equal(c.double(), ref)
    elif positive:
        off = float(((c.double() - ref) / ref).mean())
        assert abs(off) <= cuts * STEP, off             # each cut at most a step of the whole
    else:
        assert bool(((c.double() - ref).abs() <= cuts * STEP * (x.abs() @ y.abs().t())).all())
