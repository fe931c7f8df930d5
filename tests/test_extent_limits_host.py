"""Pitches and matrices that no address space holds are refused, by every entry
point and for every matrix: the byte offsets that they stand for wrap 64 bits,
so that the other checks (and the kernels) would see a small matrix.  Runs
without a device only, where a call that passes its checks gives 4: the
addresses here are made up."""
import ctypes

import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")

# far apart, 16-byte aligned, never dereferenced
P = [0x7F0000000000 + i * 0x10000000 for i in range(8)]
F32, BF16 = G.OUT_F32, G.OUT_BF16
FLOAT = ctypes.c_float
OK, INVALID, MISALIGNED, ALIAS, TOO_LARGE = 0, 1, 2, 3, 7


def norm(t, M=64, K=128, **ld):
    pitch = [ld.get(n, K) for n in ("x", "r", "h", "y", "q")]
    return G.lib.gemm_rmsnorm(P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], M, K, *pitch, t, t, FLOAT(1e-5), 0)


def back(t, M=64, K=128, **ld):
    pitch = [ld.get(n, K) for n in ("dy", "h", "dr", "dh")]
    return G.lib.gemm_rmsnorm_backward(P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], 1 << 24, M, K, *pitch, t, t, t, 0)


def quant(t, M=64, K=128, layout=G.KMAJOR, **ld):
    return G.lib.gemm_mxfp8_quantize(P[0], P[1], P[2], M, K, ld.get("x", K), ld.get("q", K), t, layout, 0)


def w4(t, M=4, N=64, K=128, **ld):
    pitch = ld.get("a", K), ld.get("b", K // 2), ld.get("s", 16), ld.get("c", N)
    return G.lib.gemm_bf16_w4(P[0], P[1], P[2], P[3], P[4], M, N, K, *pitch, 64, t, 0)


def bf16(t, M=64, N=64, K=64, **ld):
    return G.lib.gemm_bf16(P[0], P[1], P[2], M, N, K, ld.get("a", K), ld.get("b", K), ld.get("c", N), t, 0)


def noalloc(t, M=64, N=64, K=64, **ld):
    return G.lib.gemm_bf16_noalloc(P[0], P[1], P[2], M, N, K, ld.get("a", K), ld.get("b", K), ld.get("c", N), t, 0)


def fused(t, M=64, N=64, K=64, **ld):
    return G.lib.gemm_bf16_fused(P[0], P[1], P[2], M, N, K, ld.get("a", M), ld.get("b", N), ld.get("c", N), t, G.MNMAJOR,
                                 G.MNMAJOR, FLOAT(1), FLOAT(0), P[3], G.ACT_RELU, 0)


def mxfp8(t, M=64, N=64, K=64, **ld):
    return G.lib.gemm_mxfp8(P[0], P[3], P[1], P[4], P[2], M, N, K, ld.get("a", K), ld.get("b", K), ld.get("c", N), 0)


def allgather(t, M=64, N=64, K=64, row0=128, **ld):
    dst = (ctypes.c_void_p * 2)(P[2], P[3])
    return G.lib.gemm_bf16_allgather(P[0], P[1], dst, 2, M, N, K, ld.get("a", K), ld.get("b", K), ld.get("c", N), row0, t, 0)


CALLS = [(norm, ("x", "r", "h", "y", "q")), (back, ("dy", "h", "dr", "dh")), (quant, ("x", "q")),
         (w4, ("a", "b", "s", "c")), (bf16, ("a", "b", "c")), (noalloc, ("a", "b", "c")), (fused, ("a", "b", "c")),
         (mxfp8, ("a", "b", "c")), (allgather, ("a", "b", "c"))]
EACH = [(call, name) for call, names in CALLS for name in names]
IDS = [f"{call.__name__}-{name}" for call, name in EACH]


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("call,name", EACH, ids=IDS)
def test_pitches_whose_bytes_wrap(call, name, t):
    """2^62 + a few elements: 2 or 4 bytes each make 2^63 (a negative number) or
    2^64 (a pitch of a few bytes)."""
    for ld in ((1 << 62) + 16, (1 << 62) + 32, (1 << 63) - 16, (1 << 61) + 16, 1 << 40):
        assert call(t, **{name: ld}) == TOO_LARGE, hex(ld)


@pytest.mark.parametrize("call,name", EACH, ids=IDS)
def test_matrices_whose_byte_range_wraps(call, name):
    """A pitch within the limit, times so many rows that the end of the matrix
    is 2^64 bytes and more behind its start."""
    rows = dict(M=1 << 26, N=1 << 26, K=1 << 26)
    if call in (norm, back, quant):
        rows = dict(M=1 << 26, K=128)
    elif call in (w4, mxfp8):
        rows = dict(M=1 << 20, N=1 << 26, K=128) if call is w4 else dict(M=1 << 26, N=1 << 26, K=128)
    if call is w4 and name in "ac":
        rows = dict(M=1 << 26, N=64, K=128)
    assert call(BF16, **rows, **{name: (1 << 39) - 64}) == TOO_LARGE


def test_slab_offsets_that_wrap():
    assert allgather(F32, row0=(1 << 31) - 65, c=(1 << 37)) == TOO_LARGE
    assert allgather(BF16, row0=(1 << 31) - 65, c=(1 << 62) + 16) == TOO_LARGE


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("call,name", EACH, ids=IDS)
def test_long_pitches_within_the_limits_pass(call, name, t):
    """Just below 2^40 bytes the extent is not what refuses a call: two such
    matrices do not fit between the others' addresses, so that only pitches
    of inputs and of last outputs get past the overlap test."""
    got = call(t, **{name: (1 << 37)})
    assert got in (ALIAS, 4), got


def test_other_statuses_keep_their_order():
    assert norm(F32, x=64) == INVALID and norm(F32, x=130) == MISALIGNED and norm(F32, x=(1 << 62) + 1) == MISALIGNED
    assert bf16(F32, a=32) == INVALID and bf16(F32, a=68) == MISALIGNED and bf16(F32, c=66) == MISALIGNED
    assert bf16(F32, c=(1 << 62) + 1) == MISALIGNED
    assert G.lib.gemm_bf16(P[0], P[1], P[0], 64, 64, 64, 64, 64, 64, F32, 0) == ALIAS
    assert bf16(F32, M=0, c=(1 << 62) + 16) == OK and norm(F32, M=0, x=(1 << 62) + 16) == OK
