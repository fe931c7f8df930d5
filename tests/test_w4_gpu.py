"""gemm_bf16_w4 against its formula in 64 bits.

Tolerance per element: a group's products are exact and added by at most 16
tensor instructions, each of which may lose up to 2^-22 of the magnitudes
that it adds (it aligns and truncates); the groups and the shares of K are
then added with one rounding each.  With S = sum |a s (q - z)|:
(16 * 2^-22 + (K / 32 + 8) 2^-24) S, plus half a step of the output's type.
"""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from operator_refs import BF16, F32, HALF_STEP, TORCH, U32, Buffer, normal, pad, w4_reference

pytestmark = pytest.mark.gpu


def operands(M, N, K, group, zeros, seed, ints=False):
    g = np.random.default_rng(seed)
    groups = -(-K // group)
    a = torch.from_numpy(g.integers(-4, 5, (M, K)).astype(np.float32)) if ints else normal(seed, M, K)
    A = Buffer(M, K, torch.bfloat16, fill=a)
    B = Buffer(N, K // 2, torch.uint8, fill=torch.from_numpy(g.integers(0, 256, (N, K // 2), dtype=np.uint8)))
    s = 2.0 ** g.integers(-2, 3, (N, groups)) if ints else 0.02 * np.exp(0.3 * g.standard_normal((N, groups)))
    S = Buffer(N, groups, torch.bfloat16, ld=pad(groups, 16) + 16, fill=torch.from_numpy(s.astype(np.float32)))
    Z = Buffer(N, groups, torch.uint8, ld=S.ld, fill=torch.from_numpy(g.integers(0, 16, (N, groups), dtype=np.uint8))) \
        if zeros else None
    return A, B, S, Z


def reference(A, B, S, Z, group, K):
    z = Z.get().numpy().astype(np.float64) if Z is not None else np.full((S.rows, S.cols), 8.0)
    return w4_reference(A.f64(), B.get().numpy(), S.f64(), z, group, K)


def run(M, N, K, group, zeros=True, ct=F32, seed=0, ints=False, stream=None):
    A, B, S, Z = operands(M, N, K, group, zeros, seed, ints)
    C = Buffer(M, N, TORCH[ct])
    G.gemm_bf16_w4(A.ptr, B.ptr, S.ptr, Z.ptr if zeros else None, C.ptr, M, N, K, A.ld, B.ld, S.ld, C.ld, group, ct,
                   stream=stream)
    torch.cuda.synchronize()
    for b in (A, B, S, Z, C):
        assert b is None or b.guards_ok()
    want, mag = reference(A, B, S, Z, group, K)
    got = C.f64()
    if ints:
        assert np.array_equal(got, want)          # every partial sum is a multiple of 1/4 below 2^22
    else:
        tol = mag * (16 * 2.0 ** -22 + (K / 32 + 8) * U32) + np.abs(want) * HALF_STEP[ct] + 1e-37
        assert np.all(np.abs(got - want) <= tol)
    return C


SHAPES = [(1, 1, 32), (1, 7, 64), (2, 128, 256), (3, 129, 288), (5, 300, 512), (8, 127, 800), (9, 256, 1024),
          (16, 1000, 2048), (17, 130, 544), (31, 260, 1312), (32, 128, 4096), (33, 200, 992), (64, 384, 2080),
          (65, 129, 256), (130, 140, 1056)]


@pytest.mark.parametrize("group", [32, 64, 128, 256, 1024])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes_and_groups(M, N, K, group):
    run(M, N, K, group, seed=M + N)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("ct", [F32, BF16])
@pytest.mark.parametrize("M", [1, 8, 12, 30, 50])
def test_outputs_and_zeros(M, ct, zeros):
    run(M, 257, 1536, 128, zeros, ct, seed=M)


@pytest.mark.parametrize("group", [32, 64, 128, 512, 1 << 20])
@pytest.mark.parametrize("M", [1, 10, 25, 70])
def test_integers_exactly(M, group):
    run(M, 200, 1440, group, seed=M, ints=True)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 8192, 8192), (4, 50, 16384), (1, 20000, 1024), (33, 3000, 4000)])
def test_larger_shapes(M, N, K):
    run(M, N, K, 128, seed=3)


def test_long_k_restages_the_activations():
    run(8, 130, 40960, 64, seed=4)
    run(64, 130, 20480, 128, seed=5)


def test_a_row_does_not_depend_on_the_batch():
    """The same activation row gives the same bits at any place of a batch of
    one size."""
    M, N, K = 8, 300, 1024
    A, B, S, Z = operands(M, N, K, 64, True, 6)
    C1, C2 = Buffer(M, N, torch.float32), Buffer(M, N, torch.float32)
    G.gemm_bf16_w4(A.ptr, B.ptr, S.ptr, Z.ptr, C1.ptr, M, N, K, A.ld, B.ld, S.ld, C1.ld, 64)
    A.t[:] = A.t.flip(0).clone()
    G.gemm_bf16_w4(A.ptr, B.ptr, S.ptr, Z.ptr, C2.ptr, M, N, K, A.ld, B.ld, S.ld, C2.ld, 64)
    assert torch.equal(C1.get(), C2.get().flip(0))


def test_nan_and_infinity_stay_in_their_row_of_c():
    M, N, K = 9, 140, 512
    A, B, S, Z = operands(M, N, K, 128, True, 7)
    A.t[2, 100] = float("nan")
    A.t[5, 7] = float("inf")
    S.t[33, 1] = float("nan")
    C = Buffer(M, N, torch.float32)
    G.gemm_bf16_w4(A.ptr, B.ptr, S.ptr, Z.ptr, C.ptr, M, N, K, A.ld, B.ld, S.ld, C.ld, 128)
    got = C.f64()
    assert np.isnan(got[2]).all() and np.isnan(got[:, 33]).all() and not np.isfinite(got[5]).any()
    rest = np.delete(np.delete(got, [2, 5], axis=0), 33, axis=1)
    assert np.isfinite(rest).all()


def test_k_zero_writes_zeros():
    C = Buffer(5, 70, torch.float32)
    G.gemm_bf16_w4(None, None, None, None, C.ptr, 5, 70, 0, 0, 0, 0, C.ld, 64)
    assert np.all(C.f64() == 0) and C.guards_ok()


def test_offsets_past_32_bits():
    """Weight rows 2^25 bytes apart: the last of 130 is 4.3e9 bytes in."""
    M, N, K, ldb = 2, 130, 256, 1 << 25
    A, B, S, Z = operands(M, N, K, 128, True, 8)
    far = torch.empty((N - 1) * ldb + 128, dtype=torch.uint8, device="cuda")
    for j in range(N):
        far[j * ldb:j * ldb + 128] = B.t[j, :128]
    C = Buffer(M, N, torch.float32)
    G.gemm_bf16_w4(A.ptr, far, S.ptr, Z.ptr, C.ptr, M, N, K, A.ld, ldb, S.ld, C.ld, 128)
    want, mag = reference(A, B, S, Z, 128, K)
    assert np.all(np.abs(C.f64() - want) <= mag * 2.0 ** -17)


def test_concurrent_streams_and_graph_replay():
    M, N, K = 4, 1024, 2048
    A, B, S, Z = operands(M, N, K, 128, True, 9)
    want = run(M, N, K, 128, seed=9).get()
    streams = [torch.cuda.Stream() for _ in range(3)]
    Cs = [Buffer(M, N, torch.float32) for _ in streams]
    torch.cuda.synchronize()
    call = lambda C, st: G.gemm_bf16_w4(A.ptr, B.ptr, S.ptr, Z.ptr, C.ptr, M, N, K, A.ld, B.ld, S.ld, C.ld, 128,  # noqa: E731
                                        stream=st)
    for _ in range(5):
        for C, st in zip(Cs, streams):
            call(C, st)
    torch.cuda.synchronize()
    assert all(torch.equal(C.get(), want) for C in Cs)
    graph = torch.cuda.CUDAGraph()
    C = Buffer(M, N, torch.float32)
    with torch.cuda.graph(graph):
        call(C, None)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(C.get(), want)
