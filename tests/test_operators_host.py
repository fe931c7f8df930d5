"""The operators around the products on the host: every documented refusal
gives its status before anything is queued, empty problems succeed, and the
workspace size is the documented one.  No kernel is launched here."""
import ctypes

import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

# far apart, 16-byte aligned, never dereferenced
X, R, H, W, Y, Q, SF, RS = (0x7F0000000000 + i * 0x10000000 for i in range(8))
F32, BF16 = G.OUT_F32, G.OUT_BF16


def norm(X=X, R=R, H=H, W=W, Y=Y, Q=Q, SF=SF, RS=RS, M=64, K=128, ldx=None, ldr=None, ldh=None, ldy=None, ldq=None,
         xt=BF16, ht=BF16, eps=1e-5):
    lds = [K if v is None else v for v in (ldx, ldr, ldh, ldy, ldq)]
    return G.lib.gemm_rmsnorm(X, R, H, W, Y, Q, SF, RS, M, K, *lds, xt, ht, ctypes.c_float(eps), 0)


def test_rmsnorm_refuses_bad_arguments():
    assert norm(M=-1) == 1 and norm(K=-1) == 1
    assert norm(xt=2) == 1 and norm(ht=-1) == 1
    assert norm(R=0, H=0, ht=9, M=0) == 0                 # without R, h_type is not looked at
    assert norm(eps=0.0) == 1 and norm(eps=-1.0) == 1 and norm(eps=float("nan")) == 1
    assert norm(X=0) == 1 and norm(W=0) == 1
    assert norm(Y=0, Q=0) == 1                             # no output
    assert norm(R=0) == 1                                  # H without R
    assert norm(SF=0) == 1                                 # codes without scales
    assert norm(K=120, ldq=128) == 1                       # codes need K % 32 == 0
    assert norm(ldx=64) == 1 and norm(ldr=64) == 1 and norm(ldh=64) == 1 and norm(ldy=64) == 1 and norm(ldq=64) == 1
    assert norm(X=X + 8) == 2 and norm(W=W + 4) == 2 and norm(RS=RS + 2) == 2 and norm(Y=Y + 2) == 2
    assert norm(ldx=132) == 2 and norm(ldq=136) == 2       # pitches of 264 and 136 bytes
    assert norm(M=1 << 31) == 7 and norm(K=1 << 31) == 7
    assert norm(ldx=1 << 40) == 7


def test_rmsnorm_refuses_overlaps():
    span = 64 * 128 * 2
    assert norm(H=X) == 3 and norm(Y=X + span - 16) == 3 and norm(Q=Y + 16) == 3
    assert norm(SF=Q + 64) == 3 and norm(RS=SF) == 3 and norm(Y=W) == 3
    assert norm(H=R, ldh=136) == 3                         # in place needs the same pitch
    assert norm(H=R + 256) == 3                            # shifted by a row


def back(dY=X, H=H, W=W, RS=RS, dR=R, dH=Y, dW=Q, ws=SF, bytes_=None, M=64, K=128, ld=None, yt=BF16, ht=BF16, dt=BF16,
         lddh=None):
    ld = K if ld is None else ld
    bytes_ = G.gemm_rmsnorm_backward_workspace(M, K) if bytes_ is None else bytes_
    return G.lib.gemm_rmsnorm_backward(dY, H, W, RS, dR, dH, dW, ws, bytes_, M, K, ld, ld, ld,
                                       ld if lddh is None else lddh, yt, ht, dt, 0)


def test_rmsnorm_backward_refuses_bad_arguments():
    assert back(M=-1) == 1 and back(K=-1) == 1 and back(M=1 << 31) == 7
    assert back(yt=3) == 1 and back(ht=3) == 1 and back(dt=3) == 1
    assert back(dY=0) == 1 and back(H=0) == 1 and back(W=0) == 1 and back(RS=0) == 1 and back(dH=0) == 1
    assert back(ws=0) == 1                                 # dW wants a workspace
    assert back(bytes_=G.gemm_rmsnorm_backward_workspace(64, 128) - 1) == 1
    assert back(ws=SF + 8) == 2 and back(dW=Q + 4) == 2 and back(W=W + 4) == 2 and back(RS=RS + 1) == 2
    assert back(ld=100) == 1 and back(ld=132) == 2
    assert back(dH=H) == 3                                 # H is read by no other name
    assert back(dH=X, dt=F32) == 3                         # in place needs the same type size
    assert back(dH=X, lddh=136) == 3
    assert back(dW=X) == 3 and back(ws=H) == 3 and back(ws=Q) == 3


def test_backward_workspace_is_the_documented_size():
    assert G.gemm_rmsnorm_backward_workspace(1, 10) == 40
    assert G.gemm_rmsnorm_backward_workspace(296, 8192) == 296 * 8192 * 4
    assert G.gemm_rmsnorm_backward_workspace(100000, 8192) == 296 * 8192 * 4
    assert G.gemm_rmsnorm_backward_workspace(0, 5) == 0 and G.gemm_rmsnorm_backward_workspace(5, -1) == 0


def quant(X=X, Q=Q, SF=SF, M=64, K=128, ldx=None, ldq=None, xt=BF16, layout=G.KMAJOR):
    ldx = (M if layout == G.MNMAJOR else K) if ldx is None else ldx
    return G.lib.gemm_mxfp8_quantize(X, Q, SF, M, K, ldx, K if ldq is None else ldq, xt, layout, 0)


def test_quantize_refuses_bad_arguments():
    assert quant(M=-1) == 1 and quant(K=-32) == 1 and quant(K=48, ldx=48, ldq=48) == 1
    assert quant(xt=2) == 1 and quant(layout=2) == 1
    assert quant(X=0) == 1 and quant(Q=0) == 1 and quant(SF=0) == 1
    assert quant(ldx=64) == 1 and quant(ldq=64) == 1
    assert quant(layout=G.MNMAJOR, M=200, ldx=128) == 1    # the pitch covers M
    assert quant(X=X + 2) == 2 and quant(Q=Q + 8) == 2 and quant(ldx=130) == 2 and quant(ldq=136) == 2
    assert quant(Q=X + 1024) == 3 and quant(SF=X + 1) == 3 and quant(SF=Q + 1) == 3
    assert quant(M=1 << 31) == 7
    assert quant(SF=SF + 1, M=0) == 0


def w4(A=X, B=H, S=W, Z=R, C=Y, M=4, N=256, K=512, lda=None, ldb=None, lds=16, ldc=None, group=64, ct=F32):
    return G.lib.gemm_bf16_w4(A, B, S, Z, C, M, N, K, K if lda is None else lda, K // 2 if ldb is None else ldb, lds,
                              N if ldc is None else ldc, group, ct, 0)


def test_w4_refuses_bad_arguments():
    assert w4(M=-1) == 1 and w4(N=-1) == 1 and w4(K=-32) == 1 and w4(K=520) == 1
    assert w4(group=16) == 1 and w4(group=96) == 1 and w4(group=0) == 1 and w4(group=-64) == 1
    assert w4(ct=2) == 1
    assert w4(A=0) == 1 and w4(B=0) == 1 and w4(S=0) == 1 and w4(C=0) == 1
    assert w4(lda=256) == 1 and w4(ldb=128) == 1 and w4(ldc=128) == 1
    assert w4(K=2048, lds=16) == 1                         # 32 groups
    assert w4(A=X + 2) == 2 and w4(B=H + 4) == 2 and w4(S=W + 2) == 2 and w4(Z=R + 1) == 2 and w4(C=Y + 4) == 2
    assert w4(lds=24) == 2 and w4(Z=0, lds=24) == 2 and w4(ldb=264) == 2 and w4(ldc=258) == 2
    assert w4(C=X) == 3 and w4(C=H + 64) == 3 and w4(C=W) == 3 and w4(C=R) == 3
    assert w4(M=1 << 31) == 7 and w4(N=1 << 31, ldc=1 << 31) == 7


def test_empty_problems_succeed():
    assert norm(M=0, X=0, W=0) == 0 and norm(K=0) == 0
    assert back(K=0) == 0 and back(M=0, dW=0) == 0
    assert quant(M=0, X=0) == 0 and quant(K=0) == 0
    assert w4(M=0, C=0) == 0 and w4(N=0, C=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device_report_it():
    assert norm() == 4 and norm(H=R) == 4 and norm(H=0) == 4 and norm(Q=0, SF=0, K=100, ldx=104, ldr=104, ldh=104,
                                                                      ldy=104) == 4
    assert back() == 4 and back(dH=X) == 4 and back(dH=R) == 4 and back(dW=0, ws=0) == 4 and back(M=0) == 4
    assert quant() == 4 and quant(layout=G.MNMAJOR) == 4
    assert w4() == 4 and w4(Z=0) == 4 and w4(K=0, ldb=0) == 4 and w4(group=1 << 40, lds=16) == 4


def test_package_exports_the_operators():
    import dense_gemm_engineering_bf16_b200 as pkg
    for name in ("gemm_rmsnorm", "gemm_rmsnorm_backward", "gemm_rmsnorm_backward_workspace", "gemm_mxfp8_quantize",
                 "gemm_bf16_w4"):
        assert getattr(pkg, name) is getattr(G, name)
    with pytest.raises(G.GemmError):
        G.gemm_mxfp8_quantize(X, Q, SF, 8, 33, 40, 48, stream=0)
