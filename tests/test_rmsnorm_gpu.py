"""gemm_rmsnorm and gemm_rmsnorm_backward against their formulas in 64 bits.

Tolerances count roundings.  The sum of K squares is added in at most
D = 32 + K / 1024 + 12 steps on any path (a thread's own elements, five
shuffles twice), each square rounded once; the root takes half of that, and
mean, + eps, root and reciprocal four more: rstd is within (D / 2 + 5) u of
the exact one, u = 2^-24.  y multiplies twice more and is rounded to its type.
"""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from operator_refs import (BF16, F32, HALF_STEP, TINY, TORCH, U32, Buffer, mx_reference, mx_values, normal, pad,
                           rmsnorm_reference)

pytestmark = pytest.mark.gpu
EPS = 1e-5


def depth(K):
    return 32 + K / 1024 + 12


def run_norm(M, K, xt=BF16, ht=BF16, residual=True, store_h=True, bf16_out=True, mx=False, rstd=True, in_place=False,
             seed=0, x=None, stream=None):
    X = Buffer(M, K, TORCH[xt], fill=normal(seed, M, K, 0.5) if x is None else x)
    R = Buffer(M, K, TORCH[ht], fill=normal(seed + 1, M, K, 0.5)) if residual else None
    before = R.f64() if residual else None
    H = None
    if residual and store_h:
        H = R if in_place else Buffer(M, K, TORCH[ht])
    w = (1 + 0.3 * normal(seed + 2, 1, K))[0].cuda()
    Y = Buffer(M, K, torch.bfloat16, ld=pad(K, 8) + 16) if bf16_out else None
    Q = Buffer(M, K, torch.uint8) if mx else None
    SF = Buffer(1, M * (K // 32), torch.uint8) if mx else None
    RS = Buffer(1, M, torch.float32) if rstd else None
    ptr = lambda b: b.ptr if b is not None else None  # noqa: E731
    ld = lambda b: b.ld if b is not None else 0       # noqa: E731
    G.gemm_rmsnorm(X.ptr, ptr(R), ptr(H), w, ptr(Y), ptr(Q), ptr(SF), ptr(RS), M, K, X.ld, ld(R), ld(H), ld(Y), ld(Q),
                   xt, ht, EPS, stream=stream)
    torch.cuda.synchronize()
    for b in (X, R, H, Y, Q, SF, RS):
        assert b is None or b.guards_ok()
    # h: the fp32 sum's rounding and the type's
    xs = X.f64()
    if residual:
        want = xs + before
        if H is not None:
            h = H.f64()
            assert np.all(np.abs(h - want) <= np.abs(want) * (HALF_STEP[ht] + 2 * U32) + TINY)
        else:
            h = torch.from_numpy((X.get().float() + torch.from_numpy(before).float()).numpy()).to(TORCH[ht]).double().numpy()
    else:
        h = xs
    y, rs = rmsnorm_reference(h, w.double().cpu().numpy(), EPS)
    rel = (depth(K) / 2 + 5) * U32
    if RS is not None:
        assert np.all(np.abs(RS.f64()[0] - rs) <= rel * rs)
    if Y is not None:
        assert np.all(np.abs(Y.f64() - y) <= np.abs(y) * (HALF_STEP[BF16] + rel + 3 * U32) + TINY)
    if Q is not None:
        codes, sf = Q.get().numpy(), SF.get().numpy().reshape(M, K // 32)
        scale = 2.0 ** (sf.astype(np.float64) - 127)
        got = mx_values(codes, sf)
        slack = np.abs(y) * (rel + 3 * U32)
        step = np.abs(y) * 2.0 ** -4 + np.repeat(scale, 32, axis=1) * 2.0 ** -10      # normal, subnormal codes
        assert np.all(np.abs(got - y) <= step + 2 * slack)
        # the scale is the smallest that fits, but for a maximum within rounding of the border
        amax = np.abs(y).reshape(M, K // 32, 32).max(axis=2)
        assert np.all(amax <= 448 * scale * (1 + rel + 3 * U32))
        assert np.all((sf == 0) | (amax >= 224 * scale * (1 - rel - 3 * U32)))
    return X, R, H, w, Y, Q, SF, RS


SIZES = [(1, 1), (1, 8), (3, 7), (9, 31), (5, 64), (17, 256), (8, 257), (2, 520), (3, 1000), (7, 1024), (3, 1032),
         (300, 1100), (5, 2048), (301, 3000), (4, 8192), (299, 8200), (2, 16384), (2, 16392), (3, 20001)]


@pytest.mark.parametrize("M,K", SIZES)
def test_norm_sizes(M, K):
    run_norm(M, K, seed=M + K)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("ht", [F32, BF16, None])
@pytest.mark.parametrize("M,K", [(13, 96), (5, 800), (400, 2080), (6, 8192), (2, 16416)])
def test_norm_types_with_both_outputs(M, K, xt, ht):
    run_norm(M, K, xt, BF16 if ht is None else ht, residual=ht is not None, mx=True, seed=7)


@pytest.mark.parametrize("M,K", [(4, 64), (3, 2048), (310, 4096), (2, 20000)])
@pytest.mark.parametrize("ht", [F32, BF16])
def test_norm_in_place_and_without_storing_h(M, K, ht):
    run_norm(M, K, BF16, ht, in_place=True, seed=3)
    run_norm(M, K, BF16, ht, store_h=False, rstd=False, seed=4)
    run_norm(M, K, BF16, ht, bf16_out=False, mx=True, rstd=False, in_place=True, seed=5)


def test_norm_in_place_gives_the_same_bits():
    M, K = 300, 3000
    a = run_norm(M, K, seed=11)
    b = run_norm(M, K, seed=11, in_place=True)
    assert torch.equal(a[2].get(), b[2].get()) and torch.equal(a[4].get(), b[4].get()) and torch.equal(a[7].get(), b[7].get())


def test_norm_zero_rows_tiny_and_large_values():
    M, K = 6, 256
    x = normal(1, M, K)
    x[0] = 0                                  # y = 0, rstd = 1 / sqrt(eps)
    x[1] *= 1e-30
    x[2] *= 1e15
    run_norm(M, K, F32, residual=False, mx=True, x=x)


def test_norm_nan_and_infinity_stay_in_their_row():
    M, K = 5, 256
    x = normal(2, M, K)
    x[1, 3] = float("nan")
    x[3, 40] = float("inf")
    X, Y, Q, SF, RS = (Buffer(M, K, torch.float32, fill=x), Buffer(M, K, torch.bfloat16), Buffer(M, K, torch.uint8),
                       Buffer(1, M * K // 32, torch.uint8), Buffer(1, M, torch.float32))
    w = torch.ones(K, device="cuda")
    G.gemm_rmsnorm(X.ptr, None, None, w, Y.ptr, Q.ptr, SF.ptr, RS.ptr, M, K, X.ld, 0, 0, Y.ld, Q.ld, F32, F32, EPS)
    y, q = Y.f64(), Q.get().numpy()
    assert np.isnan(y[1]).all() and (q[1] == 0x7F).all() and np.isnan(RS.f64()[0, 1])
    # an infinite sum: rstd = 0, finite values give 0, the infinity itself 0 * inf
    assert RS.f64()[0, 3] == 0 and np.isnan(y[3, 40]) and (np.delete(y[3], 40) == 0).all() and q[3, 40] == 0x7F
    ref, _ = rmsnorm_reference(x.double().numpy(), np.ones(K), EPS)
    for i in (0, 2, 4):
        assert np.allclose(y[i], ref[i], rtol=2.0 ** -7, atol=0)


# ---------------------------------------------------------------- backward --


def back_buffers(M, K, yt, ht, dt, residual, dw, seed, in_place=None):
    dY = Buffer(M, K, TORCH[yt], fill=normal(seed, M, K))
    H = Buffer(M, K, TORCH[ht], fill=normal(seed + 1, M, K, 0.5))
    w = (1 + 0.3 * normal(seed + 2, 1, K))[0].cuda()
    RS = torch.from_numpy(rmsnorm_reference(H.f64(), 1.0, EPS)[1]).float().cuda()
    dR = Buffer(M, K, TORCH[dt], fill=normal(seed + 3, M, K)) if residual else None
    dH = dY if in_place == "dY" else dR if in_place == "dR" else Buffer(M, K, TORCH[dt])
    dW = Buffer(1, K, torch.float32, ld=pad(K, 4) + 4) if dw else None
    need = G.gemm_rmsnorm_backward_workspace(M, K)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    return dY, H, w, RS, dR, dH, dW, ws, need


def run_back(M, K, yt=BF16, ht=BF16, dt=BF16, residual=True, dw=True, seed=0, in_place=None, stream=None):
    dY, H, w, RS, dR, dH, dW, ws, need = back_buffers(M, K, yt, ht, dt, residual, dw, seed, in_place)
    dy, h, rs, ww = dY.f64(), H.f64(), RS.double().cpu().numpy()[:, None], w.double().cpu().numpy()
    dr = dR.f64() if residual else 0.0
    G.gemm_rmsnorm_backward(dY.ptr, H.ptr, w, RS, dR.ptr if residual else None, dH.ptr, dW.ptr if dw else None,
                            ws.data_ptr() if dw else None, M, K, dY.ld, H.ld, dR.ld if residual else 0, dH.ld, yt, ht, dt,
                            workspace_bytes=need, stream=stream)
    torch.cuda.synchronize()
    for b in (dY, H, dR, dH, dW):
        assert b is None or b.guards_ok()
    assert bool((ws[need:] == 0xFF).all())
    n, g = h * rs, dy * ww
    mean = (g * n).mean(axis=1, keepdims=True)
    want = rs * (g - n * mean)
    # g: one rounding; n: one; each product of the sum: two more, then its steps;
    # n * mean, the difference, * rstd, + dr: one each
    tol = rs * (np.abs(g) * 4 * U32 + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True) * (depth(K) + 10) * U32)
    tol = tol + (np.abs(want) + np.abs(want + dr)) * 2 * U32 + np.abs(want + dr) * HALF_STEP[dt] + TINY
    assert np.all(np.abs(dH.f64() - (want + dr)) <= tol)
    if dw:
        # at most M + 40 additions on a column's path, each product rounded twice
        s = np.abs(dy * n).sum(axis=0)
        assert np.all(np.abs(dW.f64()[0] - (dy * n).sum(axis=0)) <= s * (M + 42) * U32 + TINY)
    return dH, dW


@pytest.mark.parametrize("M,K", SIZES + [(2000, 40), (700, 2000), (1000, 8), (350, 16400)])
def test_back_sizes(M, K):
    run_back(M, K, seed=M + K)


@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("ht", [F32, BF16])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("M,K", [(33, 90), (310, 2056), (3, 17000)])
def test_back_types(M, K, yt, ht, dt):
    run_back(M, K, yt, ht, dt, seed=5)
    run_back(M, K, yt, ht, dt, residual=False, dw=False, seed=6)


@pytest.mark.parametrize("M,K", [(20, 100), (320, 4096), (3, 17000)])
@pytest.mark.parametrize("where", ["dY", "dR"])
def test_back_in_place(M, K, where):
    run_back(M, K, seed=8, in_place=where)


def test_back_is_deterministic():
    a, b = run_back(1000, 3000, seed=9), run_back(1000, 3000, seed=9)
    assert torch.equal(a[0].get(), b[0].get()) and torch.equal(a[1].get(), b[1].get())


def test_back_of_no_rows_zeroes_dw():
    dW = Buffer(1, 100, torch.float32)
    G.gemm_rmsnorm_backward(None, None, None, None, None, None, dW.ptr, None, 0, 100, 0, 0, 0, 0)
    assert np.all(dW.f64() == 0) and dW.guards_ok()


def test_back_against_differences():
    """A directional derivative of L = sum dy * y(h, w) by central differences
    of the forward formula in 64 bits."""
    M, K = 40, 500
    dY, H, w, RS, dR, dH, dW, ws, need = back_buffers(M, K, F32, F32, F32, False, True, 21)
    G.gemm_rmsnorm_backward(dY.ptr, H.ptr, w, RS, None, dH.ptr, dW.ptr, ws.data_ptr(), M, K, dY.ld, H.ld, 0, dH.ld, F32,
                            F32, F32, workspace_bytes=need)
    dy, h, ww = dY.f64(), H.f64(), w.double().cpu().numpy()
    vh, vw = normal(30, M, K).double().numpy(), normal(31, 1, K)[0].double().numpy()
    loss = lambda t, s: float((dy * rmsnorm_reference(h + t * vh, ww + s * vw, EPS)[0]).sum())  # noqa: E731
    # differences of step 1e-4 are within 1e-7 of the derivative's scale; the kernel's sums within 1e-5
    for got, at in ((dH.f64() * vh, (1e-4, 0)), (dW.f64()[0] * vw, (0, 1e-4))):
        diff = (loss(*at) - loss(-at[0], -at[1])) / 2e-4
        assert abs(got.sum() - diff) <= 2e-5 * np.abs(got).sum()


# -------------------------------------------------- as a user would call it --


def test_offsets_past_32_bits():
    """Rows 2^32 bytes and more apart."""
    M, K, ld = 2, 1000, (1 << 31) + 8
    x = torch.empty(ld + 1008, dtype=torch.bfloat16, device="cuda")
    rows = normal(1, M, K).bfloat16()
    for i in range(M):
        x[i * ld:i * ld + K] = rows[i].cuda()
    w, Y = torch.ones(K, device="cuda"), Buffer(M, K, torch.bfloat16)
    G.gemm_rmsnorm(x, None, None, w, Y.ptr, None, None, None, M, K, ld, 0, 0, Y.ld, 0)
    y, _ = rmsnorm_reference(rows.double().numpy(), 1.0, EPS)
    assert np.all(np.abs(Y.f64() - y) <= np.abs(y) * 2.0 ** -7) and Y.guards_ok()


def test_other_streams_and_graph_replay():
    """Two graphs captured on one stream, each with a workspace of its own, and
    eager calls between their replays."""
    M, K = 400, 2048
    side = torch.cuda.Stream()
    sets = [back_buffers(M, K, BF16, BF16, BF16, True, True, 40 + i) for i in range(2)]
    call = lambda b: G.gemm_rmsnorm_backward(b[0].ptr, b[1].ptr, b[2], b[3], b[4].ptr, b[5].ptr, b[6].ptr,  # noqa: E731
                                             b[7].data_ptr(), M, K, b[0].ld, b[1].ld, b[4].ld, b[5].ld,
                                             workspace_bytes=b[8])
    side.wait_stream(torch.cuda.current_stream())
    want = []
    with torch.cuda.stream(side):
        for b in sets:
            call(b)
        side.synchronize()
        want = [(b[5].get(), b[6].get()) for b in sets]
        graphs = []
        for b in sets:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call(b)
            graphs.append(graph)
    for b in sets:
        b[5].t.fill_(0)
        b[6].t.fill_(0)
        b[7].fill_(0xFF)
    torch.cuda.synchronize()
    for graph in graphs:
        graph.replay()
    call(sets[0])
    torch.cuda.synchronize()
    for b, (dh, dw) in zip(sets, want):
        assert torch.equal(b[5].get(), dh) and torch.equal(b[6].get(), dw)


def test_binding_refuses_other_devices_and_types():
    M, K = 4, 64
    x, w = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), torch.ones(K, device="cuda")
    y = torch.empty_like(x)
    call = lambda **k: G.gemm_rmsnorm(*[k.get(n, d) for n, d in (("x", x), ("r", None), ("h", None), ("w", w), ("y", y),  # noqa: E731,E501
                                                                 ("q", None), ("sf", None), ("rstd", None))],
                                      M, K, K, 0, 0, K, 0)
    call()
    for bad in ({"x": x.cpu()}, {"x": x.float()}, {"w": w.bfloat16()}, {"y": y.half()}, {"rstd": y}, {"q": y, "sf": y}):
        with pytest.raises(G.GemmError):
            call(**bad)
