"""The operators in a run, as a linear layer uses them: a norm whose codes go
into the block-scaled product, the backward products from transposed codes,
the norm's gradients; and a decoding step on 4-bit weights."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from operator_refs import mx_reference, mx_values, normal, pad, rmsnorm_reference, w4_reference

pytestmark = pytest.mark.gpu
EPS = 1e-5


def quantize(x, M, K, layout=G.KMAJOR):
    q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    sf = torch.empty(M, K // 32, dtype=torch.float8_e8m0fnu, device="cuda")
    kind = G.OUT_F32 if x.dtype == torch.float32 else G.OUT_BF16
    G.gemm_mxfp8_quantize(x, q, sf, M, K, x.stride(0), K, kind, layout)
    return q, sf


def values(q, sf):
    return mx_values(q.view(torch.uint8).cpu().numpy(), sf.view(torch.uint8).cpu().numpy())


def product(a, b, M, N, K):
    c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    G.gemm_mxfp8(a[0], a[1], b[0], b[1], c, M, N, K, K, K, N)
    return c


def close(c, a, b):
    """C of gemm_mxfp8 against the values its operands stand for."""
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    assert np.all(np.abs(c.double().cpu().numpy() - want) <= 1e-3 * mag + 1e-6 + 2.0 ** -8 * np.abs(want))


def test_training_step_of_a_norm_and_a_block_scaled_linear_layer():
    M, K, N = 160, 256, 320                        # tokens, inputs, outputs
    x, r = (normal(i, M, K, 0.4).bfloat16().cuda() for i in (1, 2))
    w = (1 + 0.2 * normal(3, 1, K))[0].cuda()
    W = (normal(4, N, K) / 16).bfloat16().cuda()
    h, y = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    sf = torch.empty(M, K // 32, dtype=torch.float8_e8m0fnu, device="cuda")
    rstd = torch.empty(M, device="cuda")
    G.gemm_rmsnorm(x, r, h, w, y, q, sf, rstd, M, K, K, K, K, K, K, eps=EPS)
    out = product((q, sf), quantize(W, N, K), M, N, K)
    close(out, values(q, sf), values(*quantize(W, N, K)))
    ref, _ = rmsnorm_reference(h.double().cpu().numpy(), w.double().cpu().numpy(), EPS)
    assert np.linalg.norm(values(q, sf) - ref) <= 0.04 * np.linalg.norm(ref)       # E4M3: at most 2^-4 each

    # backward: dY = dOut . W needs W with its codes along N, dW_lin = dOut^T . y both along M
    dout = normal(5, M, N).bfloat16().cuda()
    wt = quantize(W, K, N, G.MNMAJOR)
    assert np.array_equal(wt[0].view(torch.uint8).cpu().numpy(), mx_reference(W.double().cpu().numpy().T.copy())[0])
    dy = product(quantize(dout, M, N), wt, M, K, N)
    close(dy, values(*quantize(dout, M, N)), values(*wt))
    dt, yt = quantize(dout, N, M, G.MNMAJOR), quantize(y, K, M, G.MNMAJOR)
    dlin = product(dt, yt, N, K, M)
    close(dlin, values(*dt), values(*yt))

    dh, dw = torch.empty_like(h), torch.empty(K, device="cuda")
    ws = torch.empty(G.gemm_rmsnorm_backward_workspace(M, K), dtype=torch.uint8, device="cuda")
    G.gemm_rmsnorm_backward(dy, h, w, rstd, x, dh, dw, ws, M, K, K, K, K, K)
    G.gemm_check_device_status()
    hh = h.double().cpu().requires_grad_(True)
    wd = w.double().cpu().requires_grad_(True)
    n = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + EPS) * wd
    n.backward(dy.double().cpu())
    want = hh.grad + x.double().cpu()
    # bf16 output: half a step; the fp32 part is far below
    assert torch.all((dh.double().cpu() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -16) + hh.grad.abs().max() * 2.0 ** -16)
    assert torch.all((dw.double().cpu() - wd.grad).abs() <= wd.grad.abs().max() * 2.0 ** -16)


@pytest.mark.parametrize("M", [1, 6])
def test_decoding_step_on_4_bit_weights_captured_into_a_graph(M):
    K, N, group = 512, 640, 64
    x = normal(1, M, K).bfloat16().cuda()
    stream_h = normal(2, M, K).bfloat16().cuda()
    w = torch.ones(K, device="cuda")
    rng = np.random.default_rng(3)
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).cuda()
    scales = (0.05 * torch.rand(N, pad(K // group, 16), generator=torch.Generator().manual_seed(4))).bfloat16().cuda()
    y, c = torch.empty_like(x), torch.empty(M, N, device="cuda")

    def step():
        G.gemm_rmsnorm(x, stream_h, stream_h, w, y, None, None, None, M, K, K, K, K, K, 0)
        G.gemm_bf16_w4(y, codes, scales, None, c, M, N, K, K, K // 2, scales.shape[1], N, group)

    keep = stream_h.clone()
    step()
    torch.cuda.synchronize()
    stream_h.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    graph.replay()                                 # the stream moves on in place: h = r + 2 x
    torch.cuda.synchronize()
    h = (keep.float() + x.float()).bfloat16()
    h = (h.float() + x.float()).bfloat16()
    assert torch.equal(stream_h, h)
    ref, _ = rmsnorm_reference(h.double().cpu().numpy(), 1.0, EPS)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -16))
    want, mag = w4_reference(y.double().cpu().numpy(), codes.cpu().numpy(), scales.double().cpu().numpy(),
                             np.full((N, K // group), 8.0), group, K)
    assert np.all(np.abs(c.double().cpu().numpy() - want) <= mag * (16 * 2.0 ** -22 + 24 * 2.0 ** -24))
