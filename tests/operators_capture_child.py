"""Run by test_operators_capture_gpu.py in a process of its own: a first use of
each operator inside a stream capture is refused and leaves the capture
usable; after one call outside it, the same capture works."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

from dense_gemm_engineering_bf16_b200 import gemm as G  # noqa: E402

M, K, N = 6, 256, 128
x = torch.randn(M, K, device="cuda").bfloat16()
y, dh, w = torch.empty_like(x), torch.empty_like(x), torch.ones(K, device="cuda")
rstd, dw = torch.ones(M, device="cuda"), torch.empty(K, device="cuda")
ws = torch.empty(G.gemm_rmsnorm_backward_workspace(M, K), dtype=torch.uint8, device="cuda")
q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
sf = torch.empty(M, K // 32, dtype=torch.uint8, device="cuda")
xt = torch.randn(K, 8, device="cuda").bfloat16()
codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
scales = torch.ones(N, 16, device="cuda").bfloat16()
c = torch.empty(M, N, device="cuda")
calls = {
    "norm": lambda: G.gemm_rmsnorm(x, None, None, w, y, None, None, rstd, M, K, K, 0, 0, K, 0, check=False),
    "back": lambda: G.gemm_rmsnorm_backward(x, x, w, rstd, None, dh, dw, ws, M, K, K, K, 0, K, check=False),
    "rows": lambda: G.gemm_mxfp8_quantize(x, q, sf, M, K, K, K, check=False),
    "columns": lambda: G.gemm_mxfp8_quantize(xt, q, sf, M, K, 8, K, layout=G.MNMAJOR, check=False),
    "w4": lambda: G.gemm_bf16_w4(x, codes, scales, None, c, M, N, K, K, K // 2, 16, N, 64, check=False),
}


def captured():
    graph, got = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        x.add_(0)                                  # the graph is not empty
        for name, call in calls.items():
            got[name] = call()
    graph.replay()
    torch.cuda.synchronize()
    return got


torch.cuda.synchronize()
assert set(captured().values()) == {8}, "first uses inside a capture"
for name, call in calls.items():
    assert call() == 0, name
torch.cuda.synchronize()
assert set(captured().values()) == {0}, "captured after a first call"
assert torch.all(c == -8 * x.float().sum(1, keepdim=True)) or torch.allclose(c, -8 * x.float().sum(1, keepdim=True),
                                                                             rtol=1e-4, atol=1e-3)
print("ok")
