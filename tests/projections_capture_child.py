"""Run by test_projections_gpu.py in a process of its own: a first use of each
operator inside a stream capture is refused and leaves the capture usable; after
one call outside it, the same capture works."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

from dense_gemm_engineering_bf16_b200 import gemm as G  # noqa: E402

E, M, N, K = 3, 300, 640, 512
a = torch.ones(M, K, device="cuda").bfloat16()
b = torch.ones(E, N, K, device="cuda").bfloat16()
c, db = torch.zeros(M, N, device="cuda"), torch.zeros(E, N, K, device="cuda")
dc = torch.ones(M, N, device="cuda").bfloat16()
ends = torch.tensor([100, 100, 290], dtype=torch.int32, device="cuda")
q, w = (torch.empty(n, K // 2, dtype=torch.uint8, device="cuda") for n in (M, N))
sf, sfw = (torch.empty(G.gemm_fp4_scale_bytes(n, K, G.FP4_NV), dtype=torch.uint8, device="cuda") for n in (M, N))
ct, c4 = torch.empty(K, M + 4, device="cuda").bfloat16(), torch.zeros(M, N, device="cuda")
calls = {
    "grouped": lambda: G.gemm_bf16_grouped(a, b, ends, c, E, M, N, K, K, K, N * K, N, check=False),
    "columns": lambda: G.gemm_bf16_grouped(dc, b, ends, c4, E, M, K, N, N, K, N * K, N, b_layout=G.MNMAJOR, check=False),
    "wgrad": lambda: G.gemm_bf16_grouped_wgrad(dc, a, ends, db, E, M, N, K, N, K, K, N * K, check=False),
    "rows": lambda: G.gemm_fp4_quantize(a, None, q, sf, M, K, K, K // 2, check=False),
    "transposed": lambda: G.gemm_fp4_quantize(ct, None, q, sf, M, K, M + 4, K // 2, layout=G.MNMAJOR, check=False),
    "weights": lambda: G.gemm_fp4_quantize(b, None, w, sfw, N, K, K, K // 2, check=False),
    "again": lambda: G.gemm_fp4_quantize(a, None, q, sf, M, K, K, K // 2, check=False),
    "product": lambda: G.gemm_fp4(q, sf, None, w, sfw, None, c4, M, N, K, K // 2, K // 2, N, check=False),
}
FIRST = {"grouped", "columns", "wgrad", "rows", "transposed", "product"}


def captured():
    graph, got = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        a.add_(0)                                  # the graph is not empty
        for name, call in calls.items():
            got[name] = call()
    graph.replay()
    torch.cuda.synchronize()
    return got


torch.cuda.synchronize()
got = captured()
assert all(got[name] == 8 for name in FIRST), got
for name, call in calls.items():
    assert call() == 0, name
torch.cuda.synchronize()
c.zero_()
c4.zero_()
assert set(captured().values()) == {0}, "captured after a first call"
G.gemm_check_device_status()
assert torch.all(c[:290] == K) and torch.all(c[290:] == 0)
assert torch.all(db[0] == 100) and torch.all(db[1] == 0) and torch.all(db[2] == 190)
# ones in 4 bits: the scale is E4M3(1 / 6) = 0.171875, a code 6, which stands for 1.03125
assert torch.all(c4 == K * 1.03125 ** 2)
print("ok")
