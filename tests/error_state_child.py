"""Run by test_error_state_gpu.py in a process of its own: a CUDA call that
fails on the host inside the library is that call's status, and not the next
one's."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

from dense_gemm_engineering_bf16_b200 import gemm as G  # noqa: E402

N, LAUNCH = 64, 5
a = torch.randn(N, N, device="cuda").bfloat16()
w, y = torch.ones(N, device="cuda"), torch.empty_like(a)
c = torch.empty(N, N, device="cuda")
product = lambda **k: G.gemm_bf16(a, a, c, N, N, N, N, N, N, check=False, **k)                            # noqa: E731
norm = lambda **k: G.gemm_rmsnorm(a, None, None, w, y, None, None, None, N, N, N, 0, 0, N, 0, check=False, **k)  # noqa: E731
assert product() == 0 and norm() == 0
torch.cuda.synchronize()


def in_a_spoiled_capture(call):
    """The status of a call on a stream whose capture was spoiled before it: its
    launch is refused by the runtime.  (What spoils it is itself such a call:
    a synchronisation of the stream that is being captured.)"""
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        graph.capture_begin(capture_error_mode="relaxed")
        spoiled = G.gemm_check_device_status(stream=stream, check=False)
        got = call(stream=stream)
        try:
            graph.capture_end()
        except RuntimeError:
            pass
    return spoiled, got


for call in (product, norm):
    assert in_a_spoiled_capture(call) == (LAUNCH, LAUNCH), call
    first, second = product(), norm()
    assert (first, second) == (0, 0), (first, second)
    torch.cuda.synchronize()
want = a.double() @ a.double().t()
assert torch.allclose(c.double(), want, rtol=1e-4, atol=1e-3)
print("ok")
