"""The operators take their place in a stream like any other work: what they
read may have been written on another stream that theirs waited for, eagerly or
in a captured graph.  (Their launches carry programmatic dependence, which
relaxes the order between neighbouring kernels; the wait at each kernel's
start has to restore all of it.)"""
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

pytestmark = pytest.mark.gpu
M, K, N = 64, 2048, 512


class Case:
    """One call, its input `x` (bf16, written late) and its outputs."""

    def __init__(self, name):
        gen = torch.Generator(device="cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
        self.x, self.new = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), rnd(M, K)
        h, w, y = rnd(M, K), torch.ones(K, device="cuda"), torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        q, sf = (torch.zeros(M, n, dtype=torch.uint8, device="cuda") for n in (K, K // 32))
        rstd, dw = torch.ones(M, device="cuda"), torch.zeros(K, device="cuda")
        ws = torch.empty(G.gemm_rmsnorm_backward_workspace(M, K), dtype=torch.uint8, device="cuda")
        codes = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
        scales, c = torch.ones(N, 32, device="cuda").bfloat16(), torch.zeros(M, N, device="cuda")
        x = self.x
        self.call, self.out = {
            "norm": (lambda: G.gemm_rmsnorm(x, None, None, w, y, None, None, rstd, M, K, K, 0, 0, K, 0), (y, rstd)),
            "back": (lambda: G.gemm_rmsnorm_backward(x, h, w, rstd, None, y, dw, ws, M, K, K, K, 0, K), (y, dw)),
            "rows": (lambda: G.gemm_mxfp8_quantize(x, q, sf, M, K, K, K), (q, sf)),
            "columns": (lambda: G.gemm_mxfp8_quantize(x, q.view(K, M), sf, K, M, K, M, layout=G.MNMAJOR), (q, sf)),
            "w4": (lambda: G.gemm_bf16_w4(x, codes, scales, None, c, M, N, K, K, K // 2, 32, N, 64), (c,)),
        }[name]

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.out]


def busy(a):
    for _ in range(4):                     # some hundred microseconds before the input is written
        torch.mm(a, a, out=a.new_empty(a.shape))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", ["norm", "back", "rows", "columns", "w4"])
def test_input_written_on_another_stream(name, captured):
    case = Case(name)
    case.x.copy_(case.new)
    case.call()
    want = case.results()
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    other = torch.randn(1024, device="cuda")
    busy(a)                                # the product's own set-up
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        """main: a short kernel, then (after side's long work and its write of x) the call."""
        start = torch.cuda.Event()
        start.record(main)
        with torch.cuda.stream(side):
            side.wait_event(start)
            busy(a)
            case.x.copy_(case.new)
            written = torch.cuda.Event()
            written.record(side)
        other.add_(1)
        main.wait_event(written)
        case.call()
        case.x.zero_()                     # and what follows waits for the call

    graph = torch.cuda.CUDAGraph() if captured else None
    if captured:
        with torch.cuda.graph(graph, stream=main):
            step()
    for _ in range(3):
        case.x.zero_()
        for t in case.out:
            t.zero_()
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            with torch.cuda.stream(main):
                step()
        got = case.results()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("name", ["norm", "back", "rows", "columns", "w4"])
def test_input_written_by_a_copy_or_a_memset_in_a_graph(name):
    """The node before the call is no kernel."""
    case = Case(name)
    host = case.new.cpu().pin_memory()
    case.x.copy_(case.new)
    case.call()
    want = case.results()
    case.x.zero_()
    case.call()
    zero = case.results()
    graph, after_zero = torch.cuda.CUDAGraph(), [torch.empty_like(t) for t in case.out]
    with torch.cuda.graph(graph):
        case.x.zero_()
        case.call()
        for t, o in zip(after_zero, case.out):
            t.copy_(o)
        case.x.copy_(host, non_blocking=True)
        case.call()
    for _ in range(3):
        graph.replay()
        got = case.results()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        assert all(torch.equal(g, w) for g, w in zip(after_zero, zero))
