"""The products grouped by expert and the 4-bit operators as a program uses
them: in streams and graphs, with experts' sizes that change between replays, and
in runs: a mixture-of-experts step with its gradients, a decoding step."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from test_fp4_gpu import BLOCK, VALUES, scale_values, untile
from test_grouped_gpu import check, ends_of, ints, normal

pytestmark = pytest.mark.gpu
F32, BF16, MX, NV = G.OUT_F32, G.OUT_BF16, G.FP4_MX, G.FP4_NV


def test_first_use_inside_a_capture_is_refused():
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "projections_capture_child.py")
    r = subprocess.run([sys.executable, child], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def quantised(x, form, g=None, layout=G.KMAJOR):
    M, K = x.shape if layout == G.KMAJOR else x.shape[::-1]
    q = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(G.gemm_fp4_scale_bytes(M, K, form), dtype=torch.uint8, device="cuda")
    G.gemm_fp4_quantize(x, g, q, sf, M, K, x.stride(0), K // 2, form, F32 if x.dtype == torch.float32 else BF16, layout)
    return q, sf


def values_of(q, sf, form, g=None):
    """fp64 values of codes and scales, on the GPU."""
    M, K = q.shape[0], 2 * q.shape[1]
    b = q.cpu().numpy()
    codes = np.stack((b & 15, b >> 4), 2).reshape(M, K)
    scales = scale_values(untile(sf.cpu().numpy(), M, K, form)[0], form)
    v = torch.from_numpy(VALUES[codes] * np.repeat(scales, BLOCK[form], 1)).cuda()
    return v * g.double() if g is not None else v


class Case:
    """One call, its inputs that are written late, and its outputs."""

    def __init__(self, name):
        M, N, K, E = (64, 512, 2048, 4) if name != "grad" else (600, 512, 512, 4)
        gen = torch.Generator(device="cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
        self.x, self.new = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), rnd(M, K)
        self.ends = torch.zeros(E, dtype=torch.int32, device="cuda")
        self.new_ends = ends_of([M // 4, 0, M // 2 - 5, 3])
        w, d = rnd(E, N, K), rnd(M, N)
        c, dw = torch.zeros(M, N, device="cuda"), torch.zeros(E, N, K, device="cuda")
        q, sf = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda"), \
            torch.zeros(G.gemm_fp4_scale_bytes(M, K, NV), dtype=torch.uint8, device="cuda")
        g = torch.full((1,), 0.01, device="cuda")
        wq = quantised(w[0], NV, g)
        x, ends = self.x, self.ends

        def linear():
            G.gemm_fp4_quantize(x, g, q, sf, M, K, K, K // 2)
            G.gemm_fp4(q, sf, g, wq[0], wq[1], g, c, M, N, K, K // 2, K // 2, N)

        self.call, self.out = {
            "rows": (lambda: G.gemm_bf16_grouped(x, w, ends, c, E, M, N, K, K, K, N * K, N), (c,)),
            "grad": (lambda: G.gemm_bf16_grouped_wgrad(d, x, ends, dw, E, M, N, K, N, K, K, N * K), (dw,)),
            "linear": (linear, (c, q, sf)),
        }[name]

    def write(self):
        self.x.copy_(self.new)
        self.ends.copy_(self.new_ends)

    def clear(self):
        self.x.zero_()
        self.ends.zero_()

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.out]


def busy(a):
    for _ in range(4):                     # some hundred microseconds before the inputs are written
        torch.mm(a, a, out=a.new_empty(a.shape))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", ["rows", "grad", "linear"])
def test_inputs_written_on_another_stream(name, captured):
    case = Case(name)
    case.write()
    case.call()
    want = case.results()
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    other = torch.randn(1024, device="cuda")
    busy(a)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        """main: a short kernel, then (after side's long work and its writes) the call."""
        start = torch.cuda.Event()
        start.record(main)
        with torch.cuda.stream(side):
            side.wait_event(start)
            busy(a)
            case.write()
            written = torch.cuda.Event()
            written.record(side)
        other.add_(1)
        main.wait_event(written)
        case.call()
        case.clear()                       # and what follows waits for the call

    graph = torch.cuda.CUDAGraph() if captured else None
    if captured:
        with torch.cuda.graph(graph, stream=main):
            step()
    for _ in range(3):
        case.clear()
        for t in case.out:
            t.zero_()
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            with torch.cuda.stream(main):
                step()
        assert all(torch.equal(g, w) for g, w in zip(case.results(), want))
    G.gemm_check_device_status()


def test_two_streams_at_once():
    """Nothing is shared between calls but the status block."""
    cases, want = [], []
    for name in ("rows", "grad", "linear", "rows"):
        case = Case(name)
        case.write()
        case.call()
        want.append(case.results())
        cases.append(case)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for case, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                case.call()
    for case, w in zip(cases, want):
        assert all(torch.equal(g, x) for g, x in zip(case.results(), w))
    G.gemm_check_device_status()


@pytest.mark.parametrize("M,N,K", [(24, 256, 4096), (500, 640, 1024), (4000, 4096, 1024)])
def test_a_graph_whose_experts_change_between_replays(M, N, K):
    """The host never learns the sizes: one captured call serves all of them."""
    E = 6
    a, w = ints(1, M, K, 2).bfloat16().cuda(), ints(2, E * N, K, 2).bfloat16().cuda()
    c, ends = torch.zeros(M, N, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    dw = torch.zeros(E, N, K, device="cuda")
    d = ints(3, M, N, 2).bfloat16().cuda()

    def step():
        G.gemm_bf16_grouped(a, w, ends, c, E, M, N, K, K, K, N * K, N)
        G.gemm_bf16_grouped_wgrad(d, a, ends, dw, E, M, N, K, N, K, K, N * K)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r = np.random.RandomState(M)
    for sizes in ([M, 0, 0, 0, 0, 0], [0] * 6, [0, 0, 0, 0, 0, M - 1], list(r.multinomial(M - 3, [1 / 6] * 6)),
                  [1, 1, 1, M // 2, 0, 1]):
        ends.copy_(ends_of(sizes))
        c.fill_(-1)
        graph.replay()
        G.gemm_check_device_status()
        lo = 0
        for e, n in enumerate(sizes):
            assert torch.equal(c[lo:lo + n].double(), a[lo:lo + n].double() @ w.view(E, N, K)[e].double().t())
            assert torch.equal(dw[e].double(), d[lo:lo + n].double().t() @ a[lo:lo + n].double())
            lo += n
        assert bool((c[lo:] == -1).all())


@pytest.mark.parametrize("T,D,F,E", [(64, 256, 384, 8), (700, 512, 1056, 5)])
def test_mixture_of_experts_step_with_its_gradients(T, D, F, E):
    """Norm, two grouped products with a ReLU between, and back: the inputs'
    gradients through the weights stored the same way, the weights' gradients
    accumulated over two passes.  Each step against the formula on what went in."""
    top = 2
    M = T * top
    x, gain = normal(1, T, D).bfloat16().cuda(), torch.ones(D, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    G.gemm_rmsnorm(x, None, None, gain, y, None, None, rstd, T, D, D, 0, 0, D, 0)
    choice = torch.randint(0, E - 1, (T, top), generator=torch.Generator().manual_seed(2)).cuda()    # the last one never
    order = torch.argsort(choice.view(-1), stable=True)
    counts = torch.bincount(choice.view(-1), minlength=E)
    ends, sizes = counts.cumsum(0).to(torch.int32), counts.tolist()
    a = y[order // top].contiguous()
    up, down = (normal(3, E * F, D) / 16).bfloat16().cuda(), (normal(4, E * D, F) / 16).bfloat16().cuda()
    h, out = torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), torch.empty(M, D, device="cuda")
    G.gemm_bf16_grouped(a, up, ends, h, E, M, F, D, D, D, F * D, F, BF16)
    z = torch.relu(h)
    G.gemm_bf16_grouped(z, down, ends, out, E, M, D, F, F, F, D * F, D, F32)

    def by_group(p, w, q):
        """Rows of p times each expert's w, and sum |p w|."""
        lo, ref, mag = 0, [], []
        for e, n in enumerate(sizes):
            ref.append(p[lo:lo + n].double() @ w[e].double())
            mag.append(p[lo:lo + n].double().abs() @ w[e].double().abs())
            lo += n
        return torch.cat(ref), torch.cat(mag)

    U, W = up.view(E, F, D), down.view(E, D, F)
    check(h.double(), *by_group(a, U.transpose(1, 2), F), D, BF16)
    check(out.double(), *by_group(z, W.transpose(1, 2), D), F, F32)

    dout = normal(5, M, D).bfloat16().cuda()
    dz, da = torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), torch.empty(M, D, device="cuda")
    dU, dW = torch.full((E, F, D), float("nan"), device="cuda"), torch.full((E, D, F), float("nan"), device="cuda")
    G.gemm_bf16_grouped(dout, down, ends, dz, E, M, F, D, D, F, D * F, F, BF16, G.MNMAJOR)
    dh = dz * (h > 0)
    G.gemm_bf16_grouped(dh, up, ends, da, E, M, D, F, F, D, F * D, D, F32, G.MNMAJOR)
    for beta in (0.0, 1.0):
        G.gemm_bf16_grouped_wgrad(dout, z, ends, dW, E, M, D, F, D, F, F, D * F, F32, G.KMAJOR, beta)
        G.gemm_bf16_grouped_wgrad(dh, a, ends, dU, E, M, F, D, F, D, D, F * D, F32, G.KMAJOR, beta)
    G.gemm_check_device_status()
    check(dz.double(), *by_group(dout, W, F), D, BF16)
    check(da.double(), *by_group(dh, U, D), F, F32)
    lo = 0
    for e, n in enumerate(sizes):
        for got, p, q in ((dW[e], dout, z), (dU[e], dh, a)):
            p, q = p[lo:lo + n].double(), q[lo:lo + n].double()
            check(got.double(), 2 * p.t() @ q, 2 * p.abs().t() @ q.abs(), n + 1, F32)
        lo += n


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
def test_gradients_against_differences(layout):
    """sum(C dC) is linear in the weights and in the inputs, so that a step of any
    size changes it by the gradient's product with the step: whole numbers, exact."""
    sizes, N, K = [9, 0, 70, 33], 40, 56
    E, M = len(sizes), sum(sizes)
    ends = ends_of(sizes)
    a, w, d = ints(1, M, K), ints(2, E * N, K).view(E, N, K), ints(3, M, N)
    va, vw = ints(4, M, K), ints(5, E * N, K).view(E, N, K)
    stored = (lambda t: t) if layout == G.KMAJOR else (lambda t: t.transpose(1, 2).contiguous())
    ld, stride, back = (K, N * K, G.MNMAJOR) if layout == G.KMAJOR else (N, N * K, G.KMAJOR)

    def f(a, w):
        c = torch.zeros(M, N, device="cuda")
        G.gemm_bf16_grouped(a.bfloat16().cuda(), stored(w).bfloat16().cuda(), ends, c, E, M, N, K, K, ld, stride, N, F32, layout)
        return float((c.double().cpu() * d.double()).sum())

    da, dw = torch.zeros(M, K, device="cuda"), torch.zeros(E, *stored(w).shape[1:], device="cuda")
    G.gemm_bf16_grouped(d.bfloat16().cuda(), stored(w).bfloat16().cuda(), ends, da, E, M, K, N, N, ld, stride, K, F32, back)
    G.gemm_bf16_grouped_wgrad(d.bfloat16().cuda(), a.bfloat16().cuda(), ends, dw, E, M, N, K, N, K, ld, stride, F32, layout)
    base = f(a, w)
    assert f(a + va, w) - base == float((da.double().cpu() * va.double()).sum())
    assert f(a, w + vw) - base == float((dw.double().cpu() * stored(vw).double()).sum())


@pytest.mark.parametrize("form", [MX, NV])
@pytest.mark.parametrize("M", [1, 48, 200, 3000])
def test_norm_then_4_bit_linear_layer(M, form):
    """A norm's bf16 output into 4 bits, times 4-bit weights: the product against
    what its operands stand for, those against what they were made of (half a step
    of the largest codes is one unit of the scale; quotients up to 6.375 saturate)."""
    K, N = 1056, 640
    x, gain = normal(1, M, K).bfloat16().cuda(), torch.ones(K, device="cuda")
    y = torch.empty_like(x)
    G.gemm_rmsnorm(x, None, None, gain, y, None, None, None, M, K, K, 0, 0, K, 0)
    w = (normal(2, N, K) / 32).cuda()
    gy, gw = ((t.abs().max().reshape(1) / 2688).float() if form == NV else None for t in (y.float(), w))
    yq, wq = quantised(y, form, gy), quantised(w, form, gw)
    for t, (q, sf), g in ((y, yq, gy), (w, wq, gw)):
        unit = scale_values(untile(sf.cpu().numpy(), q.shape[0], K, form)[0], form)
        unit = torch.from_numpy(np.repeat(unit, BLOCK[form], 1)).cuda() * (g.double() if g is not None else 1.0)
        assert bool(((values_of(q, sf, form, g) - t.double()).abs() <= unit * (1 + 2.0 ** -20)).all())
    c = torch.empty(M, N, device="cuda")
    G.gemm_fp4(yq[0], yq[1], gy, wq[0], wq[1], gw, c, M, N, K, K // 2, K // 2, N, form)
    G.gemm_check_device_status()
    a, b = values_of(*yq, form, gy), values_of(*wq, form, gw)
    check(c.double(), a @ b.t(), a.abs() @ b.abs().t(), K + 4, F32)


@pytest.mark.parametrize("form", [MX, NV])
def test_backward_products_from_transposed_codes(form):
    """dX = dY W and dW = dY^T X of a linear layer in 4 bits: the operands that lie
    the other way round are quantised from where they are."""
    M, N, K = 320, 416, 288
    x, w, dy = normal(1, M, K).bfloat16().cuda(), normal(2, N, K).bfloat16().cuda(), normal(3, M, N).bfloat16().cuda()
    dx, dw = torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda")
    dyq, wt = quantised(dy, form), quantised(w, form, layout=G.MNMAJOR)
    G.gemm_fp4(*dyq, None, *wt, None, dx, M, K, N, N // 2, N // 2, K, form)
    dyt, xt = quantised(dy, form, layout=G.MNMAJOR), quantised(x, form, layout=G.MNMAJOR)
    G.gemm_fp4(*dyt, None, *xt, None, dw, N, K, M, M // 2, M // 2, K, form)
    G.gemm_check_device_status()
    for t, p, q, length in ((dx, dyq, wt, N), (dw, dyt, xt, M)):
        a, b = values_of(*p, form), values_of(*q, form)
        check(t.double(), a @ b.t(), a.abs() @ b.abs().t(), length + 1, F32)
    same = quantised(w.t().contiguous(), form)
    assert torch.equal(wt[0], same[0])
    got, want = (untile(t.cpu().numpy(), K, N, form)[0] for t in (wt[1], same[1]))
    assert np.array_equal(got, want)


@pytest.mark.parametrize("T", [1, 5])
def test_decoding_step_captured_into_a_graph(T):
    """Norm, a 4-bit projection, the chosen experts' product; replayed with other tokens."""
    D, E, F = 512, 8, 640
    M = 2 * T
    gain = torch.ones(D, device="cuda")
    x, y = (torch.zeros(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w4 = quantised((normal(1, D, D) / 16).cuda(), MX)
    q = torch.empty(T, D // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(G.gemm_fp4_scale_bytes(T, D, MX), dtype=torch.uint8, device="cuda")
    proj = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    up = (normal(2, E * F, D) / 16).bfloat16().cuda()
    rows, ends = torch.zeros(M, dtype=torch.int64, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    out = torch.empty(M, F, device="cuda")

    def step():
        G.gemm_rmsnorm(x, None, None, gain, y, None, None, None, T, D, D, 0, 0, D, 0)
        G.gemm_fp4_quantize(y, None, q, sf, T, D, D, D // 2, MX)
        G.gemm_fp4(q, sf, None, w4[0], w4[1], None, proj, T, D, D, D // 2, D // 2, D, MX, BF16)
        a = proj[rows]
        G.gemm_bf16_grouped(a, up, ends, out, E, M, F, D, D, D, F * D, F)
        return a

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = step()
    for seed in range(3):
        x.copy_(normal(10 + seed, T, D).bfloat16())
        choice = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(seed + t))[:2] for t in range(T)])
        order = torch.argsort(choice.view(-1), stable=True)
        rows.copy_(order // 2)
        ends.copy_(torch.bincount(choice.view(-1), minlength=E).cumsum(0).to(torch.int32))
        graph.replay()
        G.gemm_check_device_status()
        p, w = values_of(q, sf, MX), values_of(*w4, MX)
        check(proj.double(), p @ w.t(), p.abs() @ w.abs().t(), D + 1, BF16)
        u = up.view(E, F, D).double()[choice.view(-1)[order].cuda()]
        check(out.double(), torch.einsum("md,mfd->mf", a.double(), u), torch.einsum("md,mfd->mf", a.double().abs(), u.abs()),
              D, F32)


MOST = (1 << 31) - 1


def test_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of one column: tiles, rows and offsets at the ends of their types."""
    a = torch.ones(MOST, 8, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(MOST, 8, dtype=torch.bfloat16, device="cuda")
    at = [0, 255, 256, 1 << 24, (1 << 30) + 5, MOST - 257, MOST - 1]
    a[at, 0] = torch.arange(2.0, 2.0 + len(at), device="cuda").bfloat16()
    w = torch.tensor([[3.0] + [float("nan")] * 7, [5.0] + [float("nan")] * 7], device="cuda").bfloat16()
    ends = torch.tensor([MOST - 3, MOST], dtype=torch.int32, device="cuda")
    G.gemm_bf16_grouped(a, w, ends, c, 2, MOST, 1, 1, 8, 8, 8, 8, BF16)
    G.gemm_check_device_status()
    want = [3.0 * (2 + i) for i in range(len(at) - 1)] + [5.0 * (1 + len(at))]
    assert c[at, 0].tolist() == want
    assert float(c[MOST - 4, 0]) == 3.0 and float(c[MOST - 3, 0]) == 5.0 and float(c[MOST - 2, 0]) == 5.0
    c[at, 0] = 3.0
    c[MOST - 3:, 0] = 3.0
    assert bool((c[:, 0] == 3.0).all()) and not bool(c[:, 1:].any())


def test_as_many_columns_as_an_int_counts():
    w = torch.ones(MOST, 8, dtype=torch.bfloat16, device="cuda")
    at = [0, 127, 128, 1 << 24, MOST - 129, MOST - 1]
    w[at, 0] = torch.arange(2.0, 2.0 + len(at), device="cuda").bfloat16()
    a = torch.full((1, 8), 3.0, device="cuda").bfloat16()
    c = torch.zeros(1, MOST + 1, device="cuda")
    ends = ends_of([1])
    for layout, ldb in ((G.KMAJOR, 8), (G.MNMAJOR, MOST + 1)):
        c.zero_()
        b = w if layout == G.KMAJOR else torch.nn.functional.pad(w[:, 0], (0, 1))
        G.gemm_bf16_grouped(a, b, ends, c, 1, 1, MOST, 1, 8, ldb, 0, MOST + 1, F32, layout)
        G.gemm_check_device_status()
        assert c[0, at].tolist() == [3.0 * (2 + i) for i in range(len(at))]
        c[0, at] = 3.0
        assert bool((c[0, :MOST] == 3.0).all()) and float(c[0, MOST]) == 0.0


def test_as_long_a_4_bit_reduction_as_an_int_counts():
    K, N = MOST - 31, 3
    q, w = (torch.zeros(n, K // 2, dtype=torch.uint8, device="cuda") for n in (1, N))
    sq, sw = (torch.full((G.gemm_fp4_scale_bytes(n, K, MX),), 127, dtype=torch.uint8, device="cuda") for n in (1, N))
    for i, k in enumerate([0, 255, 256, 1 << 24, (1 << 30) + 7, K - 33, K - 1]):
        q[0, k // 2] = 2 << 4 * (k & 1)                    # 1
        w[:, k // 2] = (1 + i) % 8 << 4 * (k & 1)          # 0.5, 1, 1.5, 2, 3, 4, 6
    c = torch.empty(1, 4, device="cuda")
    G.gemm_fp4(q, sq, None, w, sw, None, c, 1, N, K, K // 2, K // 2, 4, MX)
    G.gemm_check_device_status()
    assert c[0, :N].tolist() == [18.0] * N
