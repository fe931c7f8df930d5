"""gemm_mxfp8_quantize, bit for bit against the definition in 64 bits (the
scaling is exact, so that there is one rounding), in both storage orders."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from operator_refs import BF16, F32, TORCH, Buffer, mx_reference, normal

pytestmark = pytest.mark.gpu


def run(x, xt, layout, sf_offset=0, stream=None):
    """x: M x K values; stored M x K or K x M."""
    M, K = x.shape
    mn = layout == G.MNMAJOR
    X = Buffer(K if mn else M, M if mn else K, TORCH[xt], fill=x.t() if mn else x)
    Q = Buffer(M, K, torch.uint8)
    SF = Buffer(1, M * (K // 32) + sf_offset, torch.uint8)
    G.gemm_mxfp8_quantize(X.ptr, Q.ptr, SF.ptr + sf_offset, M, K, X.ld, Q.ld, xt, layout, stream=stream)
    torch.cuda.synchronize()
    assert X.guards_ok() and Q.guards_ok() and SF.guards_ok()
    values = X.f64()
    codes, sf = mx_reference(values.T.copy() if mn else values)
    got = Q.get().numpy()
    got_sf = SF.get().numpy()[0, sf_offset:].reshape(M, K // 32)
    assert np.array_equal(got_sf, sf)
    nan = (codes == 0x7F)
    assert np.array_equal(got[nan] & 0x7F, codes[nan]) and np.array_equal(got[~nan], codes[~nan])
    return got, got_sf


SIZES = [(1, 32), (2, 64), (3, 96), (63, 128), (64, 160), (65, 256), (129, 1024), (130, 1056), (7, 8192), (40, 8224),
         (1000, 992), (2, 40000)]


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("M,K", SIZES)
def test_sizes(M, K, xt, layout):
    run(normal(M + K, M, K, 1.0), xt, layout)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
def test_every_exponent_and_border(layout):
    """Blocks whose largest value is at, just below and just above 448 times
    each power of two, down to fp32's subnormals and up to its largest."""
    rows = []
    for e in range(-149, 128):
        for m in (1.0, 1.5, 1.75, 1.75 * (1 - 2.0 ** -23), 1.75 * (1 + 2.0 ** -23), 2 - 2.0 ** -23):
            r = np.zeros(32)
            r[:] = np.linspace(-1, 1, 32) * 0.9
            r[5] = -m
            with np.errstate(over="ignore"):
                rows.append((r * 2.0 ** e).astype(np.float32))
    x = torch.from_numpy(np.stack(rows))
    x = x[torch.isfinite(x).all(dim=1)]
    run(x, F32, layout)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_zeros_nan_and_infinities(xt, layout):
    x = normal(3, 6, 96)
    x[0] = 0
    x[1, :32] = -0.0
    x[2, 40] = float("nan")
    x[3, 33] = float("inf")
    x[3, 34] = -float("inf")
    x[4, 64:] = float("nan")
    got, sf = run(x, xt, layout)
    assert sf[0].tolist() == [0, 0, 0] and sf[4, 2] == 0
    assert (got[3, 33:35] & 0x7F == 0x7F).all() and (got[4, 64:] & 0x7F == 0x7F).all()


def test_scales_at_an_odd_address():
    run(normal(5, 70, 320), BF16, G.KMAJOR, sf_offset=3)
    run(normal(6, 70, 320), BF16, G.MNMAJOR, sf_offset=3)


def test_every_bf16_value():
    """All finite bf16 values, 32 of one exponent to a block."""
    bits = np.arange(1 << 16, dtype=np.uint32)
    x = torch.from_numpy((bits << 16).view(np.float32).copy()).reshape(-1, 32)
    run(x[torch.isfinite(x).all(dim=1)], BF16, G.KMAJOR)


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
def test_offsets_past_32_bits(layout):
    """Source rows 2^32 bytes apart."""
    M, K = (2, 64) if layout == G.KMAJOR else (64, 32)
    ld = (1 << 31) + 8 if layout == G.KMAJOR else 1 << 27          # 31 * 2^28 bytes to the last row
    rows, cols = (M, K) if layout == G.KMAJOR else (K, M)
    x = torch.empty((rows - 1) * ld + 64, dtype=torch.bfloat16, device="cuda")
    v = normal(9, rows, cols).bfloat16()
    for i in range(rows):
        x[i * ld:i * ld + cols] = v[i].cuda()
    Q, SF = Buffer(M, K, torch.uint8), Buffer(1, M * K // 32, torch.uint8)
    G.gemm_mxfp8_quantize(x, Q.ptr, SF.ptr, M, K, ld, Q.ld, BF16, layout)
    codes, sf = mx_reference((v if layout == G.KMAJOR else v.t()).double().numpy().copy())
    assert np.array_equal(Q.get().numpy(), codes) and np.array_equal(SF.get().numpy()[0], sf.reshape(-1))


def test_graph_replay_reads_new_values():
    M, K = 50, 256
    X = Buffer(M, K, torch.bfloat16, fill=normal(1, M, K))
    Q, SF = Buffer(M, K, torch.uint8), Buffer(1, M * K // 32, torch.uint8)
    call = lambda: G.gemm_mxfp8_quantize(X.ptr, Q.ptr, SF.ptr, M, K, X.ld, Q.ld)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    X.t[:, :K] = normal(2, M, K).cuda()
    graph.replay()
    torch.cuda.synchronize()
    codes, sf = mx_reference(X.f64())
    assert np.array_equal(Q.get().numpy(), codes) and np.array_equal(SF.get().numpy()[0], sf.reshape(-1))
