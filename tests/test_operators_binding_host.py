"""What the binding of the operators refuses before it calls the library.  The
tensors here are in host memory and the binding is told that this is the
current device, so that a call that passes its checks ends at the library's own
device check (status 4): without a device only."""
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors: only where nothing can be launched")
M, K, N = 8, 64, 32


@pytest.fixture(autouse=True)
def host_is_the_device(monkeypatch):
    G._here(0)
    monkeypatch.setitem(G._DTYPES, "device", lambda: torch.empty(0).get_device())
    monkeypatch.setitem(G._DTYPES, "stream", lambda dev: 0)


def aligned(*shape, dtype):
    """A tensor at a multiple of 16 bytes (which host allocations are)."""
    t = torch.zeros(*shape, dtype=dtype)
    assert t.data_ptr() % 16 == 0
    return t


def operands():
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    return dict(x=aligned(M, K, dtype=bf), h=aligned(M, K, dtype=bf), y=aligned(M, K, dtype=bf), dh=aligned(M, K, dtype=bf),
                q=aligned(M, K, dtype=u8), sf=aligned(M, K // 32, dtype=u8), w=aligned(K, dtype=f32),
                rstd=aligned(M, dtype=f32), dw=aligned(K, dtype=f32),
                ws=aligned(G.gemm_rmsnorm_backward_workspace(M, K), dtype=u8), codes=aligned(N, K // 2, dtype=u8),
                scales=aligned(N, 16, dtype=bf), zeros=aligned(N, 16, dtype=u8), c=aligned(M, N, dtype=f32))


CALLS = {
    "norm": lambda o, **k: G.gemm_rmsnorm(o["x"], None, None, o["w"], o["y"], o["q"], o["sf"], o["rstd"], M, K, K, 0, 0, K,
                                          K, **k),
    "back": lambda o, **k: G.gemm_rmsnorm_backward(o["x"], o["h"], o["w"], o["rstd"], None, o["dh"], o["dw"], o["ws"], M, K,
                                                   K, K, 0, K, **k),
    "quantize": lambda o, **k: G.gemm_mxfp8_quantize(o["x"], o["q"], o["sf"], M, K, K, K, **k),
    "w4": lambda o, **k: G.gemm_bf16_w4(o["x"], o["codes"], o["scales"], o["zeros"], o["c"], M, N, K, K, K // 2, 16, N, 64,
                                        **k),
}


def status(name, o):
    with pytest.raises(G.GemmError) as e:
        CALLS[name](o)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("name", CALLS)
def test_these_calls_pass_every_check(name):
    assert status(name, operands())[0] == 4


@pytest.mark.parametrize("name,what", [("norm", "w"), ("norm", "sf"), ("norm", "rstd"), ("back", "w"), ("back", "rstd"),
                                       ("back", "dw"), ("back", "ws"), ("quantize", "sf")])
def test_operands_without_a_pitch_have_to_be_contiguous(name, what):
    """A column of a matrix, a slice of wider rows, a broadcast element: the call
    would read or write elements that are not the tensor's."""
    o = operands()
    t = o[what]
    wide = torch.zeros(*t.shape, 2, dtype=t.dtype)
    o[what] = wide[..., 0]
    assert o[what].shape == t.shape and not o[what].is_contiguous()
    got, text = status(name, o)
    assert got == 1 and "not contiguous" in text
    o[what] = torch.zeros(1, dtype=t.dtype).expand(t.shape)
    assert status(name, o)[0] == 1


def test_a_matrix_with_a_pitch_may_be_a_slice():
    o = operands()
    o["x"] = torch.zeros(M, 2 * K, dtype=torch.bfloat16)[:, :K]
    with pytest.raises(G.GemmError) as e:
        G.gemm_mxfp8_quantize(o["x"], o["q"], o["sf"], M, K, 2 * K, K)
    assert e.value.status == 4


@pytest.mark.parametrize("name,what,bad", [
    ("norm", "x", torch.float16), ("back", "ws", None), ("quantize", "q", torch.bfloat16), ("w4", "c", torch.bfloat16)])
def test_without_check_a_refused_operand_is_a_status(name, what, bad):
    """As for the library's own refusals: check=False returns the status."""
    o = operands()
    assert CALLS[name](o, check=False) == 4
    o[what] = torch.zeros(*o[what].shape, 2, dtype=o[what].dtype)[..., 0] if bad is None else o[what].to(bad)
    assert CALLS[name](o, check=False) == 1
    with pytest.raises(G.GemmError):
        CALLS[name](o)


def test_a_torch_without_the_private_functions(monkeypatch):
    """The two functions that the binding asks for the current device and its
    stream are torch's own; without them its public ones answer, and without
    CUDA at all the status is the library's."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(G, "_DTYPES", {})
    asked = []

    class Queue:
        cuda_stream = 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: asked.append(dev) or Queue)
    assert status("norm", operands())[0] == 4 and asked == [-1]

    def no_cuda():
        raise AssertionError("Torch not compiled with CUDA enabled")

    monkeypatch.setattr(G, "_DTYPES", {})
    monkeypatch.setattr(torch.cuda, "current_device", no_cuda)
    for name in CALLS:
        got, text = status(name, operands())
        assert got == 4 and "Torch not compiled with CUDA enabled" in text
        assert CALLS[name](operands(), check=False) == 4


def test_no_driver_is_the_library_s_status(monkeypatch):
    monkeypatch.setattr(G, "_DTYPES", {})
    for name in CALLS:
        got, text = status(name, operands())
        assert got == 4 and "driver" in text
