"""The products grouped by expert and the 4-bit operators on the host: every
documented refusal gives its status before anything is queued, empty problems
succeed, pitches and extents are bounded before they are multiplied, and the
binding checks its tensors.  No kernel is launched here."""
import ctypes

import pytest
import torch

import dense_gemm_engineering_bf16_b200 as pkg
from dense_gemm_engineering_bf16_b200 import gemm as G

# far apart, 16-byte aligned, never dereferenced
P = [0x7F0000000000 + i * 0x10000000 for i in range(8)]
F32, BF16, MX, NV, KM, MN = G.OUT_F32, G.OUT_BF16, G.FP4_MX, G.FP4_NV, G.KMAJOR, G.MNMAJOR
OK, INVALID, MISALIGNED, ALIAS, NO_DEVICE, TOO_LARGE = 0, 1, 2, 3, 4, 7
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")


def grouped(A=P[0], B=P[1], ends=P[2], C=P[3], groups=4, M=64, N=128, K=96, lda=None, ldb=None, strideb=None, ldc=None,
            ct=F32, layout=KM):
    wide, high = (K, N) if layout == KM else (N, K)
    ldb = wide if ldb is None else ldb
    return G.lib.gemm_bf16_grouped(A, B, ends, C, groups, M, N, K, K if lda is None else lda, ldb,
                                   high * ldb if strideb is None else strideb, N if ldc is None else ldc, ct, layout, 0)


def wgrad(dC=P[0], A=P[1], ends=P[2], dB=P[3], groups=4, M=64, N=128, K=96, lddc=None, lda=None, lddb=None, stridedb=None,
          dt=F32, layout=KM, beta=0.0):
    wide, high = (K, N) if layout == KM else (N, K)
    lddb = wide if lddb is None else lddb
    return G.lib.gemm_bf16_grouped_wgrad(dC, A, ends, dB, groups, M, N, K, N if lddc is None else lddc,
                                         K if lda is None else lda, lddb, high * lddb if stridedb is None else stridedb, dt,
                                         layout, ctypes.c_float(beta), 0)


def quantize(X=P[0], scale=0, Q=P[1], sf=P[2], M=64, K=128, ldx=None, ldq=None, form=NV, xt=BF16, layout=KM):
    return G.lib.gemm_fp4_quantize(X, scale, Q, sf, M, K, (K if layout == KM else M) if ldx is None else ldx,
                                   K // 2 if ldq is None else ldq, form, xt, layout, 0)


def product(A=P[0], sfa=P[1], ga=0, B=P[2], sfb=P[3], gb=0, C=P[4], M=64, N=128, K=256, lda=None, ldb=None, ldc=None,
            form=NV, ct=F32):
    return G.lib.gemm_fp4(A, sfa, ga, B, sfb, gb, C, M, N, K, K // 2 if lda is None else lda,
                          K // 2 if ldb is None else ldb, N if ldc is None else ldc, form, ct, 0)


def test_grouped_refuses_bad_arguments():
    assert grouped(groups=-1) == INVALID and grouped(M=-1) == INVALID and grouped(N=-1) == INVALID and grouped(K=-1) == INVALID
    assert grouped(ct=2) == INVALID and grouped(layout=2) == INVALID and grouped(layout=-1) == INVALID
    assert grouped(A=0) == INVALID and grouped(B=0) == INVALID and grouped(ends=0) == INVALID and grouped(C=0) == INVALID
    assert grouped(lda=88) == INVALID and grouped(ldb=88) == INVALID and grouped(ldc=120) == INVALID
    assert grouped(layout=MN, ldb=120) == INVALID
    assert grouped(strideb=127 * 96 + 88) == INVALID and grouped(strideb=0) == INVALID
    assert grouped(A=P[0] + 2) == MISALIGNED and grouped(B=P[1] + 8) == MISALIGNED and grouped(C=P[3] + 4) == MISALIGNED
    assert grouped(ends=P[2] + 2) == MISALIGNED
    assert grouped(lda=100) == MISALIGNED and grouped(ldb=100) == MISALIGNED and grouped(ldc=130) == MISALIGNED
    assert grouped(strideb=128 * 96 + 4) == MISALIGNED and grouped(K=92, lda=96, ldb=92) == MISALIGNED
    assert grouped(C=P[0]) == ALIAS and grouped(C=P[1] + 2 * 3 * 128 * 96) == ALIAS and grouped(C=P[2]) == ALIAS
    assert grouped(groups=1025) == TOO_LARGE and grouped(M=1 << 31) == TOO_LARGE and grouped(K=1 << 31) == TOO_LARGE
    assert grouped(N=1 << 31, ldc=1 << 31) == TOO_LARGE


def test_wgrad_refuses_bad_arguments():
    assert wgrad(groups=-1) == INVALID and wgrad(M=-1) == INVALID and wgrad(N=-1) == INVALID and wgrad(K=-1) == INVALID
    assert wgrad(dt=2) == INVALID and wgrad(layout=2) == INVALID
    assert wgrad(dC=0) == INVALID and wgrad(A=0) == INVALID and wgrad(ends=0) == INVALID and wgrad(dB=0) == INVALID
    assert wgrad(lddc=120) == INVALID and wgrad(lda=88) == INVALID and wgrad(lddb=88) == INVALID
    assert wgrad(stridedb=128 * 96 - 16) == INVALID and wgrad(layout=MN, lddb=120) == INVALID
    assert wgrad(dC=P[0] + 2) == MISALIGNED and wgrad(A=P[1] + 8) == MISALIGNED and wgrad(dB=P[3] + 4) == MISALIGNED
    assert wgrad(ends=P[2] + 1) == MISALIGNED and wgrad(lda=100) == MISALIGNED and wgrad(lddb=98) == MISALIGNED
    assert wgrad(stridedb=128 * 96 + 2) == MISALIGNED
    assert wgrad(dB=P[0]) == ALIAS and wgrad(dB=P[1] - 4 * 3 * 128 * 96) == ALIAS and wgrad(dB=P[2]) == ALIAS
    assert wgrad(groups=1025) == TOO_LARGE and wgrad(M=1 << 31) == TOO_LARGE


def test_quantiser_refuses_bad_arguments():
    assert quantize(M=-1) == INVALID and quantize(K=-32) == INVALID and quantize(K=48) == INVALID
    assert quantize(form=2) == INVALID and quantize(form=-1) == INVALID and quantize(xt=2) == INVALID
    assert quantize(layout=2) == INVALID and quantize(form=MX, scale=P[5]) == INVALID
    assert quantize(X=0) == INVALID and quantize(Q=0) == INVALID and quantize(sf=0) == INVALID
    assert quantize(ldx=120) == INVALID and quantize(ldq=48) == INVALID and quantize(layout=MN, ldx=56) == INVALID
    assert quantize(X=P[0] + 2) == MISALIGNED and quantize(Q=P[1] + 8) == MISALIGNED and quantize(sf=P[2] + 8) == MISALIGNED
    assert quantize(scale=P[5] + 2) == MISALIGNED and quantize(ldx=132) == MISALIGNED and quantize(ldq=72) == MISALIGNED
    assert quantize(Q=P[0]) == ALIAS and quantize(sf=P[0]) == ALIAS and quantize(sf=P[1]) == ALIAS
    assert quantize(scale=P[1] + 4) == ALIAS and quantize(scale=P[2]) == ALIAS
    assert quantize(M=1 << 31) == TOO_LARGE and quantize(K=1 << 31) == TOO_LARGE


def test_4_bit_product_refuses_bad_arguments():
    assert product(M=-1) == INVALID and product(N=-1) == INVALID and product(K=-32) == INVALID and product(K=48) == INVALID
    assert product(form=2) == INVALID and product(ct=2) == INVALID
    assert product(form=MX, ga=P[5]) == INVALID and product(form=MX, gb=P[5]) == INVALID
    for name in ("A", "sfa", "B", "sfb", "C"):
        assert product(**{name: 0}) == INVALID
    assert product(lda=112) == INVALID and product(ldb=112) == INVALID and product(ldc=120) == INVALID
    assert product(A=P[0] + 8) == MISALIGNED and product(B=P[2] + 1) == MISALIGNED and product(C=P[4] + 4) == MISALIGNED
    assert product(sfa=P[1] + 4) == MISALIGNED and product(sfb=P[3] + 8) == MISALIGNED
    assert product(ga=P[5] + 1) == MISALIGNED and product(gb=P[5] + 2) == MISALIGNED
    assert product(lda=136) == MISALIGNED and product(ldb=136) == MISALIGNED and product(ldc=130) == MISALIGNED
    for name in range(4):
        assert product(C=P[name]) == ALIAS
    assert product(C=P[5], ga=P[5] + 16) == ALIAS and product(C=P[5], gb=P[5]) == ALIAS
    assert product(M=1 << 31) == TOO_LARGE and product(N=1 << 31, ldc=1 << 31) == TOO_LARGE


def test_empty_problems_succeed():
    assert grouped(groups=0, ends=0) == OK and grouped(M=0, A=0) == OK and grouped(N=0, C=0) == OK
    assert wgrad(groups=0, ends=0) == OK and wgrad(N=0, dB=0) == OK and wgrad(K=0, dB=0) == OK
    assert quantize(M=0, X=0) == OK and quantize(K=0, Q=0) == OK
    assert product(M=0, C=0) == OK and product(N=0, C=0) == OK


@no_gpu
def test_valid_calls_without_a_device_report_it():
    for ct in (F32, BF16):
        for layout in (KM, MN):
            assert grouped(ct=ct, layout=layout) == NO_DEVICE and wgrad(dt=ct, layout=layout, beta=1.0) == NO_DEVICE
            assert quantize(xt=ct, layout=layout) == NO_DEVICE and quantize(xt=ct, layout=layout, form=MX) == NO_DEVICE
        assert product(ct=ct) == NO_DEVICE and product(ct=ct, form=MX) == NO_DEVICE
    assert grouped(groups=1, strideb=0) == NO_DEVICE and grouped(groups=1, strideb=-5) == NO_DEVICE
    assert grouped(K=0, A=0, B=0) == NO_DEVICE and wgrad(M=0, A=0, dC=0) == NO_DEVICE
    assert grouped(groups=1024) == NO_DEVICE and wgrad(groups=1024, M=0) == NO_DEVICE
    assert grouped(strideb=127 * 96 + 96) == NO_DEVICE and grouped(strideb=1 << 30) in (ALIAS, NO_DEVICE)
    assert quantize(scale=P[5]) == NO_DEVICE and product(ga=P[5], gb=P[6]) == NO_DEVICE
    assert product(K=0, A=0, B=0, sfa=0, sfb=0) == NO_DEVICE


@no_gpu
@pytest.mark.parametrize("ld", [(1 << 62) + 16, (1 << 62) + 32, (1 << 63) - 16, (1 << 61) + 16, 1 << 40])
def test_pitches_and_strides_whose_bytes_wrap(ld):
    for call, names in ((grouped, ("lda", "ldb", "ldc", "strideb")), (wgrad, ("lddc", "lda", "lddb", "stridedb")),
                        (quantize, ("ldx", "ldq")), (product, ("lda", "ldb", "ldc"))):
        for name in names:
            more = {"strideb": 128 * 96} if call is grouped and name == "ldb" else {"stridedb": 128 * 96} if name == "lddb" else {}
            assert call(**{name: ld}, **more) == TOO_LARGE, (call.__name__, name)


@no_gpu
def test_matrices_whose_byte_range_wraps():
    huge = (1 << 38) - 64
    assert grouped(M=1 << 26, lda=huge) == TOO_LARGE and grouped(M=1 << 26, ldc=huge) == TOO_LARGE
    assert grouped(N=1 << 26, ldc=1 << 26, ldb=huge, strideb=huge) == TOO_LARGE
    assert wgrad(M=1 << 26, lda=huge) == TOO_LARGE and wgrad(M=1 << 26, lddc=huge) == TOO_LARGE
    assert wgrad(N=1 << 26, lddc=1 << 26, lddb=huge, stridedb=huge) == TOO_LARGE
    assert quantize(M=1 << 26, ldx=huge) == TOO_LARGE and quantize(M=1 << 26, ldq=huge) == TOO_LARGE
    assert product(M=1 << 26, lda=huge) == TOO_LARGE and product(M=1 << 26, ldc=huge) == TOO_LARGE
    # more scale tiles than a 32-bit coordinate counts
    assert product(M=1 << 30, K=1 << 30, ldc=128, C=1 << 60, A=16, B=1 << 61, sfa=1 << 62, sfb=3 << 61) == TOO_LARGE


def test_scale_bytes():
    for form, block in ((MX, 32), (NV, 16)):
        for rows, K in ((1, 32), (128, 128), (129, 160), (8192, 8192), (5, 96), (1 << 31 - 1, 32)):
            assert G.gemm_fp4_scale_bytes(rows, K, form) == 512 * -(-rows // 128) * -(-K // (4 * block))
        assert G.gemm_fp4_scale_bytes(0, 32, form) == G.gemm_fp4_scale_bytes(4, 0, form) == 0
        assert G.gemm_fp4_scale_bytes(-1, 32, form) == G.gemm_fp4_scale_bytes(4, 1 << 31, form) == 0
    assert G.gemm_fp4_scale_bytes(4, 32, 2) == 0


def test_package_exports_the_operators():
    for name in ("gemm_bf16_grouped", "gemm_bf16_grouped_wgrad", "gemm_fp4", "gemm_fp4_quantize", "gemm_fp4_scale_bytes",
                 "FP4_MX", "FP4_NV"):
        assert getattr(pkg, name) is getattr(G, name)


# ---------------------------------------------------------------- binding --

E, M_, N_, K_ = 3, 16, 64, 128


def operands(form=NV):
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    zeros = lambda *s, dtype: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(a=zeros(M_, K_, dtype=bf), b=zeros(E, N_, K_, dtype=bf), ends=zeros(E, dtype=i32), c=zeros(M_, N_, dtype=f32),
                dc=zeros(M_, N_, dtype=bf), db=zeros(E, N_, K_, dtype=f32), q=zeros(M_, K_ // 2, dtype=u8),
                w=zeros(N_, K_ // 2, dtype=u8), sf=zeros(G.gemm_fp4_scale_bytes(M_, K_, form), dtype=u8),
                sfw=zeros(G.gemm_fp4_scale_bytes(N_, K_, form), dtype=u8), g=zeros(1, dtype=f32), gw=zeros(1, dtype=f32))


CALLS = {
    "grouped": lambda o, **k: G.gemm_bf16_grouped(o["a"], o["b"], o["ends"], o["c"], E, M_, N_, K_, K_, K_, N_ * K_, N_, **k),
    "wgrad": lambda o, **k: G.gemm_bf16_grouped_wgrad(o["dc"], o["a"], o["ends"], o["db"], E, M_, N_, K_, N_, K_, K_, N_ * K_,
                                                      **k),
    "quantize": lambda o, **k: G.gemm_fp4_quantize(o["a"], o["g"], o["q"], o["sf"], M_, K_, K_, K_ // 2, **k),
    "product": lambda o, **k: G.gemm_fp4(o["q"], o["sf"], o["g"], o["w"], o["sfw"], o["gw"], o["c"], M_, N_, K_, K_ // 2,
                                         K_ // 2, N_, **k),
}


@pytest.fixture
def host_is_the_device(monkeypatch):
    G._here(0)
    monkeypatch.setitem(G._DTYPES, "device", lambda: torch.empty(0).get_device())
    monkeypatch.setitem(G._DTYPES, "stream", lambda dev: 0)


def status(name, o):
    with pytest.raises(G.GemmError) as e:
        CALLS[name](o)
    return e.value.status, str(e.value)


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_binding_passes_valid_calls_on(name, host_is_the_device):
    assert status(name, operands())[0] == NO_DEVICE
    assert CALLS[name](operands(), check=False) == NO_DEVICE


@no_gpu
@pytest.mark.parametrize("name,what,dtype", [
    ("grouped", "a", torch.float16), ("grouped", "b", torch.float32), ("grouped", "ends", torch.int64),
    ("grouped", "c", torch.bfloat16), ("wgrad", "dc", torch.float32), ("wgrad", "db", torch.bfloat16),
    ("wgrad", "ends", torch.float32), ("quantize", "q", torch.int8), ("quantize", "sf", torch.float8_e8m0fnu),
    ("quantize", "g", torch.bfloat16), ("product", "w", torch.int32), ("product", "sfw", torch.float8_e8m0fnu),
    ("product", "gw", torch.float64), ("product", "c", torch.bfloat16)])
def test_binding_checks_types(name, what, dtype, host_is_the_device):
    o = operands()
    o[what] = o[what].to(dtype)
    got, text = status(name, o)
    assert got == INVALID and str(dtype) in text
    assert CALLS[name](o, check=False) == INVALID


@no_gpu
def test_binding_takes_the_formats_own_types(host_is_the_device):
    o = operands()
    o["sf"], o["sfw"] = (o[n].view(torch.float8_e4m3fn) for n in ("sf", "sfw"))
    if hasattr(torch, "float4_e2m1fn_x2"):
        o["q"], o["w"] = (o[n].view(torch.float4_e2m1fn_x2) for n in ("q", "w"))
    assert status("quantize", o)[0] == NO_DEVICE and status("product", o)[0] == NO_DEVICE


@no_gpu
@pytest.mark.parametrize("name,what", [("grouped", "ends"), ("wgrad", "ends"), ("quantize", "sf"), ("product", "sf"),
                                       ("product", "sfw")])
def test_binding_wants_operands_without_a_pitch_contiguous(name, what, host_is_the_device):
    o = operands()
    o[what] = torch.zeros(*o[what].shape, 2, dtype=o[what].dtype)[..., 0]
    got, text = status(name, o)
    assert got == INVALID and "not contiguous" in text


@no_gpu
def test_binding_refuses_what_is_no_64_bit_number(host_is_the_device):
    for name in CALLS:
        for bad in (1 << 63, 2.5, "8"):
            with pytest.raises(G.GemmError) as e:
                CALLS[name](operands(), stream=bad) if bad == 1 << 63 else \
                    G.gemm_fp4_quantize(None, None, None, None, bad, 32, 32, 16, stream=0)
            assert e.value.status == INVALID


def test_call_by_words():
    """The words mean what the entry points' arguments mean, and nothing that a type does not hold passes."""
    import struct
    call = lambda entry, form, *w: G.lib.gemm_call(entry, struct.pack(form, *w))  # noqa: E731
    assert call(0, "<15q", *P[:4], 4, 64, 128, 96, 96, 96, 128 * 96, 128, 0, 2, 0) == INVALID      # layout
    assert call(0, "<15q", *P[:4], 4, 0, 128, 96, 96, 96, 128 * 96, 128, 0, 0, 0) == OK
    assert call(0, "<15q", *P[:4], 4, 0, 128, 96, 96, 96, 128 * 96, 128, 1 << 32, 0, 0) == INVALID
    assert call(0, "<15q", *P[:3], P[0], 4, 64, 128, 96, 96, 96, 128 * 96, 128, 0, 0, 0) == ALIAS
    assert call(1, "<14qf4xq", *P[:4], 4, 64, 0, 96, 96, 96, 96, 128 * 96, 0, 0, 1.0, 0) == OK
    assert call(1, "<14qf4xq", *P[:4], 4, 64, 128, 96, 128, 96, 98, 128 * 96, 0, 0, 1.0, 0) == MISALIGNED
    assert call(1, "<14qf4xq", *P[:4], 4, 64, 128, 96, 128, 96, 96, 128 * 96, 0, (1 << 32) + 1, 1.0, 0) == INVALID
    assert call(2, "<12q", P[0], 0, P[1], P[2], 64, 0, 128, 64, NV, BF16, KM, 0) == OK
    assert call(2, "<12q", P[0], 0, P[1], P[0], 64, 128, 128, 64, NV, BF16, KM, 0) == ALIAS
    assert call(2, "<12q", P[0], 0, P[1], P[2], 64, 128, 128, 64, NV - (1 << 32), BF16, KM, 0) == INVALID
    assert call(3, "<16q", P[0], P[1], 0, P[2], P[3], 0, P[4], 0, 128, 256, 128, 128, 128, NV, F32, 0) == OK
    assert call(3, "<16q", P[0], P[1], 0, P[2], P[3], 0, P[4], 64, 128, 256, 112, 128, 128, NV, F32, 0) == INVALID
    assert call(3, "<16q", P[0], P[1], 0, P[2], P[3], 0, P[4], 64, 128, 256, 128, 128, 128, NV, 1 << 32, 0) == INVALID
    assert call(4, "<16q", *[0] * 16) == INVALID and call(-1, "<16q", *[0] * 16) == INVALID
    assert G.lib.gemm_call(0, None) == INVALID
    if not torch.cuda.is_available():
        assert call(0, "<15q", *P[:4], 4, 64, 128, 96, 96, 96, 128 * 96, 128, 0, 0, 0) == NO_DEVICE
        assert call(1, "<14qf4xq", *P[:4], 4, 64, 128, 96, 128, 96, 96, 128 * 96, 0, 0, 1.0, 0) == NO_DEVICE
        assert call(2, "<12q", P[0], P[5], P[1], P[2], 64, 128, 128, 64, NV, BF16, KM, 0) == NO_DEVICE
        assert call(3, "<16q", P[0], P[1], 0, P[2], P[3], 0, P[4], 64, 128, 256, 128, 128, 128, NV, F32, 0) == NO_DEVICE


@no_gpu
def test_binding_refuses_formats_it_does_not_know(host_is_the_device):
    for name in ("quantize", "product"):
        with pytest.raises(G.GemmError) as e:
            CALLS[name](operands(), format=7)
        assert e.value.status == INVALID
