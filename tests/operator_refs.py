"""Plain references in 64 bits for the operators around the products, written
from their formulas, and guarded buffers to run the kernels on."""
import numpy as np
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

F32, BF16 = G.OUT_F32, G.OUT_BF16
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}      # of a rounding, relative
U32 = 2.0 ** -24
TINY = 1e-37                                        # below fp32's normal range


def pad(n, multiple):
    return -(-n // multiple) * multiple


class Buffer:
    """rows x cols of a type inside a larger allocation: two guard rows on
    either side and `extra` columns on the right, all filled with a byte
    pattern (a NaN in every type used here) that must survive."""

    def __init__(self, rows, cols, dtype, ld=None, fill=None, align=16):
        esize = torch.empty(0, dtype=dtype).element_size()
        self.rows, self.cols, self.dtype, self.esize = rows, cols, dtype, esize
        self.ld = ld if ld is not None else pad(cols, align // esize) + align // esize
        self.raw = torch.full(((rows + 4) * self.ld * esize,), 0xFF, dtype=torch.uint8, device="cuda")
        self.all = self.raw.view(dtype).view(rows + 4, self.ld)
        self.t = self.all[2:2 + rows]
        if fill is not None:
            self.t[:, :cols] = fill.to(dtype).cuda()

    @property
    def ptr(self):
        return self.t.data_ptr()

    def get(self):
        return self.t[:, :self.cols].detach().cpu()

    def f64(self):
        return self.get().to(torch.float64).numpy()

    def guards_ok(self):
        b = self.raw.view(self.rows + 4, self.ld * self.esize)
        inner = b[2:2 + self.rows, self.cols * self.esize:]
        return bool((b[:2] == 0xFF).all() and (b[2 + self.rows:] == 0xFF).all() and (inner == 0xFF).all())


def normal(seed, rows, cols, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    return x * torch.exp(spread * torch.randn(cols, generator=g)) if spread else x


def mx_reference(v):
    """E8M0 bytes and E4M3 codes of fp64 values v (rows x cols, cols % 32 == 0),
    by comparisons with the powers of two themselves."""
    rows, cols = v.shape
    b = v.reshape(rows, cols // 32, 32)
    finite = np.isfinite(b)
    amax = np.max(np.where(finite, np.abs(b), 0.0), axis=2)
    limits = 448.0 * 2.0 ** np.arange(-127, 128, dtype=np.float64)      # index = byte
    byte = np.searchsorted(limits, amax, side="left").astype(np.int64)
    scaled = np.where(finite, b, 0.0) * 2.0 ** (127.0 - byte)[:, :, None]
    codes = torch.from_numpy(scaled.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    codes[~finite] = 0x7F
    return codes.reshape(rows, cols), byte.astype(np.uint8)


def mx_values(codes, sf):
    """fp64 values that codes and scale bytes stand for."""
    c = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()
    return c * np.repeat(2.0 ** (sf.astype(np.float64) - 127), 32, axis=1)


def rmsnorm_reference(h, w, eps):
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def w4_reference(a, codes, scales, zeros, group, K):
    """C and sum |a s (q - z)| from a [M, K], code bytes [N, >= K/2], scales
    [N, groups], zeros [N, groups] (all fp64 or integer arrays)."""
    b = codes[:, :K // 2].astype(np.int64)
    q = np.empty((codes.shape[0], K))
    q[:, 0::2], q[:, 1::2] = b % 16, b // 16
    at = np.arange(K) // group
    w = (q - zeros[:, at]) * scales[:, at]
    return a @ w.T, np.abs(a) @ np.abs(w).T
