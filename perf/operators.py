"""Timed cases of the operators around the library's matrix products: the RMS
norm with the residual's addition (forward and backward, with a bf16 or an
MXFP8 output), the MXFP8 quantiser in both storage orders, and the product
with 4-bit weights and group scales.

Every case can be run in two ways.  With ``own`` false, ``run`` computes the
operator from elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true it makes the library's call.  ``exact`` computes the same
outputs in 64 bits from the operator's definition.
"""
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-5
# rows of per-block partial sums that the backward pass may keep
PARTIAL_ROWS = 296


def listed():
    return [
        # one generated token: the norm before a decoder layer's first product
        {"name": "norm_token", "op": "norm", "M": 1, "K": 8192, "x": "bf16", "h": "bf16", "out": "bf16", "rstd": False},
        # a decoding batch whose layer runs on the block-scaled product
        {"name": "norm_batch_mx", "op": "norm", "M": 16, "K": 8192, "x": "bf16", "h": "bf16", "out": "mx", "rstd": False},
        # training with an fp32 residual stream, ragged sizes
        {"name": "norm_train_ragged", "op": "norm", "M": 4000, "K": 3000, "x": "bf16", "h": "f32", "out": "bf16", "rstd": True},
        # a long prompt, or a training step on the block-scaled product
        {"name": "norm_prompt_mx", "op": "norm", "M": 8192, "K": 8192, "x": "bf16", "h": "bf16", "out": "mx", "rstd": True},
        # a small training step of a norm without a residual branch
        {"name": "back_small", "op": "back", "M": 1000, "K": 2000, "dy": "bf16", "h": "bf16", "dh": "bf16", "res": False},
        # training with an fp32 residual stream, ragged sizes
        {"name": "back_train_ragged", "op": "back", "M": 4000, "K": 3000, "dy": "bf16", "h": "f32", "dh": "f32", "res": True},
        # a large training step with a bf16 stream
        {"name": "back_large", "op": "back", "M": 8192, "K": 8192, "dy": "bf16", "h": "bf16", "dh": "bf16", "res": True},
        # activations of a prompt on their way into gemm_mxfp8
        {"name": "quant_rows", "op": "quant", "M": 1000, "K": 8192, "x": "bf16", "layout": "k"},
        # a weight or gradient stored the other way round, for the products of the backward pass
        {"name": "quant_transposed", "op": "quant", "M": 8192, "K": 8192, "x": "bf16", "layout": "mn"},
        # one generated token through a square projection
        {"name": "w4_token", "op": "w4", "M": 1, "N": 4096, "K": 4096, "group": 128, "zeros": False, "c": "bf16"},
        # a decoding batch through a large projection
        {"name": "w4_batch", "op": "w4", "M": 16, "N": 8192, "K": 8192, "group": 128, "zeros": True, "c": "f32"},
        # a larger batch, fine groups and ragged sizes
        {"name": "w4_ragged", "op": "w4", "M": 33, "N": 3000, "K": 4000, "group": 32, "zeros": True, "c": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "back", "quant", "w4"])
    if op == "w4":
        c = {"op": op, "M": _log(rng, 1, 64), "N": _log(rng, 256, 8192), "K": 32 * _log(rng, 16, 256),
             "group": rng.choice([32, 64, 128, 256]), "zeros": rng.random() < 0.5, "c": rng.choice(["bf16", "f32"])}
        return c
    K = _log(rng, 256, 16384)
    M = _log(rng, 1, min(8192, (1 << 25) // K))
    if op == "norm":
        out = rng.choice(["bf16", "mx"])
        if out == "mx":
            K = max(32, K // 32 * 32)
        return {"op": op, "M": M, "K": K, "x": rng.choice(["bf16", "f32"]), "h": rng.choice(["bf16", "f32", "none"]),
                "out": out, "rstd": rng.random() < 0.5}
    if op == "back":
        h = rng.choice(["bf16", "f32"])
        return {"op": op, "M": M, "K": K, "dy": rng.choice(["bf16", "f32"]), "h": h, "dh": h, "res": rng.random() < 0.5}
    return {"op": op, "M": M, "K": max(32, K // 32 * 32), "x": rng.choice(["bf16", "f32"]),
            "layout": rng.choice(["k", "mn"])}


def _pad(n, multiple):
    return -(-n // multiple) * multiple


def _normal(g, rows, cols, dtype, spread=0.0):
    """Normal values whose columns have scales of their own (a few of them
    far larger than the rest, as activations have)."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    if spread:
        x = x * torch.exp(spread * torch.randn(cols, generator=g, device=DEVICE))
    return x.to(dtype)


def _empty(rows, cols, dtype):
    return torch.empty(rows, cols, dtype=dtype, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    s = dict(case)
    if op == "norm":
        ld = s["ld"] = _pad(K, 8)
        s["X"] = _normal(g, M, ld, TYPES[case["x"]], 0.7)
        s["W"] = 1 + 0.2 * torch.randn(K, generator=g, device=DEVICE)
        if case["h"] != "none":
            s["R"] = _normal(g, M, ld, TYPES[case["h"]], 0.7)
            s["H"] = _empty(M, ld, TYPES[case["h"]])
        if case["out"] == "bf16":
            s["Y"] = _empty(M, ld, torch.bfloat16)
        else:
            s["ldq"] = _pad(K, 16)
            s["Q"] = _empty(M, s["ldq"], torch.float8_e4m3fn)
            s["SF"] = _empty(M, K // 32, torch.float8_e8m0fnu)
        if case["rstd"]:
            s["rstd"] = torch.empty(M, device=DEVICE)
    elif op == "back":
        ld = s["ld"] = _pad(K, 8)
        s["dY"] = _normal(g, M, ld, TYPES[case["dy"]]) * 0.01
        s["H"] = _normal(g, M, ld, TYPES[case["h"]], 0.7)
        s["W"] = 1 + 0.2 * torch.randn(K, generator=g, device=DEVICE)
        s["rstd"] = torch.rsqrt(s["H"][:, :K].double().square().mean(1) + EPS).float()
        if case["res"]:
            s["dR"] = _normal(g, M, ld, TYPES[case["dh"]]) * 0.01
        s["dH"] = _empty(M, ld, TYPES[case["dh"]])
        s["dW"] = torch.empty(K, device=DEVICE)
        s["work"] = torch.empty(min(M, PARTIAL_ROWS) * K, device=DEVICE)
    elif op == "quant":
        if case["layout"] == "k":
            s["ld"] = _pad(K, 8)
            s["X"] = _normal(g, M, s["ld"], TYPES[case["x"]], 0.7)
        else:
            s["ld"] = _pad(M, 8)
            s["X"] = _normal(g, K, s["ld"], TYPES[case["x"]], 0.7)
        s["ldq"] = _pad(K, 16)
        s["Q"] = _empty(M, s["ldq"], torch.float8_e4m3fn)
        s["SF"] = _empty(M, K // 32, torch.float8_e8m0fnu)
    else:
        N, G = case["N"], case["group"]
        groups = -(-K // G)
        s["A"] = _normal(g, M, K, torch.bfloat16)
        s["ldb"] = _pad(K // 2, 16)
        s["B"] = torch.randint(0, 256, (N, s["ldb"]), generator=g, device=DEVICE, dtype=torch.uint8)
        s["lds"] = _pad(groups, 16)
        s["S"] = (0.02 * torch.exp(0.3 * torch.randn(N, s["lds"], generator=g, device=DEVICE))).to(torch.bfloat16)
        s["Z"] = torch.randint(5, 11, (N, s["lds"]), generator=g, device=DEVICE, dtype=torch.uint8) \
            if case["zeros"] else None
        s["ldc"] = _pad(N, 8)
        s["C"] = _empty(M, s["ldc"], TYPES[case["c"]])
    return s


# ------------------------------------------------------------ plain forms --


def _blocks_to_mx(y):
    """Codes and scales of the last axis, 32 at a time: the scale is the
    smallest power of two that brings the block's largest value within 448."""
    rows, cols = y.shape
    b = y.reshape(rows, cols // 32, 32)
    m, e = torch.frexp(b.abs().amax(2))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, -127, e).clamp(-127, 127)
    q = (torch.ldexp(b, -e[:, :, None])).to(torch.float8_e4m3fn).reshape(rows, cols)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_norm(s):
    K = s["K"]
    x = s["X"][:, :K].float()
    out = {}
    if s["h"] != "none":
        out["h"] = (x + s["R"][:, :K].float()).to(TYPES[s["h"]])
        x = out["h"].float()
    rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
    y = x * rstd[:, None] * s["W"]
    if s["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        out["codes"], out["scales"] = _blocks_to_mx(y)
    if s["rstd"] is not False:
        out["rstd"] = rstd
    return out


def _plain_back(s):
    K = s["K"]
    dy, h, r = s["dY"][:, :K].float(), s["H"][:, :K].float(), s["rstd"][:, None]
    n = h * r
    gw = dy * s["W"]
    dh = r * (gw - n * (gw * n).mean(1, keepdim=True))
    if s["res"]:
        dh = dh + s["dR"][:, :K].float()
    return {"dh": dh.to(TYPES[s["dh"]]), "dw": (dy * n).sum(0)}


def _plain_quant(s):
    x = s["X"][:, :s["K"]] if s["layout"] == "k" else s["X"][:, :s["M"]].t()
    codes, scales = _blocks_to_mx(x.float())
    return {"codes": codes, "scales": scales}


def _plain_w4(s):
    N, K, G = s["N"], s["K"], s["group"]
    b = s["B"][:, :K // 2]
    q = torch.stack((b & 15, b >> 4), 2).reshape(N, K).float()
    at = torch.arange(K, device=q.device) // G
    z = s["Z"][:, at].float() if s["Z"] is not None else 8.0
    w = (q - z) * s["S"][:, at].float()
    return {"c": (s["A"].float() @ w.t()).to(TYPES[s["c"]])}


# ------------------------------------------------------- the library's calls --


def _own(s):
    import dense_gemm_engineering_bf16_b200 as lib
    code = {"f32": lib.OUT_F32, "bf16": lib.OUT_BF16}
    op, M, K = s["op"], s["M"], s["K"]
    if op == "norm":
        res = s["h"] != "none"
        rstd = s["rstd"] if s["rstd"] is not False else None
        ld = s["ld"]
        mx = s["out"] == "mx"
        lib.gemm_rmsnorm(s["X"], s["R"] if res else None, s["H"] if res else None, s["W"], None if mx else s["Y"],
                         s["Q"] if mx else None, s["SF"] if mx else None, rstd, M, K, ld, ld, ld, ld,
                         s["ldq"] if mx else 0, code[s["x"]], code[s["h"]] if res else code[s["x"]], EPS)
        out = {"h": s["H"][:, :K]} if res else {}
        if mx:
            out["codes"], out["scales"] = s["Q"][:, :K], s["SF"]
        else:
            out["y"] = s["Y"][:, :K]
        if rstd is not None:
            out["rstd"] = rstd
        return out
    if op == "back":
        ld = s["ld"]
        lib.gemm_rmsnorm_backward(s["dY"], s["H"], s["W"], s["rstd"], s["dR"] if s["res"] else None, s["dH"], s["dW"],
                                  s["work"], M, K, ld, ld, ld, ld, code[s["dy"]], code[s["h"]], code[s["dh"]])
        return {"dh": s["dH"][:, :K], "dw": s["dW"]}
    if op == "quant":
        lib.gemm_mxfp8_quantize(s["X"], s["Q"], s["SF"], M, K, s["ld"], s["ldq"], code[s["x"]],
                                lib.KMAJOR if s["layout"] == "k" else lib.MNMAJOR)
        return {"codes": s["Q"][:, :K], "scales": s["SF"]}
    lib.gemm_bf16_w4(s["A"], s["B"], s["S"], s["Z"], s["C"], M, s["N"], K, K, s["ldb"], s["lds"], s["ldc"], s["group"],
                     code[s["c"]])
    return {"c": s["C"][:, :s["N"]]}


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "back": _plain_back, "quant": _plain_quant, "w4": _plain_w4}[s["op"]](s)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    n = M * K
    mx = n + n // 32
    if op == "norm":
        moved = n * BYTES[case["x"]] + 4 * K + (2 * n * BYTES[case["h"]] if case["h"] != "none" else 0)
        moved += mx if case["out"] == "mx" else 2 * n
        return {"bytes": moved + (4 * M if case["rstd"] else 0), "flops": 5 * n}
    if op == "back":
        moved = n * (BYTES[case["dy"]] + BYTES[case["h"]] + BYTES[case["dh"]] * (2 if case["res"] else 1))
        return {"bytes": moved + 8 * K + 4 * M, "flops": 9 * n}
    if op == "quant":
        return {"bytes": n * BYTES[case["x"]] + mx, "flops": 2 * n}
    N, groups = case["N"], -(-K // case["group"])
    weights = N * K // 2 + N * groups * (3 if case["zeros"] else 2)
    return {"bytes": weights + 2 * n + M * N * BYTES[case["c"]], "flops": 2 * M * N * K}


# ---------------------------------------------------------------- in 64 bits --


def _exact_mx(y):
    """What the codes stand for before their rounding (value over scale), and
    the scales, by logarithms (bf16 and fp32 values are at least 1.7e-7 apart
    there, so the offset only takes up the logarithm's own error)."""
    top = y.abs().unflatten(1, (-1, 32)).max(2).values
    e = torch.ceil(torch.log2(top / 448) - 1e-9).clamp(min=-127)
    scale = torch.pow(2.0, e)
    return y / scale.repeat_interleave(32, 1), scale


def exact(case, seed):
    s = prepare(case, seed)
    op, K, M = case["op"], case["K"], case["M"]
    out = {}
    if op == "norm":
        v = s["X"].double()[:, :K]
        if case["h"] != "none":
            v = s["R"].double()[:, :K].add(v)
            out["h"] = v
            v = v.to(TYPES[case["h"]]).double()      # the norm is of the stored sum
        rms = (v.pow(2).sum(1).div(K) + EPS).sqrt()
        y = v.div(rms.unsqueeze(1)).mul(s["W"].double().unsqueeze(0))
        if case["out"] == "bf16":
            out["y"] = y
        else:
            out["codes"], out["scales"] = _exact_mx(y)
        if case["rstd"]:
            out["rstd"] = rms.reciprocal()
        return out
    if op == "back":
        dy, h = s["dY"].double()[:, :K], s["H"].double()[:, :K]
        rstd = s["rstd"].double().unsqueeze(1)
        dot = torch.einsum("ij,ij,j->i", dy, h, s["W"].double()).unsqueeze(1)
        dh = dy * s["W"].double() * rstd - h * (dot * rstd.pow(3) / K)
        if case["res"]:
            dh += s["dR"].double()[:, :K]
        return {"dh": dh, "dw": torch.einsum("ij,ij,i->j", dy, h, rstd.squeeze(1))}
    if op == "quant":
        x = s["X"].double()[:, :K] if case["layout"] == "k" else s["X"].double()[:, :M].t().contiguous()
        out["codes"], out["scales"] = _exact_mx(x)
        return out
    # group by group: scale times (codes . x - zero * sum x)
    N, G = case["N"], case["group"]
    a, b = s["A"].double(), s["B"].long()
    c = torch.zeros(M, N, dtype=torch.float64, device=a.device)
    for i, lo in enumerate(range(0, K, G)):
        hi = min(K, lo + G)
        codes = b[:, lo // 2:hi // 2]
        part = a[:, lo:hi:2] @ (codes % 16).double().t() + a[:, lo + 1:hi:2] @ (codes // 16).double().t()
        zero = s["Z"][:, i].double() if case["zeros"] else torch.full((N,), 8.0, dtype=torch.float64, device=a.device)
        c += s["S"][:, i].double() * (part - a[:, lo:hi].sum(1, keepdim=True) * zero)
    return {"c": c}
