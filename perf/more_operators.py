"""Timed cases of the products that leave the dense bf16 path: products grouped
by expert (forward, gradient of the inputs, gradient of the weights) and 4-bit
floating-point projections (activations quantised, then multiplied with 4-bit
weights; and the product alone).

Every case can be run in two ways.  With ``own`` false, ``run`` computes the
operator from elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true it makes the library's calls.  ``exact`` computes the same
outputs in 64 bits from the operator's definition.
"""
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
BLOCK = {"mx": 32, "nv": 16}        # elements that share a scale


def listed():
    return [
        # one generated token: its two experts of eight
        {"name": "experts_token", "op": "grouped", "M": 2, "N": 4096, "K": 2048, "groups": 8, "sizes": "even",
         "b": "k", "c": "bf16", "spare": 0},
        # a decoding batch of 64 tokens, two of 64 experts each
        {"name": "experts_batch", "op": "grouped", "M": 128, "N": 2048, "K": 4096, "groups": 64, "sizes": "skewed",
         "b": "k", "c": "bf16", "spare": 0},
        # a long prompt or a training step, forward
        {"name": "experts_prompt", "op": "grouped", "M": 16384, "N": 4096, "K": 2048, "groups": 32, "sizes": "skewed",
         "b": "k", "c": "bf16", "spare": 0},
        # its input gradient on ragged sizes, most experts without a token, a buffer longer than its tokens
        {"name": "experts_back_ragged", "op": "grouped", "M": 5000, "N": 1000, "K": 2500, "groups": 24, "sizes": "few",
         "b": "n", "c": "f32", "spare": 77},
        # the weights' gradient of a small layer, for an fp32 accumulator
        {"name": "wgrad_small", "op": "wgrad", "M": 1000, "N": 1024, "K": 512, "groups": 8, "sizes": "skewed",
         "b": "k", "c": "f32", "spare": 0},
        # the weights' gradient of a large training step
        {"name": "wgrad_large", "op": "wgrad", "M": 16384, "N": 4096, "K": 2048, "groups": 32, "sizes": "skewed",
         "b": "n", "c": "bf16", "spare": 0},
        # one generated token through a 4-bit projection
        {"name": "fp4_token", "op": "linear", "M": 1, "N": 8192, "K": 8192, "format": "nv", "x": "bf16", "layout": "k",
         "c": "bf16"},
        # a decoding batch, power-of-two scales
        {"name": "fp4_batch", "op": "linear", "M": 64, "N": 4096, "K": 4096, "format": "mx", "x": "bf16", "layout": "k",
         "c": "f32"},
        # a long prompt
        {"name": "fp4_prompt", "op": "linear", "M": 8192, "N": 8192, "K": 8192, "format": "nv", "x": "bf16",
         "layout": "k", "c": "bf16"},
        # ragged sizes, fp32 activations
        {"name": "fp4_ragged", "op": "linear", "M": 1000, "N": 2500, "K": 2016, "format": "mx", "x": "f32",
         "layout": "k", "c": "f32"},
        # an operand stored the other way round, as the products of a backward pass need it
        {"name": "fp4_transposed", "op": "linear", "M": 4096, "N": 2048, "K": 4096, "format": "nv", "x": "bf16",
         "layout": "mn", "c": "bf16"},
        # the product alone, of operands that were quantised before
        {"name": "fp4_product", "op": "product", "M": 4096, "N": 8192, "K": 4096, "format": "mx", "x": "bf16",
         "layout": "k", "c": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "wgrad", "linear", "linear", "product"])
    if op in ("grouped", "wgrad"):
        groups = _log(rng, 1, 64)
        N, K = _log(rng, 64, 4096), _log(rng, 64, 4096)
        M = _log(rng, 1, 16384)
        while groups * N * K > 1 << 29:     # the listed weights' bytes
            groups = max(1, groups // 2)
        while M * N * K > 1 << 37:          # the listed prompt's work
            M //= 2
        return {"op": op, "M": M, "N": N, "K": K, "groups": groups, "sizes": rng.choice(["even", "skewed", "few"]),
                "b": rng.choice("kn"), "c": rng.choice(["bf16", "f32"]), "spare": rng.choice([0, 0, rng.randint(1, 300)])}
    return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 256, 8192), "K": 32 * _log(rng, 8, 256),
            "format": rng.choice(["mx", "nv"]), "x": rng.choice(["bf16", "f32"]), "layout": rng.choice(["k", "k", "mn"]),
            "c": rng.choice(["bf16", "f32"])}


def _pad(n, multiple):
    return -(-n // multiple) * multiple


def _normal(g, rows, cols, dtype, spread=0.0):
    """Normal values whose columns have scales of their own (a few of them
    far larger than the rest, as activations have)."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    if spread:
        x = x * torch.exp(spread * torch.randn(cols, generator=g, device=DEVICE))
    return x.to(dtype)


def _group_ends(case, seed):
    """Where each group's rows end: as even as they can be, by expert's
    popularity, or so with three quarters of the experts never chosen."""
    g = torch.Generator().manual_seed(seed)
    M, E = case["M"], case["groups"]
    rank = torch.randperm(E, generator=g)
    if case["sizes"] == "even":
        counts = M // E + (rank < M % E).long()
    else:
        p = torch.exp(0.7 * torch.randn(E, generator=g))
        if case["sizes"] == "few":
            p = p * (rank < max(1, E // 4))
        counts = torch.bincount(torch.multinomial(p, M, replacement=True, generator=g), minlength=E)
    return counts.cumsum(0).to(torch.int32), int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case)
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    if op in ("grouped", "wgrad"):
        E, rows = case["groups"], M + case["spare"]
        ends, s["longest"] = _group_ends(case, seed)
        s["ends"], s["rows"] = ends.to(DEVICE), rows
        s["lda"] = _pad(K, 8)
        s["A"] = _normal(g, rows, s["lda"], torch.bfloat16, 0.5)
        # an expert's matrix is N rows of K ("k") or K rows of N ("n")
        high, wide = (N, _pad(K, 8)) if case["b"] == "k" else (K, _pad(N, 8))
        s["ldb"] = wide
        s["ldc"] = _pad(N, 8)
        if op == "grouped":
            s["B"] = _normal(g, E * high, wide, torch.bfloat16).mul_(K ** -0.5).view(E, high, wide)
            s["C"] = torch.zeros(rows, s["ldc"], dtype=TYPES[case["c"]], device=DEVICE)
        else:
            s["dC"] = _normal(g, rows, s["ldc"], torch.bfloat16).mul_(0.01)
            s["dB"] = torch.empty(E, high, wide, dtype=TYPES[case["c"]], device=DEVICE)
        return s
    f = case["format"]
    s["ldx"] = _pad(K if case["layout"] == "k" else M, 8)
    s["X"] = _normal(g, M if case["layout"] == "k" else K, s["ldx"], TYPES[case["x"]], 0.5)
    s["ldq"] = _pad(K // 2, 16)
    s["gx"] = s["gw"] = None
    if f == "nv":       # a calibrated scale of the whole tensor
        s["gx"] = torch.full((1,), 0.0081, device=DEVICE)
        s["gw"] = torch.full((1,), 0.0021, device=DEVICE)
    w = torch.randn(N, K, generator=g, device=DEVICE)
    codes, scales = _quantise(w, s["gw"], f)
    s["W"], s["sfw"] = _packed(codes, s["ldq"]), _tiled(scales)
    del w, codes, scales
    s["ldc"] = _pad(N, 8)
    s["C"] = torch.empty(M, s["ldc"], dtype=TYPES[case["c"]], device=DEVICE)
    if op == "product":
        codes, scales = _quantise(_activations(s).float(), s["gx"], f)
        s["Q"], s["sf"] = _packed(codes, s["ldq"]), _tiled(scales)
        del s["X"]
    else:
        s["Q"] = torch.empty(M, s["ldq"], dtype=torch.uint8, device=DEVICE)
        s["sf"] = torch.empty(_pad(M, 128) * _pad(-(-K // BLOCK[f]), 4), dtype=torch.uint8, device=DEVICE)
    return s


def _activations(s):
    return s["X"][:, :s["K"]] if s["layout"] == "k" else s["X"][:, :s["M"]].t()


# ------------------------------------------------------------ plain forms --


def _quantise(x, g, f):
    """4-bit codes (0 .. 15) and scale bytes of the rows of x: blocks of 32
    with the smallest power of two that brings the block's largest value
    within 6, or blocks of 16 with that value's sixth in E4M3 under the
    tensor's scale g."""
    b = x.reshape(x.shape[0], -1, BLOCK[f])
    top = b.abs().amax(2)
    if f == "mx":
        m, e = torch.frexp(top)
        e = torch.where(m > 0.75, e - 2, e - 3)
        e = torch.where(m == 0, -127, e).clamp(-127, 127)
        scale = (e + 127).to(torch.uint8)
        q = torch.ldexp(b, -e[:, :, None])
    else:
        e4m3 = (top / (6 * g)).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
        scale = e4m3.view(torch.uint8)
        q = b / (e4m3.float() * g)[:, :, None]
    a = q.abs()
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    code = code + 8 * torch.signbit(b)
    return code.reshape(x.shape), scale


def _packed(codes, ld):
    """Two codes a byte, the even one in the low half."""
    out = torch.zeros(codes.shape[0], ld, dtype=torch.uint8, device=codes.device)
    out[:, :codes.shape[1] // 2] = codes[:, 0::2] | codes[:, 1::2] << 4
    return out


def _tiled(scales):
    """Scale bytes in tiles of 128 rows x 4: row r of a tile at 16 (r % 32) + 4 (r / 32)."""
    rows, cols = scales.shape
    full = torch.zeros(_pad(rows, 128), _pad(cols, 4), dtype=torch.uint8, device=scales.device)
    full[:rows, :cols] = scales
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _dequantised(q, sf, rows, K, f):
    """fp32 values of codes and tiled scales, the tensor's scale aside."""
    b = q[:, :K // 2]
    code = torch.stack((b & 15, b >> 4), 2).reshape(rows, K)
    a = (code & 7).float()
    v = torch.where(a < 4, a / 2, torch.where(a < 6, a - 2, 2 * a - 8))
    v = torch.where(code > 7, -v, v)
    blocks = K // BLOCK[f]
    s = sf.view(-1, _pad(blocks, 4) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, _pad(blocks, 4))[:rows, :blocks]
    s = torch.exp2(s.float() - 127) if f == "mx" else s.contiguous().view(torch.float8_e4m3fn).float()
    return (v.view(rows, blocks, -1) * s[:, :, None]).view(rows, K)


def _plain_fp4(s):
    M, N, K, f = s["M"], s["N"], s["K"], s["format"]
    if s["op"] == "linear":
        codes, scales = _quantise(_activations(s).float(), s["gx"], f)
        x = _dequantised(_packed(codes, s["ldq"]), _tiled(scales), M, K, f)
    else:
        x = _dequantised(s["Q"], s["sf"], M, K, f)
    c = x @ _dequantised(s["W"], s["sfw"], N, K, f).t()
    if f == "nv":
        c = c * (s["gx"] * s["gw"])
    return {"c": c.to(TYPES[s["c"]])}


def _rows_of_groups(s):
    """[groups, longest] row numbers and whether there is such a row."""
    ends = s["ends"].long()
    starts = torch.cat((ends.new_zeros(1), ends[:-1]))
    rows = starts[:, None] + torch.arange(max(1, s["longest"]), device=ends.device)
    return starts, rows.clamp(max=s["rows"] - 1), rows < ends[:, None]


def _plain_grouped(s):
    starts, rows, there = _rows_of_groups(s)
    a = s["A"][:, :s["K"]].float()[rows] * there[:, :, None]
    b = s["B"].float()
    b = b[:, :, :s["K"]].transpose(1, 2) if s["b"] == "k" else b[:, :, :s["N"]]
    c = torch.bmm(a, b)
    row = torch.arange(s["rows"], device=c.device)
    group = torch.searchsorted(s["ends"].long(), row, right=True).clamp(max=s["groups"] - 1)
    c = c[group, (row - starts[group]).clamp(max=c.shape[1] - 1)]
    used = (row < s["ends"][-1])[:, None]
    return {"c": torch.where(used, c.to(s["C"].dtype), s["C"][:, :s["N"]])}


def _plain_wgrad(s):
    _, rows, there = _rows_of_groups(s)
    a = s["A"][:, :s["K"]].float()[rows] * there[:, :, None]
    dc = s["dC"][:, :s["N"]].float()[rows] * there[:, :, None]
    db = torch.bmm(dc.transpose(1, 2), a) if s["b"] == "k" else torch.bmm(a.transpose(1, 2), dc)
    return {"db": db.to(TYPES[s["c"]])}


# ------------------------------------------------------- the library's calls --


def _own(s):
    import dense_gemm_engineering_bf16_b200 as lib
    c_type = {"f32": lib.OUT_F32, "bf16": lib.OUT_BF16}
    op, M, N, K = s["op"], s["M"], s["N"], s["K"]
    if op in ("grouped", "wgrad"):
        layout = lib.KMAJOR if s["b"] == "k" else lib.MNMAJOR
        E, rows, ldb = s["groups"], s["rows"], s["ldb"]
        stride = (N if s["b"] == "k" else K) * ldb
        if op == "grouped":
            lib.gemm_bf16_grouped(s["A"], s["B"], s["ends"], s["C"], E, rows, N, K, s["lda"], ldb, stride, s["ldc"],
                                  c_type[s["c"]], layout)
            return {"c": s["C"][:, :N]}
        lib.gemm_bf16_grouped_wgrad(s["dC"], s["A"], s["ends"], s["dB"], E, rows, N, K, s["ldc"], s["lda"], ldb, stride,
                                    c_type[s["c"]], layout)
        return {"db": s["dB"][:, :, :K if s["b"] == "k" else N]}
    form = {"mx": lib.FP4_MX, "nv": lib.FP4_NV}[s["format"]]
    if op == "linear":
        lib.gemm_fp4_quantize(s["X"], s["gx"], s["Q"], s["sf"], M, K, s["ldx"], s["ldq"], form, c_type[s["x"]],
                              lib.KMAJOR if s["layout"] == "k" else lib.MNMAJOR)
    lib.gemm_fp4(s["Q"], s["sf"], s["gx"], s["W"], s["sfw"], s["gw"], s["C"], M, N, K, s["ldq"], s["ldq"], s["ldc"],
                 form, c_type[s["c"]])
    return {"c": s["C"][:, :N]}


def run(s):
    if own:
        return _own(s)
    return {"grouped": _plain_grouped, "wgrad": _plain_wgrad, "linear": _plain_fp4, "product": _plain_fp4}[s["op"]](s)


def work(case):
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    if op in ("grouped", "wgrad"):
        E = case["groups"]
        used = min(M, max(1, E // 4) if case["sizes"] == "few" else E)
        if op == "grouped":
            moved = 2 * used * N * K + 2 * M * K + M * N * BYTES[case["c"]]
        else:
            moved = E * N * K * BYTES[case["c"]] + 2 * M * (N + K)
        return {"bytes": moved + 4 * E, "flops": 2 * M * N * K}
    block = BLOCK[case["format"]]
    x = M * K * BYTES[case["x"]] if op == "linear" else M * K // 2 + M * K // block
    return {"bytes": x + N * K // 2 + N * K // block + M * N * BYTES[case["c"]], "flops": 2 * M * N * K}


# ---------------------------------------------------------------- in 64 bits --


def _nearest(v, bits, lowest):
    """v >= 0 to the nearest number of `bits` bits whose exponent is at least `lowest`, ties to even."""
    e = torch.floor(torch.log2(v.clamp(min=1e-300))).clamp(min=lowest)
    step = torch.pow(2.0, e - (bits - 1))
    return torch.round(v / step) * step


def _exact_values(x, g, f):
    """What the quantised rows of x stand for, the tensor's scale aside."""
    b = x.unflatten(1, (-1, BLOCK[f]))
    top = b.abs().max(2).values
    if f == "mx":       # bf16 and fp32 values are at least 1.7e-7 apart in log2: the offset only takes up its error
        scale = torch.pow(2.0, torch.ceil(torch.log2(top / 6) - 1e-9).clamp(min=-127))
        unit = scale
    else:
        scale = _nearest(top / (6 * g), 4, -6).clamp(2.0 ** -9, 448)
        unit = scale * g
    v = _nearest(b.abs() / unit.unsqueeze(2), 2, 0).clamp(max=6) * b.sign() * scale.unsqueeze(2)
    return v.flatten(1)


def _exact_codes(q, sf, rows, K, f):
    """The same of stored codes and scales, field by field."""
    out = torch.empty(rows, K, dtype=torch.float64, device=q.device)
    for half in range(2):
        c = (q[:, :K // 2].long() >> (4 * half)) & 15
        e, m = c >> 1 & 3, (c & 1).double()
        v = torch.where(e > 0, (2 + m) * torch.pow(2.0, e.double() - 2), m / 2)
        out[:, half::2] = torch.where(c > 7, -v, v)
    r = torch.arange(rows, device=q.device)[:, None]
    b = torch.arange(K // BLOCK[f], device=q.device)[None, :]
    tiles = _pad(K // BLOCK[f], 4) // 4
    byte = sf[((r // 128) * tiles + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4].long()
    if f == "mx":
        s = torch.pow(2.0, byte.double() - 127)
    else:
        e, m = byte >> 3 & 15, (byte & 7).double()
        s = torch.where(e > 0, (8 + m) * torch.pow(2.0, e.double() - 10), m * 2.0 ** -9)
    return out * s.repeat_interleave(BLOCK[f], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    if op in ("linear", "product"):
        f = case["format"]
        g = s["gx"].double() if f == "nv" else None
        x = _exact_values(_activations(s).double(), g, f) if op == "linear" else _exact_codes(s["Q"], s["sf"], M, K, f)
        c = torch.einsum("mk,nk->mn", x, _exact_codes(s["W"], s["sfw"], N, K, f))
        return {"c": c * g * s["gw"].double() if f == "nv" else c}
    a = s["A"].double()[:, :K]
    lo, parts = 0, []
    c = s["C"].double()[:, :N].clone() if op == "grouped" else None
    for e, hi in enumerate(s["ends"].tolist()):
        if op == "grouped":
            b = s["B"][e].double()
            c[lo:hi] = a[lo:hi] @ (b[:, :K].t() if case["b"] == "k" else b[:, :N])
        else:
            d = s["dC"][lo:hi, :N].double()
            parts.append(d.t() @ a[lo:hi] if case["b"] == "k" else a[lo:hi].t() @ d)
        lo = hi
    return {"c": c} if op == "grouped" else {"db": torch.stack(parts)}
