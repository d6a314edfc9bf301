"""Cases that measure the 8-bit-float operators: the norm that writes 8-bit
activations, the quantisers, the block-scaled product and its grouped form.

Format. An 8-bit tensor holds e4m3 values (largest 448) and one fp32 scale for
each block: one row x 128 columns of an activation, 128 x 128 of a weight
matrix. The value a byte stands for is byte * scale. A scale is the smallest
power of two with amax / scale <= 448 over its block (1 for a block of zeros),
so dividing by it is exact and a byte is the nearest e4m3 value (ties to even).
8-bit activations are stored with rows of ld = columns rounded up to 16 bytes,
zero padded.

Operators (M rows, N output features, K input features, KB = ceil(K / 128)):
  norm      s = x + residual, rounded to the residual's type;
            h = s / sqrt(mean(s^2) + eps) * weight; h as 8 bits and scales,
            and / or as bf16
  quantize  an activation [M][K] to 8 bits and scales
  swiglu    gate|up [M][2 K] to the 8 bits and scales of silu(gate) * up
  encode    weights [N][K] to 8 bits and scales of 128 x 128 blocks
  linear    y[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in b} xq[m][k] wq[n][k] + bias[n]
  grouped   the same with the weights of the expert e whose rows
            [offsets[e], offsets[e + 1]) hold row m
"""
import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    _DEV = torch.device("cuda")
else:
    _DEV = torch.device("cpu")

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BLOCK = 128
_EPS = 1e-6


def listed():
    return [
        # one token of a decode step: the residual is added, the next layer's input written as 8 bits
        {"name": "norm 1x2048", "op": "norm", "rows": 1, "cols": 2048, "x": "bf16", "res": "bf16", "y": False},
        # a small batch whose layer output is still fp32, read by an 8-bit layer and a codebook layer (bf16)
        {"name": "norm 37x3584 f32", "op": "norm", "rows": 37, "cols": 3584, "x": "f32", "res": "f32", "y": True},
        # long prompts
        {"name": "norm 8192x3584", "op": "norm", "rows": 8192, "cols": 3584, "x": "bf16", "res": "bf16", "y": False},
        # the input of an MLP's down projection in a decode batch
        {"name": "quantize 32x11008", "op": "quantize", "rows": 32, "cols": 11008, "x": "bf16"},
        # between the MLP's two products in a prefill
        {"name": "swiglu 2048x14336", "op": "swiglu", "rows": 2048, "cols": 14336, "x": "bf16"},
        # an MLP weight matrix brought into the format
        {"name": "encode 14336x3584", "op": "encode", "rows": 14336, "cols": 3584, "x": "f32"},
        # gate or up projection of one token
        {"name": "linear 1x11008x2048", "op": "linear", "M": 1, "N": 11008, "K": 2048, "out": "bf16", "bias": False},
        # down projection of a ragged decode batch
        {"name": "linear 29x2048x11008", "op": "linear", "M": 29, "N": 2048, "K": 11008, "out": "f32", "bias": True},
        # up projection of a prefill
        {"name": "linear 2048x14336x3584", "op": "linear", "M": 2048, "N": 14336, "K": 3584, "out": "bf16",
         "bias": False},
        # eight tokens, two experts each
        {"name": "grouped 16 e8 2048x2048", "op": "grouped", "M": 16, "E": 8, "N": 2048, "K": 2048, "out": "bf16",
         "bias": False},
        # a prefill over a few large experts
        {"name": "grouped 4096 e8 3584x3584", "op": "grouped", "M": 4096, "E": 8, "N": 3584, "K": 3584, "out": "bf16",
         "bias": False},
        # many small experts with uneven loads, some of them empty
        {"name": "grouped 3001 e64 1000x2048", "op": "grouped", "M": 3001, "E": 64, "N": 1000, "K": 2048, "out": "f32",
         "bias": True},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; half of them as they fall, half rounded to 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 32:
        v = v // 16 * 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "quantize", "swiglu", "encode", "linear", "linear", "grouped", "grouped"])
    if op in ("norm", "quantize", "swiglu", "encode"):
        cols = _spread(rng, 64, 14336)
        rows = _spread(rng, 1, max(1, min(8192, 28_000_000 // cols)))
        c = {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["bf16", "f32"])}
        if op == "norm":
            c["res"] = rng.choice(["bf16", "f32", "none"])
            c["y"] = rng.random() < 0.5
        return c
    N, K = _spread(rng, 64, 14336), _spread(rng, 64, 14336)
    out, bias = rng.choice(["bf16", "f32"]), rng.random() < 0.5
    if op == "linear":
        return {"op": op, "M": _spread(rng, 1, max(1, min(2048, 100_000_000_000 // (N * K)))), "N": N, "K": K,
                "out": out, "bias": bias}
    N, K = min(N, 4096), min(K, 4096)
    E = _spread(rng, 2, max(2, min(64, 130_000_000 // (N * K))))
    return {"op": op, "M": _spread(rng, 1, 4096), "E": E, "N": N, "K": K, "out": out, "bias": bias}


def _ld(cols):
    return -(-cols // 16) * 16


def _activations(gen, rows, cols, scale=1.0):
    """Normal values, with the few large channels that activations of language models have."""
    x = torch.randn(rows, cols, device=_DEV, generator=gen) * scale
    big = torch.rand(cols, device=_DEV, generator=gen) < 0.004
    return x * torch.where(big, 15.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op in ("norm", "quantize", "swiglu"):
        rows, cols, dt = case["rows"], case["cols"], _DT[case["x"]]
        s["x"] = _activations(gen, rows, cols * (2 if op == "swiglu" else 1)).to(dt)
        if op == "norm":
            s["weight"] = 1.0 + 0.2 * torch.randn(cols, device=_DEV, generator=gen)
            s["res"], s["sum"] = None, None
            if case["res"] != "none":
                s["res"] = (_activations(gen, rows, cols) * 4.0).to(_DT[case["res"]])
                s["sum"] = torch.empty_like(s["res"])
            s["y"] = torch.empty(rows, cols, device=_DEV, dtype=torch.bfloat16) if case["y"] else None
        s["q"] = torch.empty(rows, _ld(cols), device=_DEV, dtype=torch.float8_e4m3fn)
        s["scales"] = torch.empty(rows, -(-cols // _BLOCK), device=_DEV)
    elif op == "encode":
        rows, cols = case["rows"], case["cols"]
        s["x"] = (torch.randn(rows, cols, device=_DEV, generator=gen) * 0.02).to(_DT[case["x"]])
        s["q"] = torch.empty(rows, cols, device=_DEV, dtype=torch.float8_e4m3fn)
        s["scales"] = torch.empty(-(-rows // _BLOCK), -(-cols // _BLOCK), device=_DEV)
    else:
        M, N, K, E = case["M"], case["N"], case["K"], case.get("E", 1)
        kb, nb = -(-K // _BLOCK), -(-N // _BLOCK)
        # 8-bit values as a quantiser leaves them, and scales of any size, as stored checkpoints have them
        xq = torch.zeros(M, _ld(K), device=_DEV)
        xq[:, :K] = torch.randn(M, K, device=_DEV, generator=gen) * 100.0
        s["xq"] = xq.clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["xs"] = 0.01 * torch.exp(0.5 * torch.randn(M, kb, device=_DEV, generator=gen))
        wq = torch.empty(E, N, K, device=_DEV, dtype=torch.float8_e4m3fn)
        for e in range(E):
            wq[e] = (torch.randn(N, K, device=_DEV, generator=gen) * 110.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["wq"] = wq
        s["ws"] = 2e-4 * torch.exp(0.3 * torch.randn(E, nb, kb, device=_DEV, generator=gen))
        s["bias"] = torch.randn(E, N, device=_DEV, generator=gen) if case["bias"] else None
        if op == "grouped":
            r = np.random.RandomState(int(seed) % (1 << 31))
            p = np.exp(r.randn(E))
            counts = r.multinomial(M, p / p.sum())
            s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), device=_DEV, dtype=torch.int32)
            s["most"] = int(counts.max())
        s["y"] = torch.empty(M, N, device=_DEV, dtype=_DT[case["out"]])
        if own:
            import vq_compressed_linear_b200 as hxq
            s["layer"] = hxq.Fp8Linear(wq if op == "grouped" else wq[0], s["ws"] if op == "grouped" else s["ws"][0])
            s["out"] = hxq.HXQ_OUT_BF16 if case["out"] == "bf16" else hxq.HXQ_OUT_F32
            if op == "linear" and s["bias"] is not None:
                s["bias1"] = s["bias"][0]
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import vq_compressed_linear_b200 as hxq
    op = s["case"]["op"]
    if op == "norm":
        hxq.rmsnorm(s["x"], s["weight"], _EPS, residual=s["res"], sum_out=s["sum"], y=s["y"], q=s["q"],
                    scales=s["scales"])
        return {"q": s["q"], "scales": s["scales"], "sum": s["sum"], "y": s["y"]}
    if op == "quantize":
        hxq.fp8_quantize(s["x"], q=s["q"], scales=s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "swiglu":
        hxq.fp8_swiglu(s["x"], q=s["q"], scales=s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "encode":
        hxq.fp8_encode(s["x"], q=s["q"], scales=s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "linear":
        return s["layer"].forward(s["xq"], s["xs"], bias=s.get("bias1"), out_dtype=s["out"], y=s["y"])
    return s["layer"].forward_grouped(s["xq"], s["xs"], s["offsets"], bias=s["bias"], out_dtype=s["out"], y=s["y"])


# ---- plain forms --------------------------------------------------------------

def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, and 1 for 0: amax = m 2^e with m in [1/2, 1), 448 = 7/8 2^9."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 120)
    s = ((e + 127) << 23).view(torch.float32)  # 2^e from its bits
    return torch.where(amax > 0, s, torch.ones_like(s))


def _quantize(h):
    """[M][K] to e4m3 [M][ld] and scales [M][KB]."""
    M, K = h.shape
    kb = -(-K // _BLOCK)
    hp = torch.nn.functional.pad(h, (0, kb * _BLOCK - K)).view(M, kb, _BLOCK)
    sc = _scale_of(hp.abs().amax(2))
    q = (hp / sc[:, :, None]).float().to(torch.float8_e4m3fn).view(M, kb * _BLOCK)
    return {"q": q[:, :_ld(K)].contiguous(), "scales": sc}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "quantize":
        return _quantize(s["x"].float())
    if op == "swiglu":
        # in 64 bits: an amax next to a border of its scale decides between two scales
        g, u = s["x"].double().chunk(2, dim=1)
        return _quantize(g / (1 + torch.exp(-g)) * u)
    if op == "norm":
        t = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["res"].dtype)
        d = t.double()  # as above
        h = d / torch.sqrt(d.square().mean(1, keepdim=True) + _EPS) * s["weight"].double()
        out = _quantize(h)
        out["sum"] = None if s["res"] is None else t
        out["y"] = h.to(torch.bfloat16) if s["y"] is not None else None
        return out
    if op == "encode":
        w = s["x"].float()
        N, K = w.shape
        nb, kb = -(-N // _BLOCK), -(-K // _BLOCK)
        wp = torch.nn.functional.pad(w, (0, kb * _BLOCK - K, 0, nb * _BLOCK - N)).view(nb, _BLOCK, kb, _BLOCK)
        sc = _scale_of(wp.abs().amax((1, 3)))
        q = (wp / sc[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * _BLOCK, kb * _BLOCK)
        return {"q": q[:N, :K].contiguous(), "scales": sc}
    # products: 8-bit values times their scales in fp32, then fp32 matrix products
    c = s["case"]
    N, K = c["N"], c["K"]
    x = s["xq"][:, :K].float() * s["xs"].repeat_interleave(_BLOCK, 1)[:, :K]
    w = s["wq"].float() * s["ws"].repeat_interleave(_BLOCK, 1)[:, :N].repeat_interleave(_BLOCK, 2)[:, :, :K]
    if op == "linear":
        y = x @ w[0].t()
        if s["bias"] is not None:
            y = y + s["bias"][0]
        return y.to(s["y"].dtype)
    # grouped: every expert's rows padded to the fullest expert's, one batched product
    off = s["offsets"].long()
    row = torch.arange(c["M"], device=_DEV)
    e = torch.searchsorted(off[1:], row, right=True)
    at = row - off[e]
    xp = torch.zeros(c["E"], max(1, s["most"]), K, device=_DEV)
    xp[e, at] = x
    y = torch.bmm(xp, w.transpose(1, 2))[e, at]
    if s["bias"] is not None:
        y = y + s["bias"][e]
    return y.to(s["y"].dtype)


# ---- from the definitions, in 64 bits -----------------------------------------

def _pow2_64(e):
    """2^e for whole e from -400 to 400, exactly (a power function need not be)."""
    table = torch.tensor([2.0 ** i for i in range(-400, 401)], device=_DEV, dtype=torch.float64)
    return table[e.long() + 400]


def _e4m3_64(v):
    """The nearest e4m3 value (ties to even) of |v| <= 448: steps of 2^(exponent - 3), exponents from -6."""
    mag = v.abs()
    _, e = torch.frexp(mag)
    step = _pow2_64((e - 1).clamp(min=-6) - 3)
    return torch.round(mag / step) * step * torch.sign(v)


def _blocks_64(h, rows):
    """e4m3 values and scales of a float64 matrix in blocks of rows x 128, without padding it."""
    M, K = h.shape
    rb = torch.arange(M, device=_DEV) // rows
    cb = torch.arange(K, device=_DEV) // _BLOCK
    kb, nb = -(-K // _BLOCK), -(-M // rows)
    a = torch.zeros(M, kb, device=_DEV, dtype=torch.float64)
    a.scatter_reduce_(1, cb.expand(M, K), h.abs(), "amax")
    if rows > 1:
        t = torch.zeros(nb, kb, device=_DEV, dtype=torch.float64)
        a = t.scatter_reduce_(0, rb[:, None].expand(M, kb), a, "amax")
    sc = _pow2_64(torch.ceil(torch.log2(torch.where(a > 0, a, 448.0) / 448.0)))
    sc = torch.where(a > 448.0 * sc, sc * 2, sc)             # log2 may round across a border: settle it exactly
    sc = torch.where(a <= 224.0 * sc, sc / 2, sc)
    sc = torch.where(a > 0, sc, torch.ones_like(sc))
    full = sc[rb] if rows > 1 else sc
    return _e4m3_64(h / full.gather(1, cb.expand(M, K))), sc


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "quantize", "swiglu"):
        x = s["x"].double()
        out = {}
        if op == "swiglu":
            K = case["cols"]
            h = x[:, K:] * x[:, :K] * torch.sigmoid(x[:, :K])
        elif op == "norm":
            if s["res"] is not None:
                x = (x + s["res"].double()).to(s["res"].dtype).double()
            h = x * torch.rsqrt(torch.mean(x * x, dim=1) + _EPS)[:, None] * s["weight"].double()
            out = {"sum": x if s["res"] is not None else None, "y": h if s["y"] is not None else None}
        else:
            h = x
        q, sc = _blocks_64(h, 1)
        pad = torch.zeros(case["rows"], _ld(case["cols"]) - case["cols"], device=_DEV, dtype=torch.float64)
        return {"q": torch.cat([q, pad], 1), "scales": sc, **out}
    if op == "encode":
        q, sc = _blocks_64(s["x"].double(), _BLOCK)
        return {"q": q, "scales": sc}
    M, N, K = case["M"], case["N"], case["K"]
    kb = torch.arange(K, device=_DEV) // _BLOCK
    nb = torch.arange(N, device=_DEV) // _BLOCK
    y = torch.zeros(M, N, device=_DEV, dtype=torch.float64)
    off = [0, M] if op == "linear" else s["offsets"].tolist()
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = s["xq"][a:b, :K].double() * s["xs"][a:b].double()[:, kb]
        w = s["wq"][e].double() * s["ws"][e].double()[nb][:, kb]
        y[a:b] = torch.einsum("mk,nk->mn", x, w)
        if s["bias"] is not None:
            y[a:b] += s["bias"][e].double()
    return y


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op in ("norm", "quantize", "swiglu", "encode"):
        M, K = case["rows"], case["cols"]
        kb = -(-K // _BLOCK)
        if op == "encode":
            return {"bytes": M * K * (size[case["x"]] + 1) + -(-M // _BLOCK) * kb * 4, "flops": 3 * M * K}
        b = M * K * (size[case["x"]] * (2 if op == "swiglu" else 1) + 1) + M * kb * 4
        if op == "norm":
            b += K * 4 + (2 * M * K * size[case["res"]] if case["res"] != "none" else 0)
            b += 2 * M * K if case["y"] else 0
        return {"bytes": b, "flops": (8 if op != "quantize" else 3) * M * K}
    M, N, K, E = case["M"], case["N"], case["K"], case.get("E", 1)
    kb = -(-K // _BLOCK)
    used = min(E, M)  # experts that can have a row at all
    b = M * K + M * kb * 4 + used * (N * K + -(-N // _BLOCK) * kb * 4) + M * N * size[case["out"]]
    return {"bytes": b + (used * N * 4 if case["bias"] else 0), "flops": 2 * M * N * K}
