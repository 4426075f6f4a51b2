"""Cases of the layer operators for training and serving in 4-bit floating point:
layer norm, its gradient, quantisation to microscaled 4-bit floats, the product of
two such matrices, and the gradients' global norm with clipping.

Each case is one call (or, of the quantisation, one call and its inverse) as a
program makes it, with the inputs that such a program has in hand.  With ``own``
false the operators are computed in their plain form (elementary torch operations in
32 bits, rounded once at the end); with ``own`` true through the library's entry
points.  ``exact`` computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
E2M1_MAX = 6.0
MIN_SCALE = 2.0 ** -126
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5
CLIP_EPS = 1e-6
SCALE_TYPE = {16: E4M3, 32: torch.float8_e8m0fnu}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # one token of a decode step: residual added, output quantised for an 8-bit product
        dict(name="layernorm 1 token e4m3", op="layernorm", M=1, N=4096, dtype="bf16", residual=True, quant=0),
        # a large training batch with the residual stream, 1 GiB of traffic
        dict(name="layernorm train bf16", op="layernorm", M=8192, N=16384, dtype="bf16", residual=True, quant=-1),
        # gradient of rows whose length and pitch are no multiple of 16 bytes, in fp32
        dict(name="layernorm grad ragged f32", op="layernorm_grad", M=2047, N=5001, dtype="f32", residual=False),
        # gradient of the large training batch, the residual's gradient added
        dict(name="layernorm grad bf16 large", op="layernorm_grad", M=16384, N=8192, dtype="bf16", residual=True),
        # a prompt's activations before a 4-bit product, an odd count of tokens
        dict(name="mx4 quantise prompt", op="mx4_quantise", M=2047, K=8192, dtype="bf16", block=16, scaled=True),
        # a large projection's fp32 weights laid out once for serving
        dict(name="mx4 quantise weight", op="mx4_quantise", M=16384, K=16384, dtype="f32", block=32, scaled=False),
        # one token through a small square projection: the latency case
        dict(name="mx4 1 token", op="mx4_matmul", M=1, N=4096, K=4096, out="bf16", block=16, scaled=True),
        # a few sequences' tokens, odd sizes, logits wanted in fp32
        dict(name="mx4 17 tokens ragged", op="mx4_matmul", M=17, N=8191, K=8160, out="f32", block=32, scaled=False),
        # a training batch through a large projection
        dict(name="mx4 train", op="mx4_matmul", M=8192, N=16384, K=8192, out="bf16", block=16, scaled=True),
        # the few small parameters of a head or an adapter: the norm and the factor for the optimiser
        dict(name="grad norm small f32", op="grad_norm", tensors=8, elements=50_000, matrix="f32", vector="f32", clip=False),
        # mixed precision: gradients of matrices in bf16, of vectors in fp32
        dict(name="grad norm mixed", op="grad_norm", tensors=96, elements=40_000_000, matrix="bf16", vector="f32", clip=False),
        # a large model's share, clipped in place for an optimiser that takes no factor
        dict(name="grad clip bf16 large", op="grad_norm", tensors=160, elements=300_000_000, matrix="bf16", vector="bf16", clip=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high, step):
    """A size over the logarithm of the range: a multiple of `step`, or (one in four) any."""
    n = _log(rng, low, high)
    return n if rng.random() < 0.25 else max(step, n // step * step)


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_grad", "mx4_quantise", "mx4_matmul", "mx4_matmul", "grad_norm"])
    if op in ("layernorm", "layernorm_grad"):
        N = _width(rng, 64, 32768, 8)
        M = max(1, min(_log(rng, 1, 16384), (1 << 27) // N))
        case = dict(op=op, M=M, N=N, dtype=rng.choice(["f16", "bf16", "bf16", "f32"]), residual=rng.random() < 0.6)
        if case["dtype"] == "f32":
            case["M"] = max(1, M // 2)
        if op == "layernorm":
            case["quant"] = rng.choice([-1, -1, 0, 64, 128])
        return case
    if op == "mx4_quantise":
        K = max(32, _log(rng, 64, 32768) // 32 * 32)
        M = max(1, min(_log(rng, 1, 16384), (1 << 27) // K))
        block = rng.choice([16, 32])
        return dict(op=op, M=M, K=K, dtype=rng.choice(["f16", "bf16", "bf16", "f32"]), block=block,
                    scaled=block == 16 and rng.random() < 0.7)
    if op == "mx4_matmul":
        K = max(32, _log(rng, 64, 16384) // 32 * 32)
        N = _width(rng, 16, 16384, 16)
        M = max(1, min(_log(rng, 1, 8192), (1 << 39) // (N * K)))
        block = rng.choice([16, 16, 32])
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["f32", "bf16", "bf16", "f16"]), block=block,
                    scaled=block == 16 and rng.random() < 0.7)
    matrix = rng.choice(["f32", "bf16", "bf16", "f16"])
    return dict(op=op, tensors=_log(rng, 1, 400), elements=_log(rng, 20_000, 100_000_000), matrix=matrix,
                vector=rng.choice([matrix, "f32"]), clip=rng.random() < 0.5)


def tensor_sizes(case):
    """Element counts of a model's matrices and of its short odd vectors."""
    count, total = case["tensors"], case["elements"]
    vectors = [min(1 + 37 * k % 5000, max(1, total // (2 * count))) for k in range(count // 2)]
    matrices = count - len(vectors)
    left = max(matrices, total - sum(vectors))
    return [left // matrices + (left % matrices if k == 0 else 0) for k in range(matrices)], vectors


def _matrix(M, N, dtype, g, scale=1.0):
    """Normal values of which a few are far larger, as activations and gradients have them."""
    v = torch.randn(M, N, generator=g, device="cuda").mul_(scale)
    return v.mul_(1 + 8 * (torch.rand(M, N, generator=g, device="cuda") < 0.002)).to(DTYPES[dtype])


def _packed(M, K, block, scaled, g):
    """Codes, tiled scales and tensor scale of a random matrix whose channels differ in size."""
    v = _matrix(M, K, "f32", g, 0.05).mul_(torch.rand(M, 1, generator=g, device="cuda") + 0.5)
    ts = v.abs().amax().div(E4M3_MAX * E2M1_MAX).view(1) if scaled else None
    codes, scales = _codes(v, block, ts)
    codes = codes.view(M, K)
    return codes[:, 0::2] | codes[:, 1::2] << 4, _tiled(scales), ts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("layernorm", "layernorm_grad"):
        M, N, dt = case["M"], case["N"], case["dtype"]
        s["w"] = (1 + 0.2 * torch.randn(N, generator=g, device="cuda")).to(DTYPES[dt])
        s["b"] = (0.1 * torch.randn(N, generator=g, device="cuda")).to(DTYPES[dt])
        s["x"] = _matrix(M, N, dt, g).add_(0.25)
        s["r"] = _matrix(M, N, dt, g, 0.02 if op == "layernorm_grad" else 2.0) if case["residual"] else None
        if op == "layernorm_grad":
            s["dy"] = _matrix(M, N, dt, g, 0.02)
            s["mean"] = torch.cat([x.float().mean(1) for x in s["x"].split(4096)])
            s["rstd"] = torch.cat([(x.float().var(1, correction=0) + EPS).rsqrt() for x in s["x"].split(4096)])
    elif op == "mx4_quantise":
        s["x"] = _matrix(case["M"], case["K"], case["dtype"], g, 0.5)
        s["ts"] = s["x"].abs().amax().float().div(E4M3_MAX * E2M1_MAX).view(1) if case["scaled"] else None
        s["out"] = torch.bfloat16 if case["dtype"] == "f32" else DTYPES[case["dtype"]]
    elif op == "mx4_matmul":
        s["a"] = _packed(case["M"], case["K"], case["block"], case["scaled"], g)
        s["b"] = _packed(case["N"], case["K"], case["block"], case["scaled"], g)
    else:
        # the tensors are parts of flat storages, each from a multiple of 64 elements on; what is between stays 0
        s["parts"] = []
        for key, sizes in zip(("matrix", "vector"), tensor_sizes(case)):
            starts = [0]
            for n in sizes:
                starts.append(starts[-1] + -(-n // 64) * 64)
            valid = torch.zeros(max(1, starts[-1]), device="cuda", dtype=torch.bool)
            for at, n in zip(starts, sizes):
                valid[at:at + n] = True
            s[key] = _matrix(1, valid.numel(), case[key], g, 1e-3).view(-1).mul_(valid)
            s["parts"] += [s[key][at:at + n] for at, n in zip(starts, sizes)]
        s["max_norm"] = 1.0
    return s


# The plain forms -------------------------------------------------------------------------------------------------

def _to_e4m3(t):
    return t.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)


def _quantised(y, quant):
    """(codes, scales) of the rows of y, a scale per row (quant 0) or per group of columns."""
    M, N = y.shape
    group = quant or N
    b = torch.nn.functional.pad(y, (0, -N % group)).view(M, -1, group) if N % group else y.view(M, -1, group)
    scales = (b.abs().amax(2) / E4M3_MAX).clamp_min(MIN_SCALE)
    return b / scales[:, :, None], scales


def _layernorm(s, c):
    h = s["x"].float()
    h = h + s["r"].float() if c["residual"] else h
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = (d.square().mean(1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["w"].float() + s["b"].float()
    out = {"mean": mean, "rstd": rstd}
    if c["residual"]:
        out["h"] = h.to(s["x"].dtype)
    if c["quant"] < 0:
        return out | {"y": y.to(s["x"].dtype)}
    q, scales = _quantised(y, c["quant"])
    return out | {"y": _to_e4m3(q).view(c["M"], -1)[:, :c["N"]], "scales": scales}


def _layernorm_grad(s, c):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dx = dx + s["r"].float() if c["residual"] else dx
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _tiled(scales):
    """M x G scale bytes in tiles of 128 rows and 4 blocks: row r of a tile has its 4 bytes at 16 (r % 32) + 4 (r / 32);
    a tile row's tiles follow each other; zeros fill the last ones."""
    M, G = scales.shape
    t = torch.nn.functional.pad(scales, (0, -G % 4, 0, -M % 128))
    return t.view(-1, 4, 32, (G + 3) // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, (G + 3) // 4, 512)


def _untiled(tiles, M, G):
    return tiles.view(*tiles.shape[:2], 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles.shape[0] * 128, -1)[:M, :G]


def _scale_values(codes, block):
    """What scale bytes stand for: e4m3 for blocks of 16, powers of two (their exponent's code) for blocks of 32."""
    if block == 16:
        return codes.view(E4M3).float()
    return torch.where(codes > 0, codes.int() << 23, 1 << 22).view(torch.float32)


def _rounded_to_e2m1(y):
    """4-bit codes nearest to y, halves to even, the sign in bit 3."""
    a = y.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
    code += (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte()
    return code + 8 * torch.signbit(y).byte()


def _codes(x, block, ts):
    """4-bit codes (blocks as rows) and scale bytes (M x K / block) of x."""
    M = x.shape[0]
    b = x.float().view(M, -1, block)
    amax = b.abs().amax(2)
    if block == 16:
        s = _to_e4m3(amax / (E2M1_MAX if ts is None else E2M1_MAX * ts))
        d = s.float() if ts is None else s.float() * ts
        codes = s.view(torch.uint8)
    else:
        e = (torch.frexp(amax).exponent - 3).clamp(min=-127)
        codes = torch.where(amax > 0, e + 127, 0).to(torch.uint8)
        d = _scale_values(codes, 32)
    y = torch.where(d[:, :, None] > 0, b / d[:, :, None], 0.0)
    return _rounded_to_e2m1(y), codes


def _values(codes, scales, ts):
    """What 4-bit codes (last dimension: a block) stand for."""
    v = torch.tensor(E2M1, device=codes.device)[(codes & 7).int()]
    v = torch.where(codes > 7, -v, v) * scales[:, :, None]
    return v if ts is None else v * ts


def _mx4_quantise(s, c):
    codes, scales = _codes(s["x"], c["block"], s["ts"])
    v = _values(codes, _scale_values(scales, c["block"]), s["ts"])
    return {"values": v.view(c["M"], c["K"]).to(s["out"]), "scales": _tiled(scales).view(SCALE_TYPE[c["block"]])}


def _mx4_wide(q, scales, ts, c, rows):
    codes = torch.stack((q & 15, q >> 4), 2).view(rows, -1, c["block"])
    G = c["K"] // c["block"]
    return _values(codes, _scale_values(_untiled(scales, rows, G).contiguous(), c["block"]), ts).view(rows, c["K"])


def _mx4_matmul(s, c):
    return (_mx4_wide(*s["a"], c, c["M"]) @ _mx4_wide(*s["b"], c, c["N"]).t()).to(DTYPES[c["out"]])


def _grad_norm(s, c):
    norm = (s["matrix"].double().square().sum() + s["vector"].double().square().sum()).sqrt().float()
    scale = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    out = {"norm": norm, "scale": scale}
    if c["clip"]:
        out |= {k: s[k].copy_(s[k].float() * scale) for k in ("matrix", "vector")}
    return out


PLAIN = {"layernorm": _layernorm, "layernorm_grad": _layernorm_grad, "mx4_quantise": _mx4_quantise,
         "mx4_matmul": _mx4_matmul, "grad_norm": _grad_norm}


# The library's ---------------------------------------------------------------------------------------------------

def _own(s, c):
    import mbarrier_async_tile_gb300 as mbt

    if c["op"] == "layernorm":
        got = mbt.tile_layernorm(s["x"], s["w"], s["b"], s["r"], eps=EPS, quant=None if c["quant"] < 0 else c["quant"])
        out = {"mean": got.mean, "rstd": got.rstd, "y": got.out}
        if c["residual"]:
            out["h"] = got.residual
        return out if c["quant"] < 0 else out | {"scales": got.scales}
    if c["op"] == "layernorm_grad":
        dx, dw, db = mbt.tile_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], dresidual=s["r"])
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "mx4_quantise":
        m = mbt.tile_mx4_quantize(s["x"], block=c["block"], tensor_scale=s["ts"])
        v = mbt.tile_mx4_dequantize(m, dtype=s["out"])
        return {"values": v, "scales": m.scales.view(SCALE_TYPE[c["block"]])}
    if c["op"] == "mx4_matmul":
        a, b = (mbt.Mx4(q, scales, ts, c["block"]) for q, scales, ts in (s["a"], s["b"]))
        return mbt.tile_mx4_matmul(a, b, out_dtype=DTYPES[c["out"]])
    call = mbt.tile_clip_grads if c["clip"] else mbt.tile_grad_norm
    got = call(s["parts"], max_norm=s["max_norm"], eps=CLIP_EPS)
    return {"norm": got.norm, "scale": got.scale} | ({"matrix": s["matrix"], "vector": s["vector"]} if c["clip"] else {})


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# The definitions in 64 bits --------------------------------------------------------------------------------------

def _exact_scales(x, block, ts):
    """Scale bytes of the blocks of x (fp64) and the divisors that they stand for."""
    amax = torch.stack([p.abs().max(1).values for p in x.split(block, 1)], 1)
    if block == 32:
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))).long().clamp(-125, 127) - 2
        return (e + 127).to(torch.uint8), 2.0 ** e.double()
    wide = (amax / 6 / (1.0 if ts is None else ts.double())).clamp(max=E4M3_MAX)
    step = 2.0 ** (torch.floor(torch.log2(wide.clamp(min=2.0 ** -6))) - 3)
    s = torch.round(wide / step) * step
    return s.float().to(E4M3).view(torch.uint8), s * (1.0 if ts is None else ts.double())


def _exact_bytes(tiles, rows, blocks):
    """Scale bytes by row and block, from the position of each in its tile."""
    r, k = torch.arange(rows, device="cuda")[:, None], torch.arange(blocks, device="cuda")[None, :]
    at = ((r // 128) * tiles.shape[1] + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
    return tiles.reshape(-1)[at]


def _exact_matrix(q, tiles, ts, block, K):
    b = _exact_bytes(tiles, q.shape[0], K // block)
    s = b.view(E4M3).double() if block == 16 else 2.0 ** (b.double() - 127)
    table = torch.tensor([*E2M1, *(-v for v in E2M1)], device="cuda", dtype=torch.float64)
    w = torch.empty(q.shape[0], K, device="cuda", dtype=torch.float64)
    w[:, 0::2] = table[(q % 16).int()]
    w[:, 1::2] = table[(q // 16).int()]
    w *= s.repeat_interleave(block, 1)
    return w if ts is None else w * ts.double()


def exact(case, seed):
    """Values of 8 bits are compared with those before they were rounded to them."""
    s, op = prepare(case, seed), case["op"]
    if op == "layernorm":
        parts = []
        for i in range(0, case["M"], 2048):
            h = s["x"][i:i + 2048].double()
            if case["residual"]:
                h += s["r"][i:i + 2048].double()
            mean = torch.einsum("ij->i", h) / case["N"]
            d = h - mean[:, None]
            rstd = 1 / torch.sqrt(torch.einsum("ij,ij->i", d, d) / case["N"] + EPS)
            y = torch.einsum("ij,i,j->ij", d, rstd, s["w"].double()) + s["b"].double()
            got = {"mean": mean, "rstd": rstd, "y": y} | ({"h": h} if case["residual"] else {})
            if case["quant"] >= 0:
                cut = y.split(case["quant"] or case["N"], 1)
                sc = torch.stack([p.abs().max(1).values for p in cut], 1).div(E4M3_MAX).clamp(min=MIN_SCALE)
                got["scales"] = sc
                got["y"] = torch.cat([p / sc[:, k:k + 1] for k, p in enumerate(cut)], 1)
            parts.append(got)
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if op == "layernorm_grad":
        N, w = case["N"], s["w"].double()
        dw, db, dx = torch.zeros(2, N, device="cuda", dtype=torch.float64).unbind() + ([],)
        for i in range(0, case["M"], 2048):
            at = slice(i, i + 2048)
            dy, r = s["dy"][at].double(), s["rstd"][at].double()
            xh = torch.einsum("ij,i->ij", s["x"][at].double() - s["mean"][at].double()[:, None], r)
            dw += torch.einsum("ij,ij->j", dy, xh)
            db += torch.einsum("ij->j", dy)
            along, level = torch.einsum("ij,j,ij->i", dy, w, xh) / N, torch.einsum("ij,j->i", dy, w) / N
            d = torch.einsum("ij,j,i->ij", dy, w, r) - torch.einsum("ij,i,i->ij", xh, along, r) - (level * r)[:, None]
            dx.append(d + s["r"][at].double() if case["residual"] else d)
        return {"dx": torch.cat(dx), "dw": dw, "db": db}
    if op == "mx4_quantise":
        block, values, scales = case["block"], [], []
        for i in range(0, case["M"], 2048):
            x = s["x"][i:i + 2048].double()
            codes, d = _exact_scales(x, block, s["ts"])
            scales.append(codes)
            d = d.repeat_interleave(block, 1)
            y = torch.where(d > 0, x / d, 0.0)
            a = y.abs().clamp(max=6.0)
            step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
            values.append(torch.sign(y) * torch.round(a / step) * step * d)
        b = torch.cat(scales)
        tiles = torch.zeros(-(-b.shape[0] // 128), -(-b.shape[1] // 4), 512, device="cuda", dtype=torch.uint8)
        index = torch.arange(tiles.numel(), device="cuda").view(tiles.shape)
        tiles.view(-1)[_exact_bytes(index, *b.shape)] = b
        return {"values": torch.cat(values), "scales": tiles.view(E4M3).double() if block == 16 else 2.0 ** (tiles.double() - 127)}
    if op == "mx4_matmul":
        a = _exact_matrix(*s["a"], case["block"], case["K"])
        (q, tiles, ts), parts = s["b"], []
        for i in range(0, case["N"], 2048):
            parts.append(a @ _exact_matrix(q[i:i + 2048], tiles[i // 128:], ts, case["block"], case["K"]).T)
        return torch.cat(parts, 1)
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for key in ("matrix", "vector"):
        for part in s[key].split(1 << 24):
            total += torch.dot(part.double(), part.double())
    norm = total ** 0.5
    scale = min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))
    out = {"norm": norm, "scale": torch.tensor(scale, device="cuda", dtype=torch.float64)}
    return out | ({k: s[k].double() * scale for k in ("matrix", "vector")} if case["clip"] else {})


def work(case):
    op = case["op"]
    if op in ("layernorm", "layernorm_grad"):
        M, N, e = case["M"], case["N"], SIZE[case["dtype"]]
        if op == "layernorm_grad":
            return {"bytes": M * N * e * (4 if case["residual"] else 3) + N * (e + 8) + 8 * M, "flops": 14 * M * N}
        out = M * N * (e if case["quant"] < 0 else 1) + 8 * M
        out += 0 if case["quant"] < 0 else 4 * M * (-(-N // case["quant"]) if case["quant"] else 1)
        return {"bytes": M * N * e * (3 if case["residual"] else 1) + 2 * N * e + out, "flops": 8 * M * N}
    if op == "mx4_quantise":
        # x in, codes and scales out and in again, values out
        M, K, e = case["M"], case["K"], SIZE[case["dtype"]]
        held = M * K // 2 + M * (K // case["block"])
        return {"bytes": M * K * (e + 2) + 2 * held, "flops": 6 * M * K}
    if op == "mx4_matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K // 2 + K // case["block"]) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    matrices, vectors = tensor_sizes(case)
    n = sum(matrices) * SIZE[case["matrix"]] + sum(vectors) * SIZE[case["vector"]]
    return {"bytes": n * (2 if case["clip"] else 1), "flops": (3 if case["clip"] else 2) * (sum(matrices) + sum(vectors))}
