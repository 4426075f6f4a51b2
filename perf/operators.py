"""Cases of the layer operators: root-mean-square norm, its gradient, the 4-bit
matrix-vector product and the AdamW step.

Each case is one call as a program makes it, with the inputs that such a program
has in hand.  With ``own`` false the operators are computed in their plain form
(elementary torch operations in 32 bits, rounded once at the end); with ``own``
true through the library's entry points.  ``exact`` computes the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126
BLOCK = 256  # elements of an 8-bit optimiser state that share a scale
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.1, 100


def listed():
    return [
        # one token of a decode step: residual added, output quantised for an 8-bit product
        dict(name="norm 1 token e4m3", op="norm", M=1, N=8192, dtype="bf16", residual=True, quant=0),
        # a prompt's tokens, an odd count, quantised by groups of 128 columns
        dict(name="norm prompt e4m3 groups", op="norm", M=2047, N=8192, dtype="bf16", residual=True, quant=128),
        # a training batch with the residual stream, 2 GiB of traffic
        dict(name="norm train f16", op="norm", M=16384, N=16384, dtype="f16", residual=True, quant=-1),
        # rows whose length and pitch are no multiple of 16 bytes, in fp32
        dict(name="norm ragged f32", op="norm", M=4097, N=8191, dtype="f32", residual=False, quant=-1),
        # gradient of an ordinary training batch, the residual's gradient added
        dict(name="norm grad bf16", op="norm_grad", M=4096, N=4096, dtype="bf16", residual=True),
        # gradient of the large training batch
        dict(name="norm grad f16 large", op="norm_grad", M=16384, N=16384, dtype="f16", residual=True),
        # one token through a small square projection: the latency case
        dict(name="w4 1 token", op="w4", T=1, N=4096, K=4096, dtype="bf16", out="bf16", group=128, zeros=False, xgroup=-1),
        # three tokens whose 8-bit values and scales come from the norm, odd row count, small groups
        dict(name="w4 3 tokens e4m3", op="w4", T=3, N=8191, K=8192, dtype="e4m3", out="bf16", group=32, zeros=False, xgroup=128),
        # a batch of eight sequences through a large projection, zero points
        dict(name="w4 8 tokens large", op="w4", T=8, N=16384, K=16384, dtype="f16", out="f16", group=64, zeros=True, xgroup=-1),
        # the few small parameters of a head or an adapter
        dict(name="adamw small f32", op="adamw", tensors=8, elements=50_000, param="f32", grad="f32", master=False, state="f32"),
        # mixed precision: bf16 parameters and gradients, fp32 master weights, many tensors
        dict(name="adamw bf16 master", op="adamw", tensors=96, elements=40_000_000, param="bf16", grad="bf16", master=True, state="f32"),
        # a large model's share with both states in 8 bits
        dict(name="adamw 8-bit large", op="adamw", tensors=160, elements=300_000_000, param="bf16", grad="bf16", master=False, state="e4m3"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high, step):
    """A size over the logarithm of the range: a multiple of `step`, or (one in four) any."""
    n = _log(rng, low, high)
    n = n if rng.random() < 0.25 else max(step, n // step * step)
    return n + step if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "w4", "adamw"])
    if op in ("norm", "norm_grad"):
        N = _width(rng, 64, 32768, 8)
        M = max(1, min(_log(rng, 1, 16384), (1 << 28) // (2 * N)))
        M += M == 3 * 1024
        case = dict(op=op, M=M, N=N, dtype=rng.choice(["f16", "bf16", "bf16", "f32"]), residual=rng.random() < 0.6)
        if op == "norm":
            case["quant"] = rng.choice([-1, -1, 0, 64, 128])
        return case
    if op == "w4":
        group = rng.choice([32, 64, 128, 128])
        K = max(group, _log(rng, 512, 16384) // group * group)
        K += group if K == 3 * 1024 else 0
        N = _width(rng, 256, 16384, 16)
        dtype = rng.choice(["bf16", "f16", "e4m3"])
        return dict(op=op, T=rng.choice([1, 1, 2, 4, 7, 8]), N=N, K=K, dtype=dtype,
                    out=rng.choice(["f32", "bf16" if dtype == "e4m3" else dtype]), group=group,
                    zeros=rng.random() < 0.5, xgroup=rng.choice([0, 128]) if dtype == "e4m3" else -1)
    param = rng.choice(["f32", "bf16", "f16"])
    return dict(op=op, tensors=_log(rng, 1, 400), elements=_log(rng, 20_000, 100_000_000), param=param,
                grad=rng.choice([param, "f32"]), master=param != "f32" and rng.random() < 0.5,
                state=rng.choice(["f32", "e4m3"]))


def tensor_sizes(case):
    """Element counts of an optimiser's tensors: matrices, and between them short odd vectors."""
    count, total = case["tensors"], case["elements"]
    vectors = [min(1 + 37 * k % 5000, max(1, total // (2 * count))) for k in range(count // 2)]
    matrices = count - len(vectors)
    left = max(matrices, total - sum(vectors))
    first = [left // matrices + (left % matrices if k == 0 else 0) for k in range(matrices)]
    return [n for pair in zip(first, vectors + [0] * (matrices - len(vectors))) for n in pair if n]


def _matrix(M, N, dtype, g, scale=1.0):
    """Normal values of which a few are far larger, as activations and gradients have them."""
    v = torch.randn(M, N, generator=g, device="cuda").mul_(scale)
    return v.mul_(1 + 8 * (torch.rand(M, N, generator=g, device="cuda") < 0.002)).to(DTYPES[dtype])


def _to_e4m3(t):
    return t.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)


def _blocks_to_e4m3(v):
    """Blocks of the flat `v` in 8 bits: codes and scales."""
    b = v.view(-1, BLOCK)
    s = (b.abs().amax(1) / E4M3_MAX).clamp_min(MIN_SCALE)
    return _to_e4m3(b / s[:, None]).view(-1), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_grad"):
        M, N, dt = case["M"], case["N"], case["dtype"]
        s["w"] = (1 + 0.2 * torch.randn(N, generator=g, device="cuda")).to(DTYPES[dt])
        s["x"] = _matrix(M, N, dt, g)
        s["r"] = _matrix(M, N, dt, g, 0.02 if op == "norm_grad" else 2.0) if case["residual"] else None
        if op == "norm_grad":
            s["dy"] = _matrix(M, N, dt, g, 0.02)
            s["rstd"] = torch.cat([(x.float().square().mean(1) + EPS).rsqrt() for x in s["x"].split(4096)])
    elif op == "w4":
        T, N, K, G = case["T"], case["N"], case["K"], case["K"] // case["group"]
        x = _matrix(T, K, "f32", g)
        s["xs"] = None
        if case["dtype"] == "e4m3":
            size = case["xgroup"] or K
            s["xs"] = torch.nn.functional.pad(x, (0, -K % size)).view(T, -1, size).abs().amax(2) / E4M3_MAX
            x = x / s["xs"].repeat_interleave(size, 1)[:, :K]
            s["x"] = _to_e4m3(x)
        else:
            s["x"] = x.to(DTYPES[case["dtype"]])
        s["q"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        wide = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
        s["s"] = (0.004 * (0.25 + torch.rand(N, G, generator=g, device="cuda"))).to(wide)
        s["z"] = torch.randint(4, 12, (N, G), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    else:
        sizes = tensor_sizes(case)
        starts, blocks = [], 0
        for n in sizes:
            starts.append(blocks * BLOCK)
            blocks += -(-n // BLOCK)
        # the tensors are parts of flat storages, each from a multiple of BLOCK elements on; what is between stays 0
        valid = torch.zeros(blocks * BLOCK, device="cuda", dtype=torch.bool)
        base = torch.empty(blocks, device="cuda", dtype=torch.int64)  # of the rounding's counters, per block
        for j, (at, n) in enumerate(zip(starts, sizes)):
            valid[at:at + n] = True
            b0, b1 = at // BLOCK, at // BLOCK - (-n // BLOCK)
            base[b0:b1] = torch.arange(b1 - b0, device="cuda") * (BLOCK // 2) + j * 0x9E3779B9

        def flat(scale):
            return _matrix(blocks, BLOCK, "f32", g, scale).view(-1).mul_(valid)

        w = flat(0.02)
        m, v = flat(2e-4), flat(1e-3).square_()
        s["p"] = w.to(DTYPES[case["param"]])
        s["w"] = w if case["master"] else None
        s["g"] = flat(1e-3).to(DTYPES[case["grad"]])
        s["m"], s["ms"] = (m, None) if case["state"] == "f32" else _blocks_to_e4m3(m)
        s["v"], s["vs"] = (v, None) if case["state"] == "f32" else _blocks_to_e4m3(v.sqrt_())
        s["base"], s["seed"] = base, seed & 0x7FFFFFFF

        def parts(f, unit=1):
            return None if f is None else [f[at // unit:at // unit + -(-n // unit)] for at, n in zip(starts, sizes)]

        s["parts"] = {k: parts(s[k]) for k in "pwgmv"} | {k: parts(s[k], BLOCK) for k in ("ms", "vs")}
        s["table"] = None
    return s


# The plain forms -------------------------------------------------------------------------------------------------

def _quantised(y, quant):
    """(codes, scales) of the rows of y, a scale per row (quant 0) or per group of columns."""
    M, N = y.shape
    group = quant or N
    b = torch.nn.functional.pad(y, (0, -N % group)).view(M, -1, group) if N % group else y.view(M, -1, group)
    scales = (b.abs().amax(2) / E4M3_MAX).clamp_min(MIN_SCALE)
    return b / scales[:, :, None], scales


def _norm(s, c):
    h = s["x"].float()
    h = h + s["r"].float() if c["residual"] else h
    rstd = (h.square().mean(1) + EPS).rsqrt()
    y = h * rstd[:, None] * s["w"].float()
    out = {"rstd": rstd}
    if c["residual"]:
        out["h"] = h.to(s["x"].dtype)
    if c["quant"] < 0:
        return out | {"y": y.to(s["x"].dtype)}
    q, scales = _quantised(y, c["quant"])
    return out | {"y": _to_e4m3(q).view(c["M"], -1)[:, :c["N"]], "scales": scales}


def _norm_grad(s, c):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = s["x"].float() * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    dx = dx + s["r"].float() if c["residual"] else dx
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0)}


def _w4_weights(s, c, wide):
    q = torch.stack((s["q"] & 15, s["q"] >> 4), 2).view(c["N"], -1, c["group"])
    z = 8 if s["z"] is None else s["z"][:, :, None].to(wide)
    return ((q.to(wide) - z) * s["s"][:, :, None].to(wide)).view(c["N"], c["K"])


def _w4_inputs(s, c, wide):
    x = s["x"].to(wide)
    if s["xs"] is None:
        return x
    xs = s["xs"].to(wide)
    return x * (xs.repeat_interleave(c["xgroup"], 1)[:, :c["K"]] if c["xgroup"] else xs)


def _w4(s, c):
    return (_w4_inputs(s, c, torch.float32) @ _w4_weights(s, c, torch.float32).t()).to(DTYPES[c["out"]])


def _hash16(base, seed):
    """16 random bits for each element of blocks whose counters begin at `base`: the 32-bit finaliser of MurmurHash3 of
    (counter xor seed), one counter for two elements."""
    full = 0xFFFFFFFF
    h = ((base[:, None] + torch.arange(BLOCK // 2, device=base.device)) & full) ^ seed
    h = (h ^ (h >> 16)) * 0x85EBCA6B & full
    h = (h ^ (h >> 13)) * 0xC2B2AE35 & full
    h = h ^ (h >> 16)
    return torch.stack((h & 0xFFFF, h >> 16), 2).view(-1, BLOCK)


def _rounded_at_random(t, r):
    """t >= 0 rounded to e4m3 values up or down by the 16 bits r, never to 0 where t > 0."""
    low = torch.where(t < 2.0 ** -6, 2.0 ** -6, 0.0)
    bits = (t + low).view(torch.int32).long() + (r << 4 | 8)
    y = (bits & ~0xFFFFF).int().view(torch.float32) - low
    return torch.where(t > 0, y.clamp_min(2.0 ** -9), y).clamp_max(E4M3_MAX)


def _adamw(s, c):
    g = s["g"].float()
    p = (s["w"] if c["master"] else s["p"]).float()
    m, v = s["m"].float(), s["v"].float()
    if c["state"] == "e4m3":
        m = (m.view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["vs"][:, None]).view(-1).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    u = v.sqrt()
    p = p * (1 - LR * DECAY) - LR / (1 - BETA1 ** STEP) * (m / (u / math.sqrt(1 - BETA2 ** STEP) + ADAM_EPS))
    s["p"].copy_(p)
    out = {"p": s["p"]}
    if c["master"]:
        out["w"] = s["w"].copy_(p)
    if c["state"] == "f32":
        return out | {"m": s["m"].copy_(m), "v": s["v"].copy_(v)}
    m, u = m.view(-1, BLOCK), u.view(-1, BLOCK)
    ms = (m.abs().amax(1) / E4M3_MAX).clamp_min(MIN_SCALE)
    vs = (u.amax(1) / E4M3_MAX).clamp_min(MIN_SCALE)
    codes = _rounded_at_random(u / vs[:, None], _hash16(s["base"], s["seed"]))
    s["m"].copy_(_to_e4m3(m / ms[:, None]).view(-1))
    s["v"].copy_(codes.to(E4M3).view(-1))
    return out | {"m": s["m"], "v": s["v"], "ms": s["ms"].copy_(ms), "vs": s["vs"].copy_(vs)}


PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "w4": _w4, "adamw": _adamw}


# The library's ---------------------------------------------------------------------------------------------------

def _own(s, c):
    import mbarrier_async_tile_gb300 as mbt

    if c["op"] == "norm":
        got = mbt.tile_rmsnorm(s["x"], s["w"], s["r"], eps=EPS, quant=None if c["quant"] < 0 else c["quant"])
        out = {"rstd": got.rstd, "y": got.out}
        if c["residual"]:
            out["h"] = got.residual
        return out if c["quant"] < 0 else out | {"scales": got.scales}
    if c["op"] == "norm_grad":
        dx, dw = mbt.tile_rmsnorm_backward(s["dy"], s["x"], s["rstd"], s["w"], dresidual=s["r"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "w4":
        return mbt.tile_w4_matvec(s["x"], s["q"], s["s"], s["z"], group=c["group"], x_scales=s["xs"],
                                  out_dtype=DTYPES[c["out"]])
    if s["table"] is None:  # an optimiser keeps its tensors' table
        t = s["parts"]
        s["table"] = mbt.AdamwTensors(t["p"], t["m"], t["v"], master=t["w"], m_scales=t["ms"], v_scales=t["vs"])
    mbt.tile_adamw(s["table"], s["parts"]["g"], step=STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS,
                   weight_decay=DECAY, seed=s["seed"])
    names = ["p"] + ["w"] * c["master"] + ["m", "v"] + ["ms", "vs"] * (c["state"] == "e4m3")
    return {k: s[k] for k in names}


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# The definitions in 64 bits --------------------------------------------------------------------------------------

def exact(case, seed):
    """Codes of 8 bits are compared with the value before it was rounded to them."""
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        parts = []
        for i in range(0, case["M"], 2048):
            h = s["x"][i:i + 2048].double()
            if case["residual"]:
                h += s["r"][i:i + 2048].double()
            rstd = 1 / torch.sqrt(torch.einsum("ij,ij->i", h, h) / case["N"] + EPS)
            y = torch.einsum("ij,i,j->ij", h, rstd, s["w"].double())
            got = {"rstd": rstd, "y": y} | ({"h": h} if case["residual"] else {})
            if case["quant"] >= 0:
                size = case["quant"] or case["N"]
                cut = y.split(size, 1)
                sc = torch.stack([p.abs().max(1).values for p in cut], 1).div(E4M3_MAX).clamp(min=MIN_SCALE)
                got["scales"] = sc
                got["y"] = torch.cat([p / sc[:, k:k + 1] for k, p in enumerate(cut)], 1)
            parts.append(got)
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if op == "norm_grad":
        w, dw, dx = s["w"].double(), torch.zeros(case["N"], device="cuda", dtype=torch.float64), []
        for i in range(0, case["M"], 2048):
            at = slice(i, i + 2048)
            dy, r = s["dy"][at].double(), s["rstd"][at].double()
            xh = torch.einsum("ij,i->ij", s["x"][at].double(), r)
            dw += torch.einsum("ij,ij->j", dy, xh)
            coef = torch.einsum("ij,j,ij->i", dy, w, xh) / case["N"]
            d = torch.einsum("ij,j,i->ij", dy, w, r) - torch.einsum("ij,i,i->ij", xh, coef, r)
            dx.append(d + s["r"][at].double() if case["residual"] else d)
        return {"dx": torch.cat(dx), "dw": dw}
    if op == "w4":
        T, N, K = case["T"], case["N"], case["K"]
        x = s["x"].double()
        if s["xs"] is not None:
            column = torch.arange(K, device="cuda") // (case["xgroup"] or K)
            x = x * s["xs"].double()[:, column]
        group, y = torch.arange(K, device="cuda") // case["group"], torch.empty(T, N, device="cuda", dtype=torch.float64)
        for i in range(0, N, 2048):
            at = slice(i, i + 2048)
            w = torch.empty(s["q"][at].shape[0], K, device="cuda", dtype=torch.float64)
            w[:, 0::2] = s["q"][at] % 16
            w[:, 1::2] = s["q"][at] // 16
            w -= 8 if s["z"] is None else s["z"][at][:, group]
            w *= s["s"][at].double()[:, group]
            y[:, at] = x @ w.T
        return y
    keys = ["p"] + ["w"] * case["master"] + ["m", "v"] + ["ms", "vs"] * (case["state"] == "e4m3")
    n, parts = s["p"].numel(), []
    for i in range(0, n, 1 << 24):
        at, bl = slice(i, i + (1 << 24)), slice(i // BLOCK, (i + (1 << 24)) // BLOCK)
        g, p = s["g"][at].double(), (s["w"] if case["master"] else s["p"])[at].double()
        m, v = s["m"][at].double(), s["v"][at].double()
        if case["state"] == "e4m3":
            m = m * s["ms"][bl].double().repeat_interleave(BLOCK)
            v = (v * s["vs"][bl].double().repeat_interleave(BLOCK)) ** 2
        m += (g - m) * (1 - BETA1)
        v += (g * g - v) * (1 - BETA2)
        mh, vh = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        p = p - LR * DECAY * p - LR * mh / (vh ** 0.5 + ADAM_EPS)
        got = {"p": p, "w": p, "m": m, "v": v}
        if case["state"] == "e4m3":
            for k, x in (("m", m), ("v", v ** 0.5)):
                sc = torch.max(x.view(-1, BLOCK).abs(), 1).values.div(E4M3_MAX).clamp(min=MIN_SCALE)
                got[k], got[k + "s"] = x / sc.repeat_interleave(BLOCK), sc
        parts.append({k: got[k] for k in keys})
    return {k: torch.cat([p[k] for p in parts]) for k in keys}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        M, N, e = case["M"], case["N"], SIZE[case["dtype"]]
        if op == "norm_grad":
            return {"bytes": M * N * e * (4 if case["residual"] else 3) + N * (e + 4) + 4 * M, "flops": 10 * M * N}
        out = M * N * (e if case["quant"] < 0 else 1) + 4 * M
        out += 0 if case["quant"] < 0 else 4 * M * (-(-N // case["quant"]) if case["quant"] else 1)
        return {"bytes": M * N * e * (3 if case["residual"] else 1) + N * e + out, "flops": 6 * M * N}
    if op == "w4":
        T, N, K = case["T"], case["N"], case["K"]
        groups = N * (K // case["group"])
        xs = 0 if case["xgroup"] < 0 else 4 * T * (-(-K // case["xgroup"]) if case["xgroup"] else 1)
        return {"bytes": N * K // 2 + groups * (3 if case["zeros"] else 2) + T * K * SIZE[case["dtype"]] + xs
                + T * N * SIZE[case["out"]], "flops": 2 * T * N * K}
    n = sum(tensor_sizes(case))
    p, g = SIZE[case["param"]], SIZE[case["grad"]]
    each = g + (p + 8 if case["master"] else 2 * p) + (16 if case["state"] == "f32" else 4 + 16 / BLOCK)
    return {"bytes": n * each, "flops": 16 * n}
