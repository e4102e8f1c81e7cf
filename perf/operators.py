"""Cases of the 8-bit operators around the sequence-parallel region.

Four kinds of pass:

``norm``      the region's forward (sum of T partials, dropout, residual add, norm) with the norm's output in
              8 bits and one scale per token and 128 columns; T = 1 and p = 0 is the plain residual add + norm.
``quant``     a tensor to 8 bits with a scale per 128 values of a row (or per 128 x 128 block), the same for its
              transpose, in one pass.
``matmul``    C[M,N] = A[M,K] B[N,K]^T of 8-bit tensors with a scale per 128 values along K.
``backward``  the gradients of such a product from dY: both 8-bit forms of dY, the transposed form of the saved
              input, dX = dY W and dW += dY^T X.

A scale is a power of two: the smallest 2^s that brings the group's largest magnitude to at most 448 (e4m3) or
57344 (e5m2); a group of zeros has scale 1.  8-bit values and scales are returned in torch's 8-bit types, whose
values they are.
"""
import torch

own = False

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
FMT = {"e4m3": E4M3, "e5m2": E5M2}
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 128


def listed():
    return [
        # one decoded token, no tensor parallelism: residual add + RMSNorm before an 8-bit product
        dict(name="norm_one_token", op="norm", T=1, S=1, B=1, H=8192, dtype="bf16", norm="rms", p=0.0),
        # the framework's training step: TP = 2, sequence 2048, micro-batch 2, dropout 0.1
        dict(name="norm_pages", op="norm", T=2, S=2048, B=2, H=768, dtype="bf16", norm="rms", p=0.1),
        # GPT-style LayerNorm region, TP = 8
        dict(name="norm_gpt_ln", op="norm", T=8, S=4096, B=1, H=4096, dtype="bf16", norm="ln", p=0.1),
        # output gradient of the framework's step (H = 768): both 8-bit forms, in the wide-range type
        dict(name="quant_dy_pages", op="quant", M=4096, K=768, src="bf16", fmt="e5m2", block=False, row=True, col=True),
        # a weight after its optimiser step, fp32 master values: 128 x 128 blocks, W and its transpose
        dict(name="quant_weight", op="quant", M=4096, K=8192, src="f32", fmt="e4m3", block=True, row=True, col=True),
        # a saved 8-bit activation transposed for the weight gradient, a ragged number of tokens
        dict(name="quant_saved_ragged", op="quant", M=16131, K=4096, src="e4m3", fmt="e4m3", block=False, row=False, col=True),
        # one decoded token through a square projection
        dict(name="mm_one_token", op="matmul", M=1, N=8192, K=8192, a="e4m3", b="e4m3", block=True, out="bf16"),
        # a small ragged decode batch through a row-parallel slice
        dict(name="mm_decode_batch", op="matmul", M=33, N=4096, K=2048, a="e4m3", b="e4m3", block=True, out="f32"),
        # the training step's column-parallel product (H = 768, a half of the widened layer)
        dict(name="mm_pages", op="matmul", M=4096, N=1536, K=768, a="e4m3", b="e4m3", block=True, out="bf16"),
        # a long prefill of the large hidden size through a column-parallel slice
        dict(name="mm_large", op="matmul", M=16384, N=4096, K=8192, a="e4m3", b="e4m3", block=True, out="bf16"),
        # training at the pages' size: gradients of the column-parallel product
        dict(name="backward_pages", op="backward", M=4096, N=1536, K=768, fmt="e5m2"),
        # GPT size, an odd number of tokens
        dict(name="backward_gpt", op="backward", M=8177, N=2048, K=4096, fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "quant", "matmul", "backward"])
    if op == "norm":
        T = rng.choice([1, 2, 4, 8])
        H = 8 * _log(rng, 8, 1024)
        B = rng.randint(1, 4)
        S = T * _log(rng, 1, max(1, min(4096, (1 << 27) // (T * H * B * T))))
        return dict(op=op, T=T, S=S, B=B, H=H, dtype="bf16", norm=rng.choice(["rms", "ln"]), p=rng.choice([0.0, 0.1, 0.5]))
    if op == "quant":
        K = _log(rng, 16, 8192)
        M = _log(rng, 1, min(16384, (1 << 25) // K))
        src = rng.choice(["bf16", "f32", "e4m3"])
        row = src != "e4m3" and rng.random() < 0.7
        return dict(op=op, M=M, K=K, src=src, fmt="e4m3" if src == "e4m3" else rng.choice(["e4m3", "e5m2"]),
                    block=src != "e4m3" and rng.random() < 0.3, row=row, col=not row or rng.random() < 0.7)
    if op == "matmul":
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 8192), _log(rng, 64, 8192)
        return dict(op=op, M=M, N=N, K=K, a=rng.choice(["e4m3", "e4m3", "e5m2"]), b="e4m3", block=rng.random() < 0.6,
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, M=_log(rng, 64, 8192), N=_log(rng, 64, 4096), K=_log(rng, 64, 4096), fmt=rng.choice(["e4m3", "e5m2"]))


def work(c):
    if c["op"] == "norm":
        rows, n = c["S"] * c["B"], c["S"] * c["B"] * c["H"]
        e = 2 if c["dtype"] == "bf16" else 4
        per = (c["T"] + 2) * e + 1 + (1 if c["p"] > 0 else 0)
        return {"bytes": n * per + rows * (-(-c["H"] // GROUP) + 4 * (1 + (c["norm"] == "ln"))) + c["H"] * e * (1 + (c["norm"] == "ln")),
                "flops": n * (c["T"] + 8)}
    if c["op"] == "quant":
        n, e = c["M"] * c["K"], {"bf16": 2, "f32": 4}.get(c["src"], 1)
        m = 1 if not c["block"] else GROUP
        scales = (c["row"] * -(-c["M"] // m) * -(-c["K"] // GROUP) + c["col"] * -(-c["K"] // m) * -(-c["M"] // GROUP)
                  + (e == 1) * c["M"] * -(-c["K"] // GROUP))
        return {"bytes": n * (e + c["row"] + c["col"]) + scales, "flops": n * 4}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "matmul":
        groups = -(-K // GROUP)
        return {"bytes": M * K + N * K + M * N * (2 if c["out"] == "bf16" else 4)
                + groups * (M + (-(-N // GROUP) if c["block"] else N)), "flops": 2 * M * N * K}
    # dY bf16 in; X and W^T in 8 bits in; dX bf16 and dW fp32 out
    return {"bytes": 2 * M * N + M * K + N * K + 2 * M * K + 4 * N * K + M * -(-K // GROUP), "flops": 4 * M * N * K}


# ---- inputs ------------------------------------------------------------------------------------------------------


def _power(byte):
    """2^(byte - 127) in fp32, for bytes 1..254 (byte 0, a subnormal power, as well)."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _room(rows, cols, device):
    """A byte matrix whose rows start 16 bytes apart or a multiple of it."""
    return torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.uint8, device=device)[:, :cols]


def _grouped(x):
    """[R, C] with C filled up with zeros to [R, groups, 128]."""
    R, C = x.shape
    G = -(-C // GROUP)
    if G * GROUP != C:
        wide = torch.zeros((R, G * GROUP), dtype=x.dtype, device=x.device)
        wide[:, :C] = x
        x = wide
    return x.reshape(R, G, GROUP)


def _to8(x, fmt, block):
    """The 8-bit values [R, C] and scale bytes of fp32 x, grouped along its rows."""
    R, C = x.shape
    g = _grouped(x)
    amax = g.abs().amax(2)
    if block:
        amax = _grouped(amax.t().contiguous()).amax(2).t()  # over 128 rows
    m, e = torch.frexp(amax)
    s = e - (9 if fmt == "e4m3" else 16) + (m > 0.875).to(e.dtype)
    s = torch.where(amax > 0, s.clamp(-127, 127), torch.zeros_like(s))
    back = ((127 - s) << 23).to(torch.int32).view(torch.float32)  # 2^-s
    if block:
        back = back.repeat_interleave(GROUP, 0)[:R]
    q, scale = _room(R, C, x.device), _room(s.shape[0], s.shape[1], x.device)
    q.copy_((g * back[:, :, None]).reshape(R, -1)[:, :C].to(FMT[fmt]).view(torch.uint8))
    scale.copy_((s + 127).to(torch.uint8))
    return q.view(FMT[fmt]), scale


def _from8(q, scale):
    """The fp32 values that 8-bit values and their scale bytes stand for."""
    R, C = q.shape
    s = _power(scale)
    if s.shape[0] != R:
        s = s.repeat_interleave(GROUP, 0)[:R]
    return (_grouped(q.float()) * s[:, :, None]).reshape(R, -1)[:, :C]


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _activation(g, R, C):
    """Token rows of differing size with some large columns, as behind a norm with a learned weight."""
    x = _normal(g, (R, C))
    x *= torch.exp(_normal(g, (1, C), 0.5))
    x *= torch.exp(_normal(g, (R, 1), 0.3))
    return x


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    if c["op"] == "norm":
        dt, shape, rows, H = ACT[c["dtype"]], (c["S"], c["B"], c["H"]), c["S"] * c["B"], c["H"]
        c["seed"] = int(seed) * 1000003 + 5  # of the dropout mask
        c["eps"] = 1e-6 if c["norm"] == "rms" else 1e-5
        c["partials"] = [_normal(g, shape, 0.5).to(dt) for _ in range(c["T"])]
        c["residual"] = _normal(g, (rows, H), 1.5).to(dt)
        c["gamma"] = (1.0 + _normal(g, (H,), 0.2)).to(dt)
        c["beta"] = _normal(g, (H,), 0.1).to(dt) if c["norm"] == "ln" else None
        return c
    M, K = c["M"], c["K"]
    if c["op"] == "quant":
        x = _activation(g, M, K)
        if c["src"] in FMT:
            c["x"], c["x_scale"] = _to8(x, c["src"], False)
        else:
            c["x"], c["x_scale"] = x.to(ACT[c["src"]]), None
        return c
    N = c["N"]
    x = _activation(g, M, K)
    w = _normal(g, (N, K), K ** -0.5)
    if c["op"] == "matmul":
        c["A"], c["a_scale"] = _to8(x, c["a"], False)
        c["B"], c["b_scale"] = _to8(w, c["b"], c["block"])
        return c
    c["dy"] = _activation(g, M, N).mul_(1e-3).to(torch.bfloat16)
    c["x"], c["x_scale"] = _to8(x, "e4m3", False)
    c["wt"], c["wt_scale"] = _to8(w.t().contiguous(), "e4m3", True)
    return c


# ---- one pass ----------------------------------------------------------------------------------------------------


def _keep(n, seed, p):
    """Philox4x32-10 keep decisions of elements 0..n-1: counter g >> 2, word g & 3, key the seed."""
    low = 0xFFFFFFFF
    q = torch.arange(-(-n // 4), device="cuda", dtype=torch.int64)
    w = [q & low, q >> 32, torch.zeros_like(q), torch.zeros_like(q)]
    k0, k1 = seed & low, (seed >> 32) & low

    def wide(a, x):  # both halves of a 32 x 32 bit product
        lower = a * (x & 0xFFFF)
        upper = a * (x >> 16) + (lower >> 16)
        return upper >> 16, ((upper & 0xFFFF) << 16) | (lower & 0xFFFF)

    for _ in range(10):
        h0, l0 = wide(0xD2511F53, w[0])
        h1, l1 = wide(0xCD9E8D57, w[2])
        w = [h1 ^ w[1] ^ k0, l1, h0 ^ w[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    threshold = int(float(torch.tensor(p, dtype=torch.float32)) * 4294967296.0)
    return (torch.stack(w, 1).reshape(-1)[:n] >= threshold)


def _p32(p):
    return float(torch.tensor(p, dtype=torch.float32))


def _norm(c):
    rows, H = c["residual"].shape
    total = c["partials"][0].reshape(rows, H).double()
    for t in c["partials"][1:]:
        total += t.reshape(rows, H)
    mask = None
    if c["p"] > 0:
        keep = _keep(rows * H, c["seed"], c["p"]).view(rows, H)
        total = torch.where(keep, total / (1.0 - _p32(c["p"])), torch.zeros_like(total))
        mask = keep.to(torch.uint8)
    h = (c["residual"].double() + total).to(c["residual"].dtype)  # the stored residual stream, rounded once
    x = h.float()
    mean = None
    if c["norm"] == "ln":
        mean = x.sum(1) / H
        x = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((x * x).sum(1) / H + c["eps"])
    y = c["gamma"].float() * (x * rstd[:, None])
    if c["beta"] is not None:
        y = y + c["beta"].float()
    q, scale = _to8(y, "e4m3", False)
    return dict(h=h, q=q, scale=scale.view(E8M0), mask=mask, rstd=rstd, mean=mean)


def run(c):
    if own:
        from residual_sp_rs_gb300 import ops
        if c["op"] == "norm":
            desc = ops.make_desc(c["T"], 0, c["S"], c["B"], c["H"], c["dtype"], c["norm"], c["p"], c["eps"], c["seed"], c["T"])
            r = ops.forward_q8(desc, c["partials"], c["residual"], c["gamma"], c["beta"])
            return dict(h=r["h"], q=r["q"], scale=r["scale"].view(E8M0), mask=r["mask"], rstd=r["rstd"], mean=r["mean"])
        if c["op"] == "quant":
            r = ops.quantize_q8(c["x"], c["fmt"], block=c["block"], rowwise=c["row"], colwise=c["col"], scale=c["x_scale"])
            return {k: v.view(E8M0) if k.startswith("scale") else v for k, v in r.items() if v is not None}
        if c["op"] == "matmul":
            return ops.matmul_q8(c["A"], c["a_scale"], c["B"], c["b_scale"], out_dtype=ACT[c["out"]])
        r = ops.linear_q8_backward(c["dy"], c["x"], c["x_scale"], c["wt"], c["wt_scale"], c["fmt"])
        return dict(dx=r["dx"], dw=r["dw"])
    if c["op"] == "norm":
        return _norm(c)
    if c["op"] == "quant":
        x = c["x"].float() if c["x_scale"] is None else _from8(c["x"], c["x_scale"])
        r = {}
        if c["row"]:
            r["q"], s = _to8(x, c["fmt"], c["block"])
            r["scale"] = s.view(E8M0)
        if c["col"]:
            r["qt"], s = _to8(x.t().contiguous(), c["fmt"], c["block"])
            r["scale_t"] = s.view(E8M0)
        return r
    if c["op"] == "matmul":
        return (_from8(c["A"], c["a_scale"]) @ _from8(c["B"], c["b_scale"]).t()).to(ACT[c["out"]])
    dy = c["dy"].float()
    by_row, by_col = _from8(*_to8(dy, c["fmt"], False)), _from8(*_to8(dy.t().contiguous(), c["fmt"], False))
    x_by_col = _from8(*_to8(_from8(c["x"], c["x_scale"]).t().contiguous(), "e4m3", False))
    dx = (by_row @ _from8(c["wt"], c["wt_scale"]).t()).to(torch.bfloat16)
    return dict(dx=dx, dw=by_col @ x_by_col.t())


# ---- the definition in 64 bits -----------------------------------------------------------------------------------


def _two64(s):
    """2^s in 64 bits, for whole s from -1022 to 1023."""
    return ((s + 1023) << 52).view(torch.float64)


def _rounded64(x, fmt, block):
    """(8-bit values, scales) of x in 64 bits: the scale by logarithms, the rounding by the step at each magnitude."""
    top, digits, least = (448.0, 3, -6) if fmt == "e4m3" else (57344.0, 2, -14)
    R, C = x.shape
    G = -(-C // GROUP)
    amax = torch.stack([x[:, i * GROUP:(i + 1) * GROUP].abs().amax(1) for i in range(G)], 1)
    if block:
        amax = torch.stack([amax[i:i + GROUP].amax(0) for i in range(0, R, GROUP)], 0)
    s = torch.ceil(torch.log2(amax.clamp_min(1e-300) / top)).to(torch.int64)
    s += (amax > top * _two64(s)).to(torch.int64)  # a logarithm next to a whole number may fall on its other side
    s -= (amax <= top * _two64(s - 1)).to(torch.int64)
    scale = _two64(torch.where(amax > 0, s.clamp(-127, 127), torch.zeros_like(s)))
    per_row = scale.repeat_interleave(GROUP, 0)[:R] if block else scale
    v = x / per_row.repeat_interleave(GROUP, 1)[:, :C]
    step = _two64((torch.frexp(v)[1].to(torch.int64) - 1).clamp_min(least) - digits)
    return torch.round(v / step) * step, scale


def _value64(q, scale):
    s = _two64(scale.to(torch.int64) - 127)
    if s.shape[0] != q.shape[0]:
        s = s.repeat_interleave(GROUP, 0)[:q.shape[0]]
    return q.float().double() * s.repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def _spread64(q, scale):
    if scale.shape[0] != q.shape[0]:
        scale = scale.repeat_interleave(GROUP, 0)[:q.shape[0]]
    return q * scale.repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm":
        rows, H = c["residual"].shape
        total = sum(t.reshape(rows, H).double() for t in c["partials"])
        mask = None
        if c["p"] > 0:
            mask = _keep(rows * H, c["seed"], c["p"]).view(rows, H)
            total = total * mask / (1.0 - _p32(c["p"]))
        h = c["residual"].double() + total
        x = h.to(c["residual"].dtype).double()  # the norm reads the stored value
        mean = x.mean(1) if c["norm"] == "ln" else None
        d = x if mean is None else x - mean[:, None]
        rstd = (d.square().mean(1) + c["eps"]).rsqrt()
        y = d * rstd[:, None] * c["gamma"].double()
        if c["beta"] is not None:
            y = y + c["beta"].double()
        q, scale = _rounded64(y, "e4m3", False)
        return dict(h=h, q=q, scale=scale, mask=None if mask is None else mask.to(torch.uint8), rstd=rstd, mean=mean)
    if c["op"] == "quant":
        x = c["x"].double() if c["x_scale"] is None else _value64(c["x"], c["x_scale"])
        r = {}
        if c["row"]:
            r["q"], r["scale"] = _rounded64(x, c["fmt"], c["block"])
        if c["col"]:
            r["qt"], r["scale_t"] = _rounded64(x.t(), c["fmt"], c["block"])
        return r
    if c["op"] == "matmul":
        return _value64(c["A"], c["a_scale"]) @ _value64(c["B"], c["b_scale"]).t()
    dy = c["dy"].double()
    dx = _spread64(*_rounded64(dy, c["fmt"], False)) @ _value64(c["wt"], c["wt_scale"]).t()
    dyt = _spread64(*_rounded64(dy.t(), c["fmt"], False))
    xt = _spread64(*_rounded64(_value64(c["x"], c["x_scale"]).t(), "e4m3", False))
    return dict(dx=dx, dw=dyt @ xt.t())
