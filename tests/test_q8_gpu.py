"""The 8-bit operators on the GPU against plain 64-bit implementations.

Tolerances, from the arithmetic:
  * Scaling by a power of two is exact and a value is rounded once, so the
    quantisation of given values is compared bit for bit; so are products
    whose sums fp32 holds exactly.
  * A product's sum in fp32 over K terms, in any order and with each addition
    rounded or cut off (at most one step, 2^-23 relative): off by at most
    K 2^-23 sum |a b|; its rounding to bf16 adds 2^-8 of the result (half a
    step, torch.finfo(bfloat16).eps / 2).
  * The norm's y is a short fp32 expression of the stored h: its value is off
    by at most 2^-18 of the row's largest |y| (a mean and a variance over H
    values summed in a tree of depth <= 40, 2^-24 each, doubled by the
    division, the root and the products), so next to a rounding border it may
    fall on the other side: one step of its 8-bit type, and the scale may
    differ only when the group's largest value is that close to its border.
"""
import math

import pytest
import torch

from residual_sp_rs_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOP = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}  # largest value, digits, least normal exponent
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from residual_sp_rs_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g) * std


# ---- the definition, in 64 bits on the host ---------------------------------------------

def two(s):
    return ((s + 1023) << 52).view(torch.float64)  # -1022 <= s <= 1023


def ref_exponent(amax, fmt):
    """Smallest s with amax <= top 2^s, at least -127; 0 for a zero amax (amax finite)."""
    top, digits, least = TOP[fmt]
    m, e = torch.frexp(amax)
    s = e.to(torch.int64) - (9 if fmt == "e4m3" else 16) + (m > 0.875).to(torch.int64)
    assert bool(((amax <= top * two(s)) | (amax == 0)).all() and ((amax > top * two(s - 1)) | (amax == 0)).all())
    return torch.where(amax > 0, s.clamp_min(-127), torch.zeros_like(s))


def ref_quant(x, fmt, block=False):
    """(8-bit values as float64, scale bytes) of float64 x, groups along the rows."""
    top, digits, least = TOP[fmt]
    R, C = x.shape
    G = -(-C // 128)
    q, byte = torch.zeros_like(x), torch.zeros((-(-R // 128) if block else R, G), dtype=torch.int64)
    for r in range(byte.shape[0]):
        rows = slice(128 * r, 128 * r + 128) if block else slice(r, r + 1)
        for g in range(G):
            v = x[rows, 128 * g:128 * g + 128]
            if not torch.isfinite(v).all():
                byte[r, g] = 255
                q[rows, 128 * g:128 * g + 128] = math.nan
                continue
            s = ref_exponent(v.abs().max(), fmt)
            byte[r, g] = s + 127
            y = v * two(-s)
            step = two((torch.frexp(y)[1].to(torch.int64) - 1).clamp_min(least) - digits)
            q[rows, 128 * g:128 * g + 128] = torch.round(y / step) * step
    return q, byte


def value(q, byte):
    """What 8-bit values and scale bytes stand for, in 64 bits."""
    q, byte = q.cpu().float().double(), byte.cpu().to(torch.int64)
    s = two(byte - 127)
    s[byte == 255] = math.nan
    if s.shape[0] != q.shape[0]:
        s = s.repeat_interleave(128, 0)[:q.shape[0]]
    return q * s.repeat_interleave(128, 1)[:, :q.shape[1]]


def same(got, want):
    got = got.cpu().float().double() if got.is_floating_point() else got.cpu().to(torch.int64)
    want = want if got.is_floating_point() else want.to(torch.int64)
    return got.shape == want.shape and bool(((got == want) | ((got != got) & (want != want))).all())


def to8(x, fmt, block=False, pad=0x7F):
    """A reference-quantised 8-bit tensor on the GPU; what lies behind a row's end is `pad` (NaN bytes)."""
    q, byte = ref_quant(x.double(), fmt, block)
    def put(m, fill):
        t = torch.full((m.shape[0], max(16, (m.shape[1] + 15) // 16 * 16) + 16), fill, dtype=torch.uint8)
        t[:, :m.shape[1]] = m
        return t.to(DEV)[:, :m.shape[1]]
    bits = q.float().to(ops.Q8_DTYPE[fmt]).view(torch.uint8)
    return put(bits, pad).view(ops.Q8_DTYPE[fmt]), put(byte.to(torch.uint8), 255 if pad else 0)


# ---- quantisation -------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 128), (1, 776), (2, 129), (7, 8), (127, 130), (128, 128), (129, 257), (130, 16), (257, 1000),
          (300, 64), (33, 4096)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype,fmt,block", [(BF16, "e4m3", False), (F32, "e5m2", False), (F32, "e4m3", True),
                                             (BF16, "e5m2", True)])
def test_quantize_bits(M, K, dtype, fmt, block):
    g = gen(M * 1000 + K)
    x = (randn(g, M, K) * torch.exp(randn(g, M, 1, std=3.0)) * torch.exp(randn(g, 1, K))).to(dtype)
    r = ops.quantize_q8(x.to(DEV), fmt, block=block, colwise=True)
    q, byte = ref_quant(x.double(), fmt, block)
    assert same(r["q"], q) and same(r["scale"], byte)
    qt, byte_t = ref_quant(x.double().t().contiguous(), fmt, block)
    assert same(r["qt"], qt) and same(r["scale_t"], byte_t)
    only = ops.quantize_q8(x.to(DEV), fmt, block=block, rowwise=False, colwise=True)
    assert only["q"] is None and same(only["qt"], qt) and same(only["scale_t"], byte_t)
    only = ops.quantize_q8(x.to(DEV), fmt, block=block)
    assert only["qt"] is None and same(only["q"], q) and same(only["scale"], byte)


@pytest.mark.parametrize("M,K", [(1, 16), (5, 300), (128, 128), (333, 140)])
@pytest.mark.parametrize("src,block", [("e4m3", False), ("e5m2", False), ("e4m3", True)])
def test_requantize_bits(M, K, src, block):
    g = gen(M + K)
    x, s = to8(randn(g, M, K) * torch.exp(randn(g, M, 1, std=2.0)), src, block)
    r = ops.quantize_q8(x, "e4m3", colwise=True, scale=s)
    v = value(x, s)
    for name, want in (("q", ref_quant(v, "e4m3")), ("qt", ref_quant(v.t().contiguous(), "e4m3"))):
        assert same(r[name], want[0]) and same(r["scale" if name == "q" else "scale_t"], want[1])


@pytest.mark.parametrize("spread,low", [(0, 120), (9, 110), (15, 40), (15, 186), (16, 100), (60, 60), (3, 2), (3, 250)])
def test_requantize_over_scale_spreads(spread, low):
    """Rows whose scales are near and far from each other, at both ends of the scale bytes, with zero rows and columns,
    columns held only by the smallest scales, and a NaN."""
    g = gen(spread * 300 + low)
    M, K = 300, 270
    bits = torch.randint(0, 256, (M, 272), generator=g, dtype=torch.uint8)
    bits[(bits & 0x7F) == 0x7F] = 0x7E
    bits[7], bits[:, 11] = 0, 0
    bits[200:230, 20:40] = 0x01                    # the least subnormal
    bits[:128, 50] = 0
    bits[40, 50] = 0x81
    s = torch.randint(low, low + spread + 1, (M, 16), generator=g).to(torch.uint8)
    s[40] = low
    s[41] = low + spread
    if spread == 9:
        bits[130, 200] = 0x7F
    x, sc = bits.to(DEV)[:, :K].view(torch.float8_e4m3fn), s.to(DEV)[:, :3]
    v = value(x, sc)
    v = torch.where(v.abs() > torch.finfo(F32).max, math.inf, v)   # what fp32 cannot hold is not a number to it
    r = ops.quantize_q8(x, "e4m3", rowwise=False, colwise=True, scale=sc)
    want, byte = ref_quant(v.t().contiguous(), "e4m3")
    assert same(r["scale_t"], byte) and same(r["qt"], want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_borders(fmt):
    """Groups of zeros, of the type's largest magnitudes and next to them, ties, fp32 subnormals and the largest fp32."""
    top, digits, least = TOP[fmt]
    rows = [torch.zeros(128), torch.full((128,), -0.0)]
    for v in (top, math.nextafter(top, 0), top * (1 + 2.0 ** -23), top * 2.0 ** -130, 1e-45, 2.0 ** -126, 3e-39,
              torch.finfo(F32).max, top * 2.0 ** 100, 1.0):
        row = torch.arange(128, dtype=F32) / 127 * v
        row[0], row[5] = v, -v / 3
        rows.append(row)
    ties = torch.arange(128, dtype=torch.float64)  # midpoints of neighbouring values of one binade, and of the least
    ties[:64] = (8 + torch.arange(64) % 8 + 0.5) / 8 if fmt == "e4m3" else (4 + torch.arange(64) % 4 + 0.5) / 4
    ties[64:] = (torch.arange(64) + 0.5) * 2.0 ** (least - digits)
    ties[127] = top
    rows.append(ties.float())
    x = torch.stack([r.float() for r in rows])
    assert torch.isfinite(x).all()
    r = ops.quantize_q8(x.to(DEV), fmt)
    q, byte = ref_quant(x.double(), fmt)
    assert same(r["q"], q) and same(r["scale"], byte)


def test_quantize_nonfinite_groups_are_nan():
    x = torch.ones(3, 300)
    x[0, 5], x[1, 200], x[2, 299] = math.inf, math.nan, -math.inf
    for block in (False, True):
        r = ops.quantize_q8(x.to(DEV), block=block, colwise=True)
        for q, s, t in ((r["q"], r["scale"], x), (r["qt"], r["scale_t"], x.t().contiguous())):
            want, byte = ref_quant(t.double(), "e4m3", block)
            assert same(q, want) and same(s, byte)


def test_quantize_strided_inputs_and_untouched_padding():
    g = gen(3)
    wide = randn(g, 40, 333).to(BF16).to(DEV)
    for x in (wide[3:37, 5:205], wide[::2, :131], wide[1:2, 7:9]):   # unaligned bases, long strides
        M, K = x.shape
        q = torch.full((M, 224), 0xAB, dtype=torch.uint8, device=DEV)
        s = torch.full((M, 32), 0xCD, dtype=torch.uint8, device=DEV)
        qt = torch.full((K, 64), 0xAB, dtype=torch.uint8, device=DEV)
        st = torch.full((K, 16), 0xCD, dtype=torch.uint8, device=DEV)
        d = ops.SpQuantizeQ8Desc(M=M, K=K, ldx=x.stride(0), ldq=224, ldq_scale=32, ldqt=64, ldqt_scale=16, x_dtype=1,
                                 q_dtype=2)
        ops.sp_quantize_q8(d, x, None, q, s, qt, st)
        want, byte = ref_quant(x.cpu().double(), "e4m3")
        G = byte.shape[1]
        assert same(q[:, :K].view(torch.float8_e4m3fn), want) and same(s[:, :G], byte)
        assert bool((q[:, K:] == 0xAB).all()) and bool((s[:, G:] == 0xCD).all())
        want, byte = ref_quant(x.cpu().double().t().contiguous(), "e4m3")
        assert same(qt[:, :M].view(torch.float8_e4m3fn), want) and same(st[:, :1], byte)
        assert bool((qt[:, M:] == 0xAB).all()) and bool((st[:, 1:] == 0xCD).all())


# ---- the product ----------------------------------------------------------------------------

MM = [(1, 1, 1), (1, 16, 128), (1, 300, 2048), (2, 130, 129), (5, 64, 640), (16, 512, 1024), (17, 33, 47), (33, 200, 1500),
      (64, 128, 256), (65, 129, 300), (128, 128, 128), (129, 255, 384), (200, 96, 2000), (256, 256, 512),
      (300, 640, 1000), (520, 24, 144), (1000, 77, 16), (700, 900, 1152)]


def whole(g, *shape):
    """Whole numbers -3..3: their products with scales 1 and 2 have sums that fp32 holds exactly."""
    return torch.randint(-3, 4, shape, generator=g).double()


def exact8(g, R, C, fmt, block):
    """8-bit tensor of whole numbers with scales 2^0 or 2^1; NaN behind every row's end."""
    q = whole(g, R, C)
    G = -(-C // 128)
    byte = torch.randint(127, 129, (-(-R // 128) if block else R, G), generator=g)
    w = max(16, (C + 15) // 16 * 16) + 16
    bits = torch.full((R, w), 0x7F, dtype=torch.uint8)
    bits[:, :C] = q.float().to(ops.Q8_DTYPE[fmt]).view(torch.uint8)
    s = torch.full((byte.shape[0], (G + 15) // 16 * 16 + 16), 255, dtype=torch.uint8)
    s[:, :G] = byte.to(torch.uint8)
    q8, s8 = bits.to(DEV)[:, :C].view(ops.Q8_DTYPE[fmt]), s.to(DEV)[:, :G]
    return q8, s8, value(q8, s8)


@pytest.mark.parametrize("M,N,K", MM)
@pytest.mark.parametrize("af,bf,ablock,bblock", [("e4m3", "e4m3", False, True), ("e5m2", "e4m3", False, False),
                                                 ("e4m3", "e5m2", True, True)])
def test_matmul_exact_sums(M, N, K, af, bf, ablock, bblock):
    g = gen(M * 7 + N * 3 + K)
    a, sa, av = exact8(g, M, K, af, ablock)
    b, sb, bv = exact8(g, N, K, bf, bblock)
    want = av @ bv.t()
    assert float(want.abs().max()) < 2.0 ** 24
    got = ops.matmul_q8(a, sa, b, sb, out_dtype=F32)
    assert same(got, want)
    assert same(ops.matmul_q8(a, sa, b, sb), want.float().to(BF16).double())  # one rounding, to nearest even
    c = whole(g, M, N)
    acc = torch.full((M, N + 3), 7.5, device=DEV)
    acc[:, :N] = c.to(DEV)
    ops.matmul_q8(a, sa, b, sb, out=acc[:, :N], accumulate=True)
    assert same(acc[:, :N], want + c) and bool((acc[:, N:] == 7.5).all())
    out = torch.full((M + 1, N + 5), 7.5, device=DEV, dtype=BF16)
    ops.matmul_q8(a, sa, b, sb, out=out[:M, 1:N + 1])   # element-aligned, strided, neighbours left alone
    assert same(out[:M, 1:N + 1], want.float().to(BF16).double())
    assert bool((out[M] == 7.5).all() and (out[:, 0] == 7.5).all() and (out[:, N + 1:] == 7.5).all())


@pytest.mark.parametrize("M,N,K", [(1300, 2600, 200), (4000, 1500, 256), (2305, 4999, 129), (4096, 4104, 384),
                                   (9000, 520, 1100), (2304, 4096, 4200), (2300, 4099, 4200), (1000, 4100, 4200)])
def test_matmul_exact_sums_many_tiles(M, N, K):
    """Several tiles per CTA (2304 x 4096 x 4200: per CTA pair), ragged on every side."""
    g = gen(M + N)
    a, sa, av = exact8(g, M, K, "e4m3", False)
    b, sb, bv = exact8(g, N, K, "e4m3", True)
    want = (av.to(DEV) @ bv.to(DEV).t()).cpu()
    assert float(want.abs().max()) < 2.0 ** 24
    assert same(ops.matmul_q8(a, sa, b, sb, out_dtype=F32), want)
    assert same(ops.matmul_q8(a, sa, b, sb), want.float().to(BF16).double())
    c = torch.ones(M, N, device=DEV)
    assert same(ops.matmul_q8(a, sa, b, sb, out=c, accumulate=True), want + 1)


def plan_of(M, N, K, out_dtype=F32):
    """What the product launches on this device."""
    ld, lds = (K + 15) // 16 * 16, ((K + 127) // 128 + 15) // 16 * 16
    d = ops.SpMatmulQ8Desc(M, N, K, ld, ld, lds, lds, N, 2, 2, 0 if out_dtype == F32 else 1, 1, 1, 0, None)
    props = torch.cuda.get_device_properties(0)
    return ops.sp_matmul_q8_plan(d, props.multi_processor_count, getattr(props, "shared_memory_per_block_optin", 232448))


# CTA pairs: one and several tiles each, with accumulators that overlap (256 columns) and not, ragged on every side
PAIRS = [(4097, 1001, 4200), (2047, 2050, 4201), (4000, 2050, 4200), (3001, 4099, 4200)]


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("af,bf,ablock,bblock", [("e4m3", "e4m3", False, True), ("e5m2", "e4m3", True, False)])
def test_matmul_exact_sums_pairs(M, N, K, af, bf, ablock, bblock):
    assert plan_of(M, N, K)["pair"] and plan_of(M, N, K, BF16)["pair"]
    g = gen(M + 3 * N)
    a, sa, av = exact8(g, M, K, af, ablock)
    b, sb, bv = exact8(g, N, K, bf, bblock)
    want = (av.to(DEV) @ bv.to(DEV).t()).cpu()
    assert float(want.abs().max()) < 2.0 ** 24
    assert same(ops.matmul_q8(a, sa, b, sb, out_dtype=F32), want)
    assert same(ops.matmul_q8(a, sa, b, sb), want.float().to(BF16).double())
    c = torch.full((M, N + 3), 1.0, device=DEV)
    assert same(ops.matmul_q8(a, sa, b, sb, out=c[:, :N], accumulate=True), want + 1)
    assert bool((c[:, N:] == 1).all())


@pytest.mark.parametrize("M,N,K", [(1, 256, 4096), (3, 72, 8192), (31, 130, 1000), (130, 300, 2048), (512, 384, 1024)])
@pytest.mark.parametrize("af,block", [("e4m3", True), ("e5m2", False)])
def test_matmul_real_values(M, N, K, af, block):
    g = gen(M + N + K)
    a, sa = to8(randn(g, M, K) * torch.exp(randn(g, M, 1, std=2.0)), af)
    b, sb = to8(randn(g, N, K, std=K ** -0.5), "e4m3", block)
    av, bv = value(a, sa), value(b, sb)
    want, room = av @ bv.t(), K * 2.0 ** -23 * (av.abs() @ bv.abs().t())
    got = ops.matmul_q8(a, sa, b, sb, out_dtype=F32).cpu().double()
    assert bool(((got - want).abs() <= room).all())
    # what a plain fp32 accumulation gives is far inside that bound: hold the whole to a tenth of fp32's own
    # worst case for the norm, sqrt(K) 2^-23 instead of K 2^-23
    assert float((got - want).norm() / (av.abs() @ bv.abs().t()).norm()) <= math.sqrt(K) * 2.0 ** -23
    got = ops.matmul_q8(a, sa, b, sb).cpu().double()
    assert bool(((got - want).abs() <= room + 2.0 ** -8 * (want.abs() + room)).all())


def test_matmul_scales_over_their_range():
    """Scale bytes near both ends, whose products are ordinary, and zeros with the largest scale."""
    g = gen(5)
    a, sa, _ = exact8(g, 20, 256, "e4m3", False)
    b, sb, _ = exact8(g, 30, 256, "e4m3", False)
    sa[:, 0], sa[:, 1], sb[:, 0], sb[:, 1] = 1, 252, 253, 3
    want = value(a, sa) @ value(b, sb).t()
    assert same(ops.matmul_q8(a, sa, b, sb, out_dtype=F32), want)
    a.view(torch.uint8)[:, :128] = 0
    sa[:, 0] = 254
    want = value(a, sa) @ value(b, sb).t()
    assert same(ops.matmul_q8(a, sa, b, sb, out_dtype=F32), want)


def test_matmul_nan_stays_in_its_row_and_column():
    g = gen(6)
    a, sa, av = exact8(g, 140, 300, "e4m3", False)
    b, sb, bv = exact8(g, 70, 300, "e4m3", False)
    sa[3, 2] = 255                       # a scale that is NaN
    b.view(torch.uint8)[9, 17] = 0x7F    # a value that is NaN
    got = ops.matmul_q8(a, sa, b, sb, out_dtype=F32).cpu()
    want = (av @ bv.t()).float()
    want[3], want[:, 9] = math.nan, math.nan
    assert same(got, want.double())


def test_scales_in_torchs_exponent_type():
    g = gen(8)
    a, sa, av = exact8(g, 20, 300, "e4m3", False)
    b, sb, bv = exact8(g, 30, 300, "e4m3", True)
    e8 = torch.float8_e8m0fnu
    assert same(ops.matmul_q8(a, sa.view(e8), b, sb.view(e8), out_dtype=F32), av @ bv.t())
    x, y = (ops.quantize_q8(a, rowwise=False, colwise=True, scale=s) for s in (sa, sa.view(e8)))
    assert torch.equal(x["qt"].view(torch.uint8), y["qt"].view(torch.uint8)) and torch.equal(x["scale_t"], y["scale_t"])


def test_results_do_not_change_from_call_to_call():
    """One token with K split in a cluster, single CTAs and pairs: the same sums in the same order every time."""
    assert plan_of(1, 2048, 8192)["split_k"] > 1 and not plan_of(1000, 4100, 4200)["pair"] and plan_of(*PAIRS[3])["pair"]
    for M, N, K in ((1, 2048, 8192), (300, 500, 1024), (1000, 4100, 4200), PAIRS[3]):
        g = torch.Generator(device=DEV).manual_seed(M)
        a = ops.quantize_q8(torch.randn(M, K, device=DEV, generator=g))
        b = ops.quantize_q8(torch.randn(N, K, device=DEV, generator=g), block=True)
        want = ops.matmul_q8(a["q"], a["scale"], b["q"], b["scale"], out_dtype=F32)
        for _ in range(10):
            assert torch.equal(ops.matmul_q8(a["q"], a["scale"], b["q"], b["scale"], out_dtype=F32), want)


def test_matmul_empty_sum_and_empty_sides():
    a, sa = ops.q8_empty(5, 0, DEV, torch.float8_e4m3fn), ops.q8_empty(5, 0, DEV)
    b, sb = ops.q8_empty(7, 0, DEV, torch.float8_e4m3fn), ops.q8_empty(7, 0, DEV)
    assert bool((ops.matmul_q8(a, sa, b, sb) == 0).all())
    c = torch.full((5, 7), 3.0, device=DEV)
    assert bool((ops.matmul_q8(a, sa, b, sb, out=c, accumulate=True) == 3).all())
    e, se = ops.q8_empty(0, 64, DEV, torch.float8_e4m3fn), ops.q8_empty(0, 1, DEV)
    f, sf = ops.q8_empty(7, 64, DEV, torch.float8_e4m3fn), ops.q8_empty(7, 1, DEV)
    assert ops.matmul_q8(e, se, f, sf).shape == (0, 7) and ops.matmul_q8(f, sf, e, se).shape == (7, 0)


# ---- the region's forward with an 8-bit norm output -------------------------------------------

def region(T, S, B, H, dtype, norm, p, seed, nshards=None):
    g = gen(seed)
    dt = {"bf16": BF16, "f32": F32}[dtype]
    desc = ops.make_desc(T, 0, S, B, H, dtype, norm, p, 1e-5, seed, T if nshards is None else nshards)
    parts = [randn(g, S, B, H, std=0.5).to(dt).to(DEV) for _ in range(T)]
    res = randn(g, desc.rows, H).to(dt).to(DEV)
    gamma = (1 + randn(g, H, std=0.3)).to(dt).to(DEV)
    beta = randn(g, H, std=0.2).to(dt).to(DEV) if norm == "ln" else None
    return desc, parts, res, gamma, beta


def check_q8_norm(desc, f, gamma, beta):
    """q and scale against the 64-bit norm of the stored h."""
    h = f["h"].cpu().double()
    mean = h.mean(1, keepdim=True) if beta is not None else torch.zeros(h.shape[0], 1, dtype=torch.float64)
    d = h - mean
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + desc.eps) * gamma.cpu().double()
    if beta is not None:
        y = y + beta.cpu().double()
    slack = 2.0 ** -18 * y.abs().amax(1, keepdim=True)
    H = y.shape[1]
    byte = f["scale"].cpu().to(torch.int64)
    for g in range(byte.shape[1]):
        v = y[:, 128 * g:128 * g + 128]
        amax = v.abs().amax(1)
        lo = ref_exponent((amax - slack[:, 0]).clamp_min(0), "e4m3") + 127
        hi = ref_exponent(amax + slack[:, 0], "e4m3") + 127
        # (an all-zero group has the scale 1; such a group is exactly zero on both sides)
        zero = amax == 0
        assert bool(((byte[:, g] >= lo) & (byte[:, g] <= hi) | zero & (byte[:, g] == 127)).all())
        s = two(byte[:, g:g + 1] - 127)
        got = f["q"][:, 128 * g:128 * g + 128].cpu().float().double() * s
        step = two((torch.frexp(v / s)[1].to(torch.int64) - 1).clamp_min(-6) - 3) * s
        # half a step, and the slack: a value pushed over a binade's end rounds with the next binade's step
        assert bool(((got - v).abs() <= 0.5 * step * (1 + 2.0 ** -18) + 2 * slack).all())


CASES = [(1, 1, 1, 768, "bf16", "rms", 0.0), (1, 1, 1, 8192, "bf16", "rms", 0.0), (1, 1, 1, 8192, "bf16", "ln", 0.0),
         (1, 3, 1, 8, "bf16", "rms", 0.0), (2, 16, 2, 64, "f32", "rms", 0.1), (2, 16, 2, 136, "f32", "ln", 0.1),
         (2, 6, 1, 264, "bf16", "rms", 0.1), (2, 64, 2, 768, "bf16", "rms", 0.1), (4, 8, 1, 1000, "bf16", "ln", 0.5),
         (8, 16, 1, 4096, "bf16", "ln", 0.1), (8, 8, 2, 8192, "bf16", "rms", 0.1), (8, 8, 1, 8192, "bf16", "ln", 0.0),
         (3, 9, 1, 16384, "bf16", "rms", 0.0), (1, 5, 1, 16384, "bf16", "ln", 0.1), (8, 8, 1, 8192, "f32", "rms", 0.0),
         (1, 400, 1, 2056, "bf16", "rms", 0.0), (5, 5, 3, 520, "bf16", "ln", 0.3)]


@pytest.mark.parametrize("T,S,B,H,dtype,norm,p", CASES)
def test_forward_q8(T, S, B, H, dtype, norm, p):
    desc, parts, res, gamma, beta = region(T, S, B, H, dtype, norm, p, H + S)
    f = ops.forward_q8(desc, parts, res, gamma, beta)
    ref = ops.forward(desc, parts, res, gamma, beta)
    assert (f["mask"] is None and ref["mask"] is None) or torch.equal(f["mask"], ref["mask"])
    # h: rounded to fp32, then to bf16: half a step of bf16 and half a step of fp32 of the exact sum, whose fp32
    # partial sums are off by at most T 2^-24 of what they add
    keep = 1.0 if f["mask"] is None else f["mask"].cpu().double()
    total = sum(t.view(-1, H).cpu().double() for t in parts) * keep / (1.0 - float(desc.p))
    slack = (T + 2) * 2.0 ** -24 * (sum(t.view(-1, H).cpu().double().abs() for t in parts) / (1.0 - float(desc.p)) +
                                    res.cpu().double().abs())
    want = res.cpu().double() + total
    half = torch.zeros_like(want) if dtype == "f32" else two(torch.frexp(want.abs() + slack)[1].to(torch.int64) - 9)
    h = f["h"].cpu().double()
    assert bool(((h - want).abs() <= half + slack).all())
    # the statistics are those of the stored h
    mean = h.mean(1) if norm == "ln" else torch.zeros(h.shape[0], dtype=torch.float64)
    rstd = 1 / torch.sqrt(((h - mean[:, None]) ** 2).mean(1) + desc.eps)
    assert float(((f["rstd"].cpu().double() - rstd) / rstd).abs().max()) < 1e-5
    if norm == "ln":
        assert bool(((f["mean"].cpu().double() - mean).abs() <= 1e-5 * torch.maximum(mean.abs(), 1 / rstd)).all())
    if dtype == "f32":
        assert torch.equal(f["h"], ref["h"]) and torch.equal(f["rstd"], ref["rstd"])
    check_q8_norm(desc, f, gamma, beta)


def test_forward_q8_rows_and_untouched_neighbours():
    T, S, B, H = 2, 24, 2, 264
    desc, parts, res, gamma, beta = region(T, S, B, H, "bf16", "rms", 0.1, 9)
    full = ops.forward_q8(desc, parts, res, gamma, beta)
    rows = desc.rows
    q = torch.full((rows, 288), 0x5A, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, 32), 0x5A, dtype=torch.uint8, device=DEV)
    h, mask, rstd = torch.empty_like(full["h"]), torch.empty_like(full["mask"]), torch.empty_like(full["rstd"])
    done = 0
    for b, e in ((0, 10), (10, 12), (12, 40)):
        ops.sp_rs_dropout_residual_norm_fwd_q8_rows(desc, b, e - b, parts, res, gamma, beta, h,
                                                    q[:, :H].view(torch.float8_e4m3fn), s[:, :3], mask, rstd, None)
        done = e
        assert bool((q[done:] == 0x5A).all() and (s[done:] == 0x5A).all())
    assert torch.equal(q[:done, :H], full["q"].view(torch.uint8)[:done]) and bool((q[:, H:] == 0x5A).all())
    assert torch.equal(s[:done, :3], full["scale"][:done]) and bool((s[:, 3:] == 0x5A).all())
    assert torch.equal(h[:done], full["h"][:done]) and torch.equal(rstd[:done], full["rstd"][:done])


def test_forward_q8_zero_rows_and_nonfinite():
    """A zero row has q = 0 and scale 1; a row with an infinity has NaN scales and nothing spreads to others."""
    for dtype, H in (("bf16", 768), ("f32", 256), ("bf16", 16384)):
        desc, parts, res, gamma, beta = region(1, 4, 1, H, dtype, "rms", 0.0, 2)
        res[1], parts[0][1] = 0, 0
        res[2, 5] = math.inf
        f = ops.forward_q8(desc, parts, res, gamma, beta)
        assert math.isinf(float(f["h"][2, 5]))
        assert bool((f["q"][1].float() == 0).all() and (f["scale"][1] == 127).all())
        assert int(f["scale"][2, 0]) == 255 and bool(f["q"][2].float().isnan()[:128].all())
        keep = torch.tensor([0, 3])
        check_q8_norm(desc, {k: f[k].cpu()[keep] if f[k].element_size() > 1 else f[k].cpu().view(torch.uint8)[keep].view(f[k].dtype)
                             for k in ("h", "q", "scale")}, gamma, beta)


# ---- a run of them together ----------------------------------------------------------------------

def step(desc, parts, res, gamma, w, dy):
    """One region and the 8-bit column-parallel product behind it, forward and backward."""
    f = ops.forward_q8(desc, parts, res, gamma)
    wq = ops.quantize_q8(w, block=True, colwise=True)
    out = ops.matmul_q8(f["q"], f["scale"], wq["q"], wq["scale"])
    g = ops.linear_q8_backward(dy, f["q"], f["scale"], wq["qt"], wq["scale_t"], "e5m2")
    b = ops.backward(desc, g["dx"], None, f["h"], gamma, f["mask"], f["rstd"])
    return f, out, g, b


def step_inputs(T, S, B, H, N, seed=3):
    desc, parts, res, gamma, _ = region(T, S, B, H, "bf16", "rms", 0.1, seed)
    g = gen(seed + 1)
    return desc, parts, res, gamma, randn(g, N, H, std=H ** -0.5).to(DEV), randn(g, desc.rows, N, std=1e-3).to(BF16).to(DEV)


def test_training_step_together():
    """Each stage against its 64-bit formula on the stage's own inputs."""
    desc, parts, res, gamma, w, dy = step_inputs(2, 50, 2, 264, 200)
    f, out, g, b = step(desc, parts, res, gamma, w, dy)
    xv = value(f["q"], f["scale"])
    wv = value(*(t.float() if t.dtype != torch.int64 else t for t in ref_quant(w.cpu().double(), "e4m3", True)))
    want = xv @ wv.t()
    room = 264 * 2.0 ** -23 * (xv.abs() @ wv.abs().t())
    assert bool(((out.cpu().double() - want).abs() <= room + 2.0 ** -8 * (want.abs() + room)).all())
    dyd = dy.cpu().double()
    dr, dc = value(*ref_quant(dyd, "e5m2")), value(*ref_quant(dyd.t().contiguous(), "e5m2"))
    want = dr @ wv
    room = 200 * 2.0 ** -23 * (dr.abs() @ wv.abs())
    assert bool(((g["dx"].cpu().double() - want).abs() <= room + 2.0 ** -8 * (want.abs() + room)).all())
    xc = value(*ref_quant(xv.t().contiguous(), "e4m3"))
    want, room = dc @ xc.t(), desc.rows * 2.0 ** -23 * (dc.abs() @ xc.abs().t())
    assert bool(((g["dw"].cpu().double() - want).abs() <= room).all())
    # the gradients against those of the unquantised layer: dY and x are within half a step of their type (2^-3 and
    # 2^-4 of a value, a half of it in the mean), so dW of random signs is off by about a tenth
    full = dyd.t() @ xv
    assert float((g["dw"].cpu().double() - full).norm() / full.norm()) < 2.0 ** -3 + 2.0 ** -4
    assert bool(torch.isfinite(b["d_res"].float()).all() and torch.isfinite(b["dgamma"]).all())


@pytest.mark.parametrize("M,N,K,dtype,fmt,block", [(1, 16, 16, BF16, "e4m3", True), (77, 95, 361, BF16, "e5m2", True),
                                                   (300, 129, 264, F32, "e4m3", False)])
def test_linear_backward_is_its_parts(M, N, K, dtype, fmt, block):
    """The same bits as the quantisations and products called one by one; dw added to what is given; no rows."""
    g = gen(M + N + K)
    dy = randn(g, M, N, std=1e-3).to(dtype).to(DEV)
    x = ops.quantize_q8(randn(g, M, K).to(DEV))
    w = ops.quantize_q8(randn(g, N, K).to(DEV), block=block, colwise=True)
    got = ops.linear_q8_backward(dy, x["q"], x["scale"], w["qt"], w["scale_t"], fmt)
    d = ops.quantize_q8(dy, fmt, colwise=True)
    xt = ops.quantize_q8(x["q"], rowwise=False, colwise=True, scale=x["scale"])
    assert torch.equal(got["dx"], ops.matmul_q8(d["q"], d["scale"], w["qt"], w["scale_t"]))
    dw = ops.matmul_q8(d["qt"], d["scale_t"], xt["qt"], xt["scale_t"], out_dtype=F32)
    assert torch.equal(got["dw"], dw)
    base = randn(g, N, K + 2).to(DEV)
    total = base.clone()
    more = ops.linear_q8_backward(dy, x["q"], x["scale"], w["qt"], w["scale_t"], fmt, dw=total[:, 1:K + 1], dx_dtype=F32)
    assert more["dx"].dtype == F32 and torch.equal(total[:, 1:K + 1], base[:, 1:K + 1] + dw)
    assert torch.equal(total[:, 0], base[:, 0]) and torch.equal(total[:, K + 1], base[:, K + 1])
    none = ops.linear_q8_backward(dy[:0], x["q"][:0], x["scale"][:0], w["qt"], w["scale_t"], fmt, dw=total[:, 1:K + 1])
    assert none["dx"].shape == (0, K) and torch.equal(total[:, 1:K + 1], base[:, 1:K + 1] + dw)
    for bad in (dict(dy=dy[:, :N - 1]), dict(fmt="e3m4"), dict(dw=total), dict(dx_dtype=torch.float16)):
        args = dict(dict(dy=dy, x_q=x["q"], x_scale=x["scale"], wt_q=w["qt"], wt_scale=w["scale_t"], fmt=fmt), **bad)
        with pytest.raises(ValueError):
            ops.linear_q8_backward(**args)


def test_gradient_against_differences():
    """dx and dw are the gradients of L = sum(dy * (x W^T)), linear in x and in W: differences of the 8-bit forward
    product itself, with steps that 8 bits hold exactly."""
    g = gen(11)
    x, sx, xv = exact8(g, 24, 128, "e4m3", False)
    w, sw, wv = exact8(g, 40, 128, "e4m3", True)
    dy = whole(g, 24, 40)
    wt, swt = to8(wv.t().contiguous(), "e4m3", True, pad=0)
    grads = ops.linear_q8_backward(dy.to(F32).to(DEV), x, sx, wt, swt, dx_dtype=F32)
    dw = grads["dw"].cpu().double()
    base = (dy * ops.matmul_q8(x, sx, w, sw, out_dtype=F32).cpu().double()).sum()
    for i, k in ((0, 0), (7, 100), (23, 127)):   # x[i,k] one step of its scale up
        up, d = x.clone(), float(two(sx[i, 0].cpu().to(torch.int64) - 127))
        up.view(torch.uint8)[i, k] = torch.tensor(float(x[i, k]) + 1).to(x.dtype).view(torch.uint8)
        moved = (dy * ops.matmul_q8(up, sx, w, sw, out_dtype=F32).cpu().double()).sum()
        assert float((moved - base) / d) == float(grads["dx"][i, k])
    for j, k in ((0, 0), (39, 64)):
        up, d = w.clone(), float(two(sw[0, 0].cpu().to(torch.int64) - 127))
        up.view(torch.uint8)[j, k] = torch.tensor(float(w[j, k]) + 1).to(w.dtype).view(torch.uint8)
        moved = (dy * ops.matmul_q8(x, sx, up, sw, out_dtype=F32).cpu().double()).sum()
        assert float((moved - base) / d) == float(dw[j, k])


def test_captured_step_replays_on_new_inputs():
    a, b = step_inputs(2, 32, 2, 264, 200, seed=3), step_inputs(2, 32, 2, 264, 200, seed=4)
    want = [tuple(t.clone() for t in (o[0]["h"], o[1], o[2]["dx"], o[2]["dw"], o[3]["dgamma"]))
            for o in (step(a[0], *b[1:]), step(a[0], *a[1:]))]
    live = [p.clone() for p in a[1]], *(t.clone() for t in a[2:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a[0], *live)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, out, g, bw = step(a[0], *live)
    for src, expect in zip((b, a), want):
        for dst, s in zip([*live[0], *live[1:]], [*src[1], *src[2:]]):
            dst.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((f["h"], out, g["dx"], g["dw"], bw["dgamma"]), expect):
            assert torch.equal(got, w)


def test_calls_on_two_streams_at_once():
    """No state is shared between calls: runs on two streams give what they give alone, every time."""
    ins = [step_inputs(2, 64, 2, 768, 520, seed=s) for s in (5, 6)]
    alone = [[t.clone() for t in (o[1], o[2]["dx"], o[2]["dw"])] for o in (step(*i) for i in ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        outs = []
        for st, i in zip(streams, ins):
            with torch.cuda.stream(st):
                outs.append(step(*i))
        torch.cuda.synchronize()
        for o, want in zip(outs, alone):
            for got, w in zip((o[1], o[2]["dx"], o[2]["dw"]), want):
                assert torch.equal(got, w)


def test_stream_argument():
    desc, parts, res, gamma, w, dy = step_inputs(2, 16, 2, 264, 72)
    want = step(desc, parts, res, gamma, w, dy)
    torch.cuda.synchronize()
    for st in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        f = ops.forward_q8(desc, parts, res, gamma, stream=st)
        wq = ops.quantize_q8(w, block=True, colwise=True, stream=st)
        out = ops.matmul_q8(f["q"], f["scale"], wq["q"], wq["scale"], stream=st)
        g = ops.linear_q8_backward(dy, f["q"], f["scale"], wq["qt"], wq["scale_t"], "e5m2", stream=st)
        torch.cuda.synchronize()
        assert torch.equal(out, want[1]) and torch.equal(g["dx"], want[2]["dx"]) and torch.equal(g["dw"], want[2]["dw"])


def test_status_word_stays_clear():
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = gen(1)
    a, sa, av = exact8(g, 100, 500, "e4m3", False)
    b, sb, bv = exact8(g, 100, 500, "e4m3", False)
    assert same(ops.matmul_q8(a, sa, b, sb, out_dtype=F32, status=word), av @ bv.t())
    assert int(word) == 0


def test_pipelined_forward_and_gather_on_one_nccl_rank():
    """The exchange's forwards with an 8-bit y, and its gather, give the plain call's bits (T = 1)."""
    import socket

    import torch.distributed as dist

    from residual_sp_rs_gb300 import sp_exchange as ex
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        port = sk.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1)
    try:
        desc, parts, res, gamma, _ = region(1, 200, 2, 264, "bf16", "rms", 0.1, 4)
        want = ops.forward_q8(desc, parts, res, gamma)
        for pipelined in (True, False):
            out = {k: torch.zeros_like(v) for k, v in want.items() if v is not None and k not in ("q", "scale")}
            q, s = ops.q8_empty(desc.rows, 264, DEV, torch.float8_e4m3fn), ops.q8_empty(desc.rows, 3, DEV)
            if pipelined:
                ex.forward_pipelined(desc, parts[0], res, gamma, None, out["h"], (q, s), out["mask"], out["rstd"], None)
            else:
                ex.forward_from_shard_rows(desc, parts[0].view(1, -1, 264), res, gamma, None, out["h"], (q, s),
                                           out["mask"], out["rstd"], None)
            fq, fs = ex.gather_q8(q, s)
            torch.cuda.synchronize()
            assert all(torch.equal(out[k], want[k]) for k in out)
            assert torch.equal(fq.view(torch.uint8), want["q"].view(torch.uint8)) and torch.equal(fs, want["scale"])
    finally:
        dist.destroy_process_group()


def test_readme_example_runs():
    """The 8-bit example, as written, behind the one before it."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), flags=re.S)
    names = {}
    for block in blocks[:2]:
        exec(compile(block, "README.md", "exec"), names)
    torch.cuda.synchronize()
    assert names["out"].shape == (4096, 1536) and names["lin"]["dw"].shape == (1536, 768)
    assert all(bool(torch.isfinite(t.float()).all()) for t in (names["out"], names["lin"]["dx"], names["g"]["dgamma"]))


# ---- bounded waits --------------------------------------------------------------------------------

TIMEOUT_SHAPES = [(1300, 2600, 200), (1000, 4100, 4200), (9, 1000, 4096), PAIRS[1]]   # single CTAs twice, K split, pairs


def _timeout_child(path):
    out = []
    for M, N, K in TIMEOUT_SHAPES:
        g = gen(M)
        a, sa, _ = exact8(g, M, K, "e4m3", False)
        b, sb, _ = exact8(g, N, K, "e4m3", True)
        word = torch.zeros(1, dtype=torch.int32, device=DEV)
        c = ops.matmul_q8(a, sa, b, sb, out_dtype=F32, status=word)
        torch.cuda.synchronize()
        out.append((c.cpu(), int(word)))
    torch.save(out, path)


def test_timed_out_wait_marks_its_tiles_and_sets_the_status_word(tmp_path):
    """The library's test hooks shorten the waits to 2 ms and make CTA 0 skip one stage, so that the waits on it run
    out: the kernel returns, that CTA's tiles are NaN, all others are right, and the status word says so."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    path = str(tmp_path / "child.pt")
    assert [(p["pair"], p["split_k"] > 1) for p in (plan_of(*s) for s in TIMEOUT_SHAPES)] == [(0, False), (0, False), (0, True), (1, False)]
    env = dict(os.environ, SPFUSE_TEST_WAIT_NS="2000000", SPFUSE_TEST_DROP_STAGE="1")
    code = f"import sys; sys.path.insert(0, {root!r}); from tests.test_q8_gpu import _timeout_child; _timeout_child({path!r})"
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    for (M, N, K), (c, word) in zip(TIMEOUT_SHAPES, torch.load(path)):
        g = gen(M)
        a, sa, av = exact8(g, M, K, "e4m3", False)
        b, sb, bv = exact8(g, N, K, "e4m3", True)
        want = (av.to(DEV) @ bv.to(DEV).t()).float().cpu()
        bad = c.isnan()
        assert word == 0x4 and bool(bad.any()) and not bool(bad.all())
        assert torch.equal(c[~bad], want[~bad])
        word = torch.zeros(1, dtype=torch.int32, device=DEV)   # and without the hooks
        assert torch.equal(ops.matmul_q8(a, sa, b, sb, out_dtype=F32, status=word).cpu(), want) and int(word) == 0
