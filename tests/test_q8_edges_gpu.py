"""The 8-bit operators where waits run out and launches take their rarer shapes.

Compared bit for bit, or with the tolerance that stands at the comparison.
"""
import os
import subprocess
import sys

import pytest
import torch

from residual_sp_rs_gb300 import ops

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from residual_sp_rs_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def child(function, path, **env):
    """Runs `function` of this module with `path` in a process of its own with these variables set."""
    code = f"import sys; sys.path.insert(0, {ROOT!r}); from tests import test_q8_edges_gpu as t; t.{function}({path!r})"
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, **env), cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return torch.load(path)


def bits(t):
    return None if t is None else t.contiguous().view(torch.uint8).cpu()


# ---- requantisation whose copies do not land ---------------------------------------------

# several tiles for each of the resident CTAs (1280 and more), ragged on both sides, and less than one
REQUANT = [(5003, 4090, dict(colwise=True)), (5000, 4096, dict(rowwise=False, colwise=True)),
           (4999, 4097, dict(block=True)), (200, 130, dict(colwise=True))]


def requantised():
    out = []
    for M, K, kw in REQUANT:
        g = torch.Generator(device=DEV).manual_seed(M)
        x = ops.quantize_q8(torch.randn(M, K, device=DEV, generator=g))
        ops.quantize_q8(x["q"], scale=x["scale"], **kw)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        r = ops.quantize_q8(x["q"], scale=x["scale"], **kw)
        end.record()
        torch.cuda.synchronize()
        out.append((begin.elapsed_time(end), {k: bits(v) for k, v in r.items()}))
    return out


def save_requantised(path):
    torch.save(requantised(), path)


@pytest.mark.parametrize("stage", [0, 1, 2])
def test_requantisation_goes_on_without_its_copies(tmp_path, stage):
    """The library's test hooks shorten the waits to 20 ms and make CTA 0 leave out one of its copies: the call takes
    that long, and the result is the same bits."""
    late = child("save_requantised", str(tmp_path / "late.pt"), SPFUSE_TEST_WAIT_NS="20000000",
                 SPFUSE_TEST_DROP_STAGE=str(stage))
    for (M, K, kw), (ms, got), (_, want) in zip(REQUANT, late, requantised()):
        tiles = -(-M // 128) * -(-K // 128)
        ctas = min(tiles, 2 * torch.cuda.get_device_properties(0).multi_processor_count)
        assert (ms >= 20) == (stage * ctas < tiles), (M, K, ms)   # CTA 0 has a tile of that number
        for name in want:
            assert (got[name] is None) == (want[name] is None), name
            assert want[name] is None or torch.equal(got[name], want[name]), (M, K, name)


# ---- the residual stream of the 8-bit forward ------------------------------------------------

@pytest.mark.parametrize("H", [768, 16384])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
def test_residual_far_below_the_partials(H, p):
    """h is the sum to one fp32 step, which is 2^-16 bf16 steps, rounded to bf16 (half a step), also where the residual
    is 2^-12 to 2^-30 of the partials or they of it; it is the other forward's h unless the sum is that near a midpoint
    of bf16 values."""
    rows = 64
    g = torch.Generator(device=DEV).manual_seed(H)
    part = torch.randn(rows, 1, H, generator=g, device=DEV)
    far = torch.tensor([0, 8, 12, 13, 16, 17, 20, 24, 30, -8, -12, -13, -16, -20, -30, 40], device=DEV).repeat(rows // 16)
    res = torch.randn(rows, H, generator=g, device=DEV) * torch.ldexp(torch.ones(rows, device=DEV), -far)[:, None]
    part[0, 0, :8], res[0, :8] = 1.0, -1.0   # and where they cancel
    part, res, gamma = part.bfloat16(), res.bfloat16(), torch.ones(H, device=DEV).bfloat16()
    d = ops.make_desc(1, 0, rows, 1, H, "bf16", "rms", p, 1e-6, 7, 1)
    f, ref = ops.forward_q8(d, [part], res, gamma), ops.forward(d, [part], res, gamma)
    keep = 1.0 if p == 0 else f["mask"].double()
    exact = res.double() + part.view(rows, H).double() * keep / (1.0 - float(d.p))   # 2^-52 off
    step = torch.ldexp(torch.ones_like(exact), (torch.frexp(exact)[1] - 8).clamp_min(-133))   # between bf16 values
    h, other = f["h"].double(), ref["h"].double()
    assert bool(((h - exact).abs() <= (0.5 + 2.0 ** -16 * (1 + 2.0 ** -6)) * step).all())
    moved = h != other
    assert bool((((h + other) / 2 - exact).abs()[moved] <= 2.0 ** -16 * (1 + 2.0 ** -6) * step[moved]).all())
    assert p == 0.1 or not bool(moved.any())


LATE_NORMS = [(768, "rms"), (4096, "ln"), (8192, "ln")]   # rows in stages of several, of one, and (T = 8) in column chunks


def norms(status):
    """The 8-bit forward of 1600 and more rows: its outputs, what the status word says, and the rows of CTA 0."""
    out = []
    for H, norm in LATE_NORMS:
        T = 8 if H == 8192 else 2
        g = torch.Generator(device=DEV).manual_seed(H)
        rand = lambda *shape: torch.randn(shape, generator=g, device=DEV).bfloat16()
        status.zero_()
        d = ops.make_desc(T, 0, 1600, 1, H, "bf16", norm, 0.1, 1e-6, 7, T, status=status)
        f = ops.forward_q8(d, [rand(1600, 1, H) for _ in range(T)], rand(1600, H), rand(H), rand(H) if norm == "ln" else None)
        torch.cuda.synchronize()
        out.append(({k: bits(v) for k, v in f.items() if v is not None}, f["rstd"].cpu(), int(status)))
    return out


def save_norms(path):
    torch.save(norms(torch.zeros(1, dtype=torch.int32, device=DEV)), path)


def test_forward_whose_wait_runs_out(tmp_path):
    """CTA 0 leaves out a stage: rows of its that it did not finish have NaN in rstd, all other rows are right, and the
    status word says so."""
    late = child("save_norms", str(tmp_path / "n.pt"), SPFUSE_TEST_WAIT_NS="2000000", SPFUSE_TEST_DROP_STAGE="1")
    props = torch.cuda.get_device_properties(0)
    for (H, norm), (got, rstd, word), (want, _, clean) in zip(LATE_NORMS, late, norms(torch.zeros(1, dtype=torch.int32, device=DEV))):
        d = ops.make_desc(8 if H == 8192 else 2, 0, 1600, 1, H, "bf16", norm, 0.1, 1e-6, 7, 8 if H == 8192 else 2)
        plan = ops.sp_plan_describe(d, props.multi_processor_count, getattr(props, "shared_memory_per_block_optin", 232448))["fwd"]
        assert plan["tma"] and (word, clean) == (0x1, 0)
        bad = rstd.isnan()
        # (in column chunks stage 1 is part of row 0, and a single row group stops there, before all the other rows)
        assert bool(bad.any()) and not bool(bad[plan["rows_per_cta"]:].any())
        assert plan["chunked"] or not bool(bad[:plan["rows_per_cta"]].all())
        for k in want:
            if k != "mean":   # of the unfinished rows it is not written either
                assert torch.equal(got[k].view(len(rstd), -1)[~bad], want[k].view(len(rstd), -1)[~bad]), (H, k)


# ---- products in a row ----------------------------------------------------------------------

def plan_of(M, N, K, out_dtype=torch.float32, ldc=None):
    """What the product launches on this device."""
    ld, lds = (K + 15) // 16 * 16, ((K + 127) // 128 + 15) // 16 * 16
    d = ops.SpMatmulQ8Desc(M, N, K, ld, ld, lds, lds, N if ldc is None else ldc, 2, 2, 0 if out_dtype == torch.float32 else 1,
                           1, 1, 0, None)
    props = torch.cuda.get_device_properties(0)
    return ops.sp_matmul_q8_plan(d, props.multi_processor_count, getattr(props, "shared_memory_per_block_optin", 232448))


def operand(R, C, seed):
    """Whole numbers -3..3 in e4m3 with scales 1 and 2: fp32 holds the sums of their products.  Values, scales, float64."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    whole = torch.randint(-3, 4, (R, C), generator=g, device=DEV)
    q, s = ops.q8_empty(R, C, DEV), ops.q8_empty(R, -(-C // 128), DEV)
    q.copy_(whole.float().to(torch.float8_e4m3fn).view(torch.uint8))
    s.copy_(torch.randint(127, 129, s.shape, generator=g, device=DEV))
    v = whole.double() * (s.double() - 126).repeat_interleave(128, 1)[:, :C]   # 2^0 and 2^1
    return q.view(torch.float8_e4m3fn), s, v


def test_kernels_in_a_row_behind_pairs():
    """The next kernel starts while the last CTAs of a pair leave: pairs behind pairs, a quantisation and a split
    product behind pairs, each launch with the bits that it has alone."""
    shapes = [(2047, 2050, 512), (1, 2048, 4096), (2047, 2050, 4201)]
    assert plan_of(*shapes[2])["pair"] and plan_of(*shapes[1])["split_k"] > 1
    ins = [(operand(M, K, M), operand(N, K, N)) for M, N, K in shapes]
    want = [a[2] @ b[2].t() for a, b in ins]
    x = ins[2][0]
    quant = ops.quantize_q8(x[0], scale=x[1], colwise=True)
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for i in (2, 2, 1, 2, 0, 2):
            (a, sa, _), (b, sb, _) = ins[i]
            outs.append((i, ops.matmul_q8(a, sa, b, sb, out_dtype=torch.float32)))
            if i == 2:
                q = ops.quantize_q8(x[0], scale=x[1], colwise=True)
        for i, c in outs:
            assert torch.equal(c.double(), want[i])
        assert all(torch.equal(bits(q[k]), bits(quant[k])) for k in quant)


# ---- swapped operands, several tiles per CTA ------------------------------------------------

# M, N, K, C's type, columns behind C's rows, columns per tile (256: the accumulators overlap), tiles of the busiest CTA
BF16, F32 = torch.bfloat16, torch.float32
SWAPPED = [(1, 50000, 4096, BF16, 0, 16, 2), (1, 50000, 4096, F32, 0, 16, 2), (18, 41193, 129, BF16, 0, 32, 2),
           (1300, 2600, 200, BF16, 1, 48, 2), (65, 30866, 4743, F32, 0, 80, 2), (138, 34730, 2608, F32, 1, 144, 2),
           (1679, 8260, 5243, F32, 1, 240, 3), (2770, 3330, 6545, BF16, 0, 256, 2), (15043, 624, 4714, F32, 1, 256, 2)]


def swapped(M, N, K, dtype, pad):
    """A product and what it is exactly; C has `pad` columns more, left alone."""
    (a, sa, av), (b, sb, bv) = operand(M, K, M), operand(N, K, N)
    c = torch.full((M, N + pad), 7.5, device=DEV, dtype=dtype)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.matmul_q8(a, sa, b, sb, out=c[:, :N], status=word)
    return c, int(word), (a, sa, b, sb), (av @ bv.t()).float()   # |sum| <= 36 K < 2^24


@pytest.mark.parametrize("M,N,K,dtype,pad,bn,turns", SWAPPED)
def test_swapped_products_of_several_tiles(M, N, K, dtype, pad, bn, turns):
    p = plan_of(M, N, K, dtype, N + pad)
    assert p["swapped"] and p["split_k"] == 1 and p["bn"] == bn and -(-p["tiles"] // p["ctas"]) == turns, p
    c, word, args, want = swapped(M, N, K, dtype, pad)
    assert word == 0 and torch.equal(c[:, :N], want.to(dtype)) and bool((c[:, N:] == 7.5).all())
    if dtype == F32:
        ops.matmul_q8(*args, out=c[:, :N], accumulate=True)
        assert torch.equal(c[:, :N], 2 * want) and bool((c[:, N:] == 7.5).all())
    for _ in range(5):   # on real values, whose sums depend on the order: the same bits every time
        outs = [ops.matmul_q8(args[0], args[1], args[2].view(torch.float8_e5m2), args[3], out_dtype=F32) for _ in range(2)]
        assert torch.equal(bits(outs[0]), bits(outs[1]))


LATE = [SWAPPED[0], SWAPPED[3], SWAPPED[7]]   # two CTAs on an SM, with an unaligned C, overlapping accumulators


def save_swapped(path):
    torch.save([(c.cpu(), word) for c, word, _, _ in (swapped(*s[:5]) for s in LATE)], path)


def test_swapped_products_whose_wait_runs_out(tmp_path):
    """CTA 0 leaves out a stage: its tiles are NaN from there on, all others right, and the status word says so."""
    late = child("save_swapped", str(tmp_path / "s.pt"), SPFUSE_TEST_WAIT_NS="2000000", SPFUSE_TEST_DROP_STAGE="1")
    for (M, N, K, dtype, pad, _, _), (c, word) in zip(LATE, late):
        want = swapped(M, N, K, dtype, pad)[3].to(dtype).cpu()
        c, bad = c[:, :N], c[:, :N].isnan()
        assert word == 0x4 and bool(bad.any()) and not bool(bad.all())
        assert torch.equal(c[~bad], want[~bad])


def test_adding_an_empty_sum_keeps_the_signs_of_zeros():
    a, sa = ops.q8_empty(5, 0, DEV, torch.float8_e4m3fn), ops.q8_empty(5, 0, DEV)
    c = torch.full((5, 5), -0.0, device=DEV)
    ops.matmul_q8(a, sa, a, sa, out=c, accumulate=True)
    assert bool(torch.signbit(c).all())
    ops.matmul_q8(a, sa, a, sa, out=c)
    assert not bool(torch.signbit(c).any()) and bool((c == 0).all())


# ---- values and scales at the ends, offsets past 32 bits ------------------------------------

@pytest.mark.parametrize("M,N", [(5, 40), (300, 300)])
def test_smallest_scale_and_infinities(M, N):
    """Scale byte 0 is 2^-127, and an infinity (e5m2) is one in its row and its sign, NaN against zeros."""
    (a, sa, av), (b, sb, bv) = operand(M, 300, 1), operand(N, 300, 2)
    sa[:, 1], sb[:, 1] = 0, 254   # 2^-127 2^127
    av, bv = av.clone(), bv.clone()
    av[:, 128:256], bv[:, 128:256] = a[:, 128:256].double(), b[:, 128:256].double()
    assert torch.equal(ops.matmul_q8(a, sa, b, sb, out_dtype=F32).double(), av @ bv.t())
    q = a.float().to(torch.float8_e5m2)   # -3..3 are e5m2 values
    x = ops.q8_empty(M, 300, DEV, torch.float8_e5m2)
    x.copy_(q)
    x.view(torch.uint8)[3, 7] = 0x7C      # infinity
    want = (av @ bv.t()).float()
    want[3] = torch.where(bv[:, 7] == 0, torch.nan, torch.sign(bv[:, 7]) * torch.inf).float()
    got = ops.matmul_q8(x, sa, b, sb, out_dtype=F32)
    assert bool(((got == want) | (got.isnan() & want.isnan())).all())


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 elements: the last rows and columns are what a call on them alone gives."""
    M, K = 131200 + 77, 32768 + 128
    x = torch.empty(M, K, device=DEV, dtype=BF16)
    for i in range(0, M, 32768):
        x[i:i + 32768].normal_()
    r = ops.quantize_q8(x, colwise=True)
    tail = x[131072:]                     # a multiple of 128 rows down
    t = ops.quantize_q8(tail, colwise=True)
    assert torch.equal(bits(r["q"][131072:]), bits(t["q"])) and torch.equal(r["scale"][131072:], t["scale"])
    assert torch.equal(bits(r["qt"][:, 131072:]), bits(t["qt"])) and torch.equal(r["scale_t"][:, 1024:], t["scale_t"])
    del x, tail, r, t
    x, s = ops.q8_empty(M, K, DEV), ops.q8_empty(M, -(-K // 128), DEV)
    for i in range(0, M, 16384):
        q, e, v = operand(min(16384, M - i), K, i)
        x[i:i + 16384], s[i:i + 16384] = q.view(torch.uint8), e
    x, v = x.view(torch.float8_e4m3fn), v[-1000:].clone()   # the last rows' values
    del q, e
    z = ops.quantize_q8(x, scale=s, rowwise=False, colwise=True)
    u = ops.quantize_q8(x[131072:], scale=s[131072:], rowwise=False, colwise=True)
    assert torch.equal(bits(z["qt"][:, 131072:]), bits(u["qt"])) and torch.equal(z["scale_t"][:, 1024:], u["scale_t"])
    del z, u
    # x as A and as B, with few and with many rows of the other operand; |sum| <= 36 K < 2^24
    w, sw, wv = operand(300, K, 5)
    for rows in (3, 300):
        c = ops.matmul_q8(x, s, w[:rows], sw[:rows], out_dtype=F32)
        assert torch.equal(c[-len(v):], (v @ wv[:rows].t()).float())
        c = ops.matmul_q8(w[:rows], sw[:rows], x, s, out_dtype=F32)
        assert torch.equal(c[:, -len(v):], (wv[:rows] @ v.t()).float())
    del x, s
    # C past 32 bits, of sums that fp32 and bf16 hold
    (a, sa, av), (b, sb, bv) = operand(66000, 16, 1), operand(33000, 16, 2)
    c = ops.matmul_q8(a, sa, b, sb, out_dtype=F32)
    assert torch.equal(c[-500:], (av[-500:] @ bv.t()).float()) and torch.equal(c[:, -500:], (av @ bv[-500:].t()).float())


def test_forward_past_32_bits():
    rows, H = 263000, 8192
    part = torch.empty(rows, 1, H, device=DEV, dtype=BF16).normal_()
    res = torch.empty(rows, H, device=DEV, dtype=BF16).normal_()
    gamma = torch.ones(H, device=DEV, dtype=BF16)
    f = ops.forward_q8(ops.make_desc(1, 0, rows, 1, H, "bf16", "rms", 0.0, 1e-6, 7, 1), [part], res, gamma)
    t = ops.forward_q8(ops.make_desc(1, 0, 1000, 1, H, "bf16", "rms", 0.0, 1e-6, 7, 1), [part[-1000:]], res[-1000:], gamma)
    assert torch.equal(f["h"][-1000:], t["h"]) and torch.equal(f["rstd"][-1000:], t["rstd"])
    assert torch.equal(bits(f["q"][-1000:]), bits(t["q"])) and torch.equal(f["scale"][-1000:], t["scale"])


# ---- the status word of the gradients ------------------------------------------------------

def gradients(word):
    """dY in e4m3 and x of whole numbers, 1300 x 700 x 600; dw added to ones."""
    x, sx, _ = operand(1300, 600, 1)
    wt, swt, _ = operand(600, 700, 2)
    g = torch.Generator(device=DEV).manual_seed(3)
    dy = torch.randint(-3, 4, (1300, 700), generator=g, device=DEV).float()
    dw = torch.ones(700, 600, device=DEV)
    r = ops.linear_q8_backward(dy, x, sx, wt, swt, dw=dw, dx_dtype=torch.float32, status=word)
    torch.cuda.synchronize()
    return r["dx"].cpu(), r["dw"].cpu()


def save_gradients(path):
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.save((*gradients(word), int(word)), path)


def test_gradients_report_a_wait_that_ran_out(tmp_path):
    """The hooks of the library make CTA 0 of either product leave out a stage: the status word says so, its tiles are
    NaN and all others right."""
    dx, dw, status = child("save_gradients", str(tmp_path / "g.pt"), SPFUSE_TEST_WAIT_NS="2000000",
                           SPFUSE_TEST_DROP_STAGE="1")
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = gradients(word)
    assert int(word) == 0 and not any(bool(t.isnan().any()) for t in want)
    assert status == 0x4
    for got, right in zip((dx, dw), want):
        bad = got.isnan()
        assert bool(bad.any()) and not bool(bad.all()) and torch.equal(got[~bad], right[~bad])


def test_gradients_refuse_a_status_word_elsewhere():
    x, sx, _ = operand(20, 30, 1)
    wt, swt, _ = operand(30, 40, 2)
    dy = torch.ones(20, 40, device=DEV)
    with pytest.raises(ValueError, match="one device"):
        ops.linear_q8_backward(dy, x, sx, wt, swt, status=torch.zeros(1, dtype=torch.int32))
    side = torch.cuda.Stream()
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    r = ops.linear_q8_backward(dy, x, sx, wt, swt, stream=side, status=word)
    side.synchronize()
    assert int(word) == 0 and bool(torch.isfinite(r["dw"]).all())
