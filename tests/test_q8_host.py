"""Host-side checks of the 8-bit entry points (no GPU): what they refuse, the
descriptors' layout and the calls that launch nothing."""
import ctypes
import os
import subprocess
import sys
import textwrap

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def spf():
    from residual_sp_rs_gb300 import build, ops
    build.build()
    return ops


def test_struct_layout_matches_header(spf):
    assert ctypes.sizeof(spf.SpQuantizeQ8Desc) == 88 and spf.SpQuantizeQ8Desc.x_dtype.offset == 64
    assert ctypes.sizeof(spf.SpMatmulQ8Desc) == 96 and spf.SpMatmulQ8Desc.a_dtype.offset == 64
    assert spf.SpMatmulQ8Desc.status.offset == 88


# ---- the region's forward with an 8-bit norm output ------------------------------

def _fwd(spf, H=64, ldq=64, lds=16, q=FAKE, scale=FAKE, h=FAKE, dtype="bf16", rows=None, **kw):
    d = spf.make_desc(2, 0, kw.pop("S", 16), 2, H, dtype, "rms", 0.1, 1e-6)
    arr = (ctypes.c_void_p * 2)(FAKE, FAKE)
    L = spf.lib()
    if rows is None:
        return L.sp_rs_dropout_residual_norm_fwd_q8(ctypes.byref(d), arr, FAKE, FAKE, None, h, q, ldq, scale, lds,
                                                    FAKE, FAKE, None, None)
    return L.sp_rs_dropout_residual_norm_fwd_q8_rows(ctypes.byref(d), *rows, arr, FAKE, FAKE, None, h, q, ldq, scale,
                                                     lds, FAKE, FAKE, None, None)


def test_fwd_q8_refusals(spf):
    assert _fwd(spf) in (0, 6)                    # valid (6 = no GPU here)
    assert _fwd(spf, S=15) == 2                   # the region's own checks
    assert _fwd(spf, H=12) == 2
    assert _fwd(spf, ldq=48) == 2                 # shorter than H
    assert _fwd(spf, ldq=72) == 2                 # no multiple of 16
    assert _fwd(spf, ldq=1 << 62) == 2
    assert _fwd(spf, lds=8) == 2
    assert _fwd(spf, lds=0) == 2
    assert _fwd(spf, H=64 * 33, ldq=64 * 33, lds=16) == 2  # 17 groups
    assert _fwd(spf, q=0) == 1 and _fwd(spf, scale=0) == 1 and _fwd(spf, h=0) == 1
    assert _fwd(spf, q=FAKE + 8) == 3 and _fwd(spf, scale=FAKE + 1) == 3
    assert _fwd(spf, S=0, q=0, scale=0) == 0      # no rows: nothing checked or touched
    assert _fwd(spf, rows=(0, 17)) == 1 and _fwd(spf, rows=(-1, 2)) == 1
    assert _fwd(spf, rows=(16, 0), q=0) == 0
    assert _fwd(spf, rows=(3, 5)) in (0, 6)


# ---- quantisation ------------------------------------------------------------------

def _quant(spf, x=FAKE, xs=None, q=FAKE, qs=FAKE, qt=FAKE, qts=FAKE, **kw):
    f = dict(M=100, K=72, ldx=72, ldx_scale=16, ldq=80, ldq_scale=16, ldqt=112, ldqt_scale=16, x_dtype=1, q_dtype=2,
             x_scale_rows=0, block=0, reserved=0)
    f.update(kw)
    d = spf.SpQuantizeQ8Desc(**f)
    return spf.lib().sp_quantize_q8(ctypes.byref(d), x, xs, q, qs, qt, qts, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=4), 4), (dict(x_dtype=-1), 4), (dict(q_dtype=0), 4), (dict(q_dtype=1), 4), (dict(q_dtype=4), 4),
    (dict(block=2), 1), (dict(reserved=1), 1), (dict(x_dtype=2, xs=FAKE, ldx=80), 1),
    (dict(M=-1), 2), (dict(K=-1), 2), (dict(M=1 << 31), 2), (dict(K=1 << 31, ldx=1 << 31), 2),
    (dict(ldx=71), 2), (dict(ldx=1 << 60), 2), (dict(ldq=64), 2), (dict(ldq=72), 2), (dict(ldq_scale=1), 2),
    (dict(ldqt=96), 2), (dict(ldqt=104), 2), (dict(ldqt_scale=8), 2),
    (dict(M=(1 << 31) - 1, K=(1 << 31) - 1, ldx=(1 << 31), ldq=1 << 31, ldqt=1 << 31), 2),
    (dict(x_dtype=2, xs=FAKE, ldx=72, x_scale_rows=1), 2),       # an 8-bit x needs 16-byte strides
    (dict(x_dtype=2, xs=FAKE, ldx=80, x_scale_rows=1, ldx_scale=4), 2),
    (dict(x=None), 1), (dict(x_dtype=2, ldx=80, x_scale_rows=1), 1), (dict(qs=None), 1), (dict(qts=None), 1),
    (dict(q=None, qt=None), 1),
    (dict(x=FAKE + 1), 3), (dict(x_dtype=0, x=FAKE + 2), 3), (dict(q=FAKE + 8), 3), (dict(qt=FAKE + 4), 3),
    (dict(qs=FAKE + 1), 3), (dict(qts=FAKE + 2), 3),
    (dict(x_dtype=3, xs=FAKE + 1, ldx=80, x_scale_rows=1), 3), (dict(x_dtype=3, x=FAKE + 8, xs=FAKE, ldx=80, x_scale_rows=1), 3),
])
def test_quantize_refusals(spf, kw, code):
    assert _quant(spf, **kw) == code


def test_quantize_accepts(spf):
    for kw in [dict(), dict(q=None, qs=None, ldq=0, ldq_scale=0), dict(qt=None, qts=None, ldqt=0, ldqt_scale=0),
               dict(block=1), dict(x_dtype=0, x=FAKE + 4), dict(x=FAKE + 2),
               dict(x_dtype=3, xs=FAKE, ldx=80, x_scale_rows=128)]:
        assert _quant(spf, **kw) in (0, 6), kw
    assert _quant(spf, M=0, x=None, qs=None, qts=None) == 0
    assert _quant(spf, K=0, x=None, qs=None, qts=None) == 0
    assert spf.lib().sp_quantize_q8(None, FAKE, None, FAKE, FAKE, None, None, None) == 1


# ---- the product -------------------------------------------------------------------

def _mm(spf, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, c=FAKE, **kw):
    f = dict(M=5, N=7, K=200, lda=208, ldb=208, lda_scale=16, ldb_scale=16, ldc=7, a_dtype=2, b_dtype=3, c_dtype=1,
             a_scale_rows=1, b_scale_rows=128, accumulate=0, status=None)
    f.update(kw)
    d = spf.SpMatmulQ8Desc(**f)
    return spf.lib().sp_matmul_q8(ctypes.byref(d), a, sa, b, sb, c, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a_dtype=1), 4), (dict(b_dtype=0), 4), (dict(a_dtype=4), 4), (dict(c_dtype=2), 4),
    (dict(accumulate=1), 4), (dict(accumulate=2), 1), (dict(a_scale_rows=0), 1), (dict(b_scale_rows=64), 1),
    (dict(M=-1), 2), (dict(N=-1), 2), (dict(K=-1), 2), (dict(M=1 << 31), 2), (dict(N=1 << 31, ldc=1 << 31), 2),
    (dict(K=1 << 31, lda=1 << 31, ldb=1 << 31), 2), (dict(lda=192), 2), (dict(lda=200), 2), (dict(ldb=201), 2),
    (dict(ldb=1 << 61), 2), (dict(lda_scale=1), 2), (dict(ldb_scale=17), 2), (dict(ldc=6), 2), (dict(ldc=1 << 60), 2),
    (dict(a=None), 1), (dict(sa=None), 1), (dict(b=None), 1), (dict(sb=None), 1), (dict(c=None), 1),
    (dict(a=FAKE + 8), 3), (dict(sa=FAKE + 4), 3), (dict(b=FAKE + 1), 3), (dict(sb=FAKE + 8), 3), (dict(c=FAKE + 1), 3),
    (dict(c=FAKE + 2, c_dtype=0), 3), (dict(status=FAKE + 2), 3),
])
def test_matmul_refusals(spf, kw, code):
    assert _mm(spf, **kw) == code


def test_matmul_accepts(spf):
    for kw in [dict(), dict(c=FAKE + 2), dict(c_dtype=0, accumulate=1, c=FAKE + 4), dict(ldc=9),
               dict(K=0, a=None, b=None, sa=None, sb=None), dict(status=FAKE + 4)]:
        assert _mm(spf, **kw) in (0, 6), kw
    assert _mm(spf, M=0, a=None, c=None) == 0
    assert _mm(spf, N=0, b=None, c=None) == 0
    assert spf.lib().sp_matmul_q8(None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == 1


def test_launch_failure_is_reported(spf):
    code = textwrap.dedent(f"""
        import sys
        sys.path.insert(0, {ROOT!r})
        from residual_sp_rs_gb300 import ops as spf
        from tests import test_q8_host as t
        print(t._fwd(spf), t._quant(spf), t._mm(spf))
    """)
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, SPFUSE_FAIL_LAUNCH="1"),
                         capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["6", "6", "6"]


# ---- the binding ---------------------------------------------------------------------

def test_binding_refuses_what_it_cannot_pass_on(spf):
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        spf.quantize_q8(x)
    with pytest.raises(ValueError, match="expected"):
        spf.quantize_q8(x.double())
    with pytest.raises(ValueError, match="expected"):
        spf.quantize_q8(x, fmt="e3m4")
    with pytest.raises(ValueError, match="nothing"):
        spf.quantize_q8(x, rowwise=False)
    a, s = torch.zeros(4, 256, dtype=f8), torch.zeros(4, 2, dtype=u8)
    with pytest.raises(ValueError, match="CUDA"):
        spf.matmul_q8(a, s, a, s)
    with pytest.raises(ValueError, match="out to add to"):
        spf.matmul_q8(a, s, a, s, accumulate=True)
    for values, scales in [(a, s[:3]), (a, torch.zeros(4, 1, dtype=u8)), (a, s.float()), (a, None), (a.float(), s)]:
        with pytest.raises(ValueError):
            spf._q8_operand("a", values, scales)
    with pytest.raises(ValueError, match="dense rows"):
        spf._q8_operand("a", torch.zeros(256, 4, dtype=f8).t(), s)
    assert spf._q8_operand("a", a, s[:1])[4] == 128   # one row of scales for four rows: a block
    assert spf._q8_operand("a", a, s)[4] == 1


def test_q8_empty_strides(spf):
    for cols in (0, 1, 15, 16, 17, 128):
        t = spf.q8_empty(3, cols, "cpu")
        assert t.shape == (3, cols) and t.stride(0) % 16 == 0 and t.stride(0) >= cols


# ---- what the product launches -----------------------------------------------------------

def _plan(spf, M, N, K, c_dtype=1, sms=152, optin=232448, ldc=None):
    ld, lds = (K + 15) // 16 * 16, ((K + 127) // 128 + 15) // 16 * 16
    d = spf.SpMatmulQ8Desc(M, N, K, ld, ld, lds, lds, N if ldc is None else ldc, 2, 2, c_dtype, 1, 1, 0, None)
    return spf.sp_matmul_q8_plan(d, sms, optin)


SIDES = (1, 16, 33, 64, 65, 128, 300, 768, 1000, 1536, 2049, 4096, 8192, 16384, 40000)


@pytest.mark.parametrize("M", SIDES)
def test_matmul_plans_fit_the_device(spf, M):
    """Shared memory, tensor memory, the ring, the join and the grid over sides and depths."""
    for N in SIDES:
        for K in (0, 1, 128, 129, 512, 768, 2048, 4200, 8192, 30000):
            for c_dtype, sms, optin in ((1, 152, 232448), (0, 152, 232448), (0, 148, 232448), (1, 16, 232448)):
                p = _plan(spf, M, N, K, c_dtype, sms, optin)
                what = (M, N, K, c_dtype, sms, p)
                cg, X, Y = 1 + p["pair"], (N if p["swapped"] else M), (M if p["swapped"] else N)
                nkb = -(-K // 128)
                assert 16 <= p["bn"] <= 256 and p["bn"] % (16 * cg) == 0, what
                assert p["tiles"] == -(-X // (128 * cg)) * -(-Y // p["bn"]), what
                # shared memory: the ring, the scales' ring, the epilogue's pieces, alignment and static arrays
                rest = 1024 + 4 * 512 * (1 + -(-p["bn"] // 128)) + (0 if p["swapped"] else 8 * 4096)
                assert p["stage_bytes"] == 128 * (128 + p["bn"] // cg) and p["smem_bytes"] == rest + p["stages"] * p["stage_bytes"], what
                assert 2 <= p["stages"] <= 12 and (p["smem_bytes"] + 2048) * p["ctas_per_sm"] <= optin, what
                # tensor memory: two accumulators (sharing less than a piece of columns; one when K is split), then the scales
                assert p["tmem_cols"] in (32, 64, 128, 256, 512) and p["tmem_cols"] * p["ctas_per_sm"] <= 512, what
                assert p["scale_col"] % 16 == 0 and p["scale_col"] + 4 + 4 * -(-p["bn"] // 128) <= p["tmem_cols"], what
                assert p["bn"] <= p["scale_col"], what
                if p["split_k"] == 1:
                    assert p["acc1_col"] >= p["bn"] - 16 and p["acc1_col"] + p["bn"] <= p["scale_col"], what
                else:
                    assert p["swapped"] and p["split_k"] in (2, 4, 8) and p["split_k"] <= nkb, what
                    assert p["bn"] * 512 <= p["stages"] * p["stage_bytes"], what     # the fp32 sums take the ring's place
                    assert p["ctas"] == p["tiles"] * p["split_k"] <= p["ctas_per_sm"] * sms, what
                assert p["ctas"] % (cg * p["split_k"]) == 0 and p["ctas"] <= max(p["ctas_per_sm"] * sms, cg), what
                assert p["block"] == (256 if p["swapped"] else 384), what


def test_matmul_plans_of_known_shapes(spf):
    one = _plan(spf, 1, 8192, 8192)
    assert one["swapped"] and one["bn"] == 16 and one["split_k"] == 4 and one["ctas_per_sm"] == 2
    large = _plan(spf, 16384, 4096, 8192)
    assert large["pair"] and large["bn"] == 256 and large["ctas"] == 152
    pages = _plan(spf, 4096, 1536, 768)
    # the estimate, in clocks: 2 turns of tiles 176 wide 5200 + 1.1 * (2 * 6 * 304 * 128 / 62 + 600) + 2 * 1200 * 1.15 = 16904,
    # 192 wide 5200 + 1.1 * (2 * 6 * 320 * 128 / 62 + 600) + 2 * 1200 = 16981
    assert not pages["pair"] and not pages["swapped"] and pages["bn"] == 176

    # the shapes that the GPU tests count on: pairs with one and with several tiles each, accumulators that overlap
    # (256 columns) and not, ragged on every side
    for M, N, K, pair, swapped, split, turns in ((1300, 2600, 200, 0, 0, 0, 2), (1000, 4100, 4200, 0, 0, 0, 1),
                                                 (9, 1000, 4096, 0, 1, 1, 1), (2304, 4096, 4200, 1, 0, 0, 2),
                                                 (4097, 1001, 4200, 1, 0, 0, 1), (2047, 2050, 4201, 1, 0, 0, 1),
                                                 (4000, 2050, 4200, 1, 0, 0, 2), (3001, 4099, 4200, 1, 0, 0, 3)):
        for c_dtype in (0, 1):
            p = _plan(spf, M, N, K, c_dtype)
            got = (p["pair"], p["swapped"], int(p["split_k"] > 1))
            assert got == (pair, swapped, split), (M, N, K, p)
            assert -(-p["tiles"] * (1 + p["pair"]) * p["split_k"] // p["ctas"]) >= turns, (M, N, K, p)
    assert _plan(spf, 4000, 2050, 4200)["bn"] == 256 and _plan(spf, 3001, 4099, 4200)["bn"] < 256


def test_matmul_plan_refusals(spf):
    info = spf.SpMatmulQ8Plan()
    assert ctypes.sizeof(info) == 72
    d = spf.SpMatmulQ8Desc(5, 7, 200, 208, 208, 16, 16, 7, 2, 3, 1, 1, 128, 0, None)
    L = spf.lib()
    assert L.sp_matmul_q8_plan(ctypes.byref(d), 152, 232448, ctypes.byref(info)) == 0 and info.tiles > 0
    assert L.sp_matmul_q8_plan(ctypes.byref(d), 0, 232448, ctypes.byref(info)) == 1
    assert L.sp_matmul_q8_plan(ctypes.byref(d), 152, 232448, None) == 1
    for optin in (1, 2048, 20000):   # no room for two stages
        assert L.sp_matmul_q8_plan(ctypes.byref(d), 152, optin, ctypes.byref(info)) == 1
    big = spf.SpMatmulQ8Desc(16384, 4096, 8192, 8192, 8192, 64, 64, 4096, 2, 2, 1, 1, 1, 0, None)
    for sms in (1, 2, 3):            # a pair needs two
        assert L.sp_matmul_q8_plan(ctypes.byref(big), sms, 232448, ctypes.byref(info)) == 0
        assert info.ctas <= sms and not (sms == 1 and info.pair)
    d.lda = 200
    assert L.sp_matmul_q8_plan(ctypes.byref(d), 152, 232448, ctypes.byref(info)) == 2
    d.lda, d.M = 208, 0
    assert L.sp_matmul_q8_plan(ctypes.byref(d), 152, 232448, ctypes.byref(info)) == 0 and info.tiles == 0


# ---- the gather across ranks -----------------------------------------------------------

def _gather_rank(rank, world, port, out, R, H):
    import torch.distributed as dist
    sys.path.insert(0, ROOT)
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    from residual_sp_rs_gb300 import ops, sp_exchange as ex
    g = torch.Generator().manual_seed(rank)
    q = ops.q8_empty(R, H, "cpu")
    s = ops.q8_empty(R, -(-H // 128), "cpu")
    q.copy_(torch.randint(0, 256, (R, H), generator=g))
    s.copy_(torch.randint(0, 256, s.shape, generator=g))
    fq, fs = ex.gather_q8(q.view(torch.float8_e4m3fn), s)
    assert fq.dtype == torch.float8_e4m3fn and fq.stride(0) % 16 == 0 and fs.stride(0) % 16 == 0
    torch.save((q, s, fq.view(torch.uint8).clone(), fs.clone()), f"{out}.{rank}")
    dist.barrier()
    dist.destroy_process_group()


@pytest.mark.parametrize("world,R,H", [(2, 3, 256), (2, 5, 264), (4, 1, 2048)])
def test_gather_q8_on_gloo_ranks(tmp_path, world, R, H):
    import socket

    import torch.multiprocessing as mp
    with socket.socket() as sock:
        sock.bind(("127.0.0.1", 0))
        port = sock.getsockname()[1]
    out = str(tmp_path / "g")
    mp.start_processes(_gather_rank, args=(world, port, out, R, H), nprocs=world, start_method="spawn")
    parts = [torch.load(f"{out}.{r}") for r in range(world)]
    for _, _, fq, fs in parts:
        assert torch.equal(fq, torch.cat([p[0] for p in parts])) and torch.equal(fs, torch.cat([p[1] for p in parts]))
