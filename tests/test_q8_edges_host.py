"""Host-side checks of the 8-bit operators' launches (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def spf():
    from residual_sp_rs_gb300 import build, ops
    build.build()
    return ops


def test_smoke_runs_pairs_and_a_split_product(spf):
    import __graft_entry__ as entry
    assert spf.sp_matmul_q8_plan(entry.product_desc(spf, *entry.PAIRS), 152, 232448)["pair"] == 1
    assert spf.sp_matmul_q8_plan(entry.product_desc(spf, *entry.SPLIT), 152, 232448)["split_k"] > 1
    assert entry.SPLIT[1:] == entry.PAIRS[1:]   # the same operands, a few rows of A


def plan(spf, M, N, K, c_dtype, ldc, sms=152, optin=232448):
    ld, lds = -(-K // 128) * 128, -(-K // 2048) * 16
    return spf.sp_matmul_q8_plan(spf.SpMatmulQ8Desc(M, N, K, ld, ld, lds, lds, ldc, 2, 2, c_dtype, 1, 1, 0, None), sms, optin)


def test_plans_of_swapped_products(spf):
    """The shapes that the GPU tests count on for swapped operands with several tiles per CTA."""
    from tests.test_q8_edges_gpu import F32, SWAPPED
    for M, N, K, dtype, pad, bn, turns in SWAPPED:
        p = plan(spf, M, N, K, 0 if dtype == F32 else 1, N + pad)
        assert (p["swapped"], p["split_k"], p["bn"], -(-p["tiles"] // p["ctas"])) == (1, 1, bn, turns), (M, N, K, p)
        assert (p["acc1_col"] < p["bn"]) == (bn == 256)


def test_clusters_never_wait_for_tensor_memory(spf):
    """The CTAs of a cluster wait for each other holding their tensor memory, so two clusters that meet on SMs (of two
    streams) must never want more than its 512 columns: shared memory keeps others out where they would."""
    sm, overhead = 228 * 1024, 1024     # an SM's shared memory; what the device keeps of it per CTA
    least = {}                          # columns -> the least shared memory of a cluster's CTA that has them
    sides = (1, 5, 16, 33, 80, 128, 144, 200, 256, 300, 700, 1000, 2049, 4096, 10000, 30000)
    for M in sides:
        for N in sides:
            for K in (128, 256, 512, 1000, 2048, 4200, 8192, 20000, 40000):
                for c_dtype, pad in ((0, 0), (1, 0), (1, 1)):
                    p = plan(spf, M, N, K, c_dtype, N + pad)
                    if p["pair"] or p["split_k"] > 1:
                        least[p["tmem_cols"]] = min(least.get(p["tmem_cols"], sm), p["smem_bytes"] + overhead)
    assert {32, 256, 512} <= set(least)

    def most(room):     # columns of the CTAs that fit into `room`
        return max([0] + [cols + most(room - size) for cols, size in least.items() if size <= room])

    assert most(sm) <= 512, least


def test_adding_an_empty_sum_launches_nothing(spf):
    """C += A B^T with K = 0 leaves C, bit for bit: there is nothing to launch, and no device is needed."""
    fake = 1 << 20
    d = spf.SpMatmulQ8Desc(5, 7, 0, 16, 16, 16, 16, 7, 2, 2, 0, 1, 1, 1, None)
    assert spf.lib().sp_matmul_q8(ctypes.byref(d), None, None, None, None, fake, None) == 0
    assert spf.lib().sp_matmul_q8(ctypes.byref(d), None, None, None, None, None, None) == 1   # its checks stay
    assert spf.lib().sp_matmul_q8(ctypes.byref(d), None, None, None, None, fake + 2, None) == 3
    assert spf.sp_matmul_q8_plan(d, 152, 232448)["ctas"] == 0
    d.accumulate = 0
    assert spf.sp_matmul_q8_plan(d, 152, 232448)["ctas"] > 0
