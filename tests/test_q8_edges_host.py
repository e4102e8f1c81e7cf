"""Host-side checks of the 8-bit operators' launches (no GPU)."""
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
