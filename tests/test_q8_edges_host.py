"""Host-side checks of the 8-bit operators' launches (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def spf():
    from residual_sp_rs_gb300 import build, ops
    build.build()
    return ops


def test_smoke_runs_a_product_in_pairs(spf):
    import __graft_entry__ as entry
    assert spf.sp_matmul_q8_plan(entry.pairs_desc(spf), 152, 232448)["pair"] == 1
