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
