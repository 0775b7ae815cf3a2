"""Register and spill budgets of the recurrence's and the state cache's kernels, from ptxas's report (no GPU needed).

Their launch shapes rest on them: the scan kernels share an SM between 16 warps (128 registers a thread), the cache's
block-per-group kernels between 32 (64), its streamed step fills one with 27 warps (72). The spill budgets are what
each was measured at."""
import shutil
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_kernel_resources import _compile, _nvcc, _parse


@pytest.fixture(scope="module")
def report():
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not found")
    out = tempfile.mkdtemp(prefix="gla_ptxas_")
    try:
        with ThreadPoolExecutor(max_workers=3) as ex:
            results = list(ex.map(_compile, [(nvcc, f, out) for f in ("gla_scan", "gla_scan_bwd", "gla_cache")]))
    finally:
        shutil.rmtree(out, ignore_errors=True)
    kernels = {}
    for name, rc, text in results:
        assert rc == 0, text
        kernels.update(_parse(text))
    return kernels


@pytest.mark.parametrize("kernel,regs,spill", [("k_scan_fwd", 128, 0), ("k_scan_bwd", 128, 16), ("k_scan_step", 64, 0),
                                               ("k_cache_store", 64, 0), ("k_cache_load", 64, 48),
                                               ("k_cache_step", 64, 48), ("k_cache_stream", 72, 32)])
def test_budget(report, kernel, regs, spill):
    found = {n: r for n, r in report.items() if kernel in n}
    assert found
    for n, (r, st, ld) in found.items():
        assert r <= regs, (n, r)
        assert st <= spill and ld <= 2 * spill, (n, st, ld)
