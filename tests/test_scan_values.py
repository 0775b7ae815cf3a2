"""Values of the elementwise recurrence where a comparison of test_scan could not fail or a launch was not reached: the
fp64 bounds of test_scan with NaN and infinities counted as wrong, packed sequences against each one alone, and calls
with more channel tiles than the device holds at once, which run in blocks without a cluster for several rounds."""
import numpy as np
import pytest
import torch

from chunkwise_linear_rnn_gla_b200 import build as gbuild, scan
from tests import test_scan as ts


@pytest.fixture(scope="module")
def lib():
    gbuild.build()


def within(got, want, dtype=torch.float32):
    """test_scan.close, for which a NaN is no match: every value has to be within its bound."""
    v, e = want
    got = ts.f64(got)
    tol = e + ts.half_step(dtype) * (np.abs(v) + e) * (dtype != torch.float32) + 1e-37
    assert got.shape == v.shape and np.isfinite(v).all() and np.isfinite(tol).all()
    ok = np.abs(got - v) <= tol
    assert ok.all(), "%d of %d off" % ((~ok).sum(), ok.size)


@pytest.fixture
def strict(monkeypatch):
    monkeypatch.setattr(ts, "close", within)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1.001])
def test_within_rejects(bad):
    v, e = np.ones(5), np.full(5, 1e-6)
    within(torch.ones(5), (v, e))
    within(torch.ones(5, dtype=torch.bfloat16), (v + 2.0 ** -9, e), torch.bfloat16)
    got = torch.ones(5)
    got[3] = bad
    with pytest.raises(AssertionError):
        within(got, (v, e))


KINDS = [("channel", "input"), ("channel", "leak"), ("preact", "input"), ("preact", "leak")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("i,shape", list(enumerate(ts.SHAPES + ts.LONG)))
def test_dense(lib, strict, i, shape, dtype):
    gate, write = KINDS[i % 4]
    ts.check(ts.make(*shape, dtype, gate, seed=i), None, write, gate)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(torch.float32, 34), (torch.bfloat16, 33)])
@pytest.mark.parametrize("T,cu", ts.PACKS)
def test_packed_and_alone(lib, strict, T, cu, dtype, D):
    """Each sequence is within the bounds in the pack and alone, so the two are within twice the bound of each other."""
    t = ts.make(1, 2, T, D, dtype, "preact", cu=cu, seed=T)
    ts.check(t, cu, "leak", "preact")
    for n in [n for n in range(len(cu) - 1) if cu[n] < cu[n + 1]][:6]:
        one = {m: t[m][:, :, cu[n]:cu[n + 1]].contiguous() for m in ("x", "z", "dh")}
        ts.check(dict(one, h0=t["h0"][n:n + 1], dhT=t["dhT"][n:n + 1]), None, "leak", "preact")


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,D,pool", [(3, 2, 77, 9), (70, 1, 256, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step(lib, strict, B, H, D, pool, dtype):
    ts.test_scan_step(None, B, H, D, pool, dtype)


@pytest.mark.gpu
def test_tokens_and_splits(lib, strict):
    ts.test_scan_step_iterated_equals_forward(None)
    ts.test_scan_split_sequence_continues(None)


# four times the 592 blocks that the device holds at once, and 5 or 7 rounds of 32 rows, which no larger cluster does in
# fewer waves x rounds: blocks of their own, which carry the state from round to round. With 8 rows a warp, one and two
# channels a lane, and with 16 (156 and 220 rows of one channel)
MANY = [(1, 2368, 156, 2), (1, 2368, 220, 1), (8, 296, 156, 1), (1, 1184, 156, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,L,D", MANY)
def test_many_tiles(lib, strict, B, H, L, D, dtype):
    ts.check(ts.make(B, H, L, D, dtype, "preact", seed=L + D), None, "leak", "preact", reuse=B > 1)


@pytest.mark.gpu
@pytest.mark.parametrize("H,L,D", [m[1:] for m in MANY if m[0] == 1])
def test_many_tiles_packed(lib, strict, H, L, D):
    cu = [2, 40, 40, 71, 150]
    ts.check(ts.make(1, H, L, D, torch.float32, "channel", cu=cu, seed=L), cu, "leak", "channel")
