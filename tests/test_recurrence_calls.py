"""Calls of the scan and of the state cache that their documentation allows: from two host threads at once, with a
pool whose storage was exchanged, and in checking mode with rows that take no part."""
import contextlib
import threading

import pytest
import torch

import chunkwise_linear_rnn_gla_b200 as gla
from chunkwise_linear_rnn_gla_b200 import _lib, build as gbuild, cache as gc, scan
from tests import test_scan as ts
from tests.test_state_cache import check_step, fill_pool, many_rows, pool_case, token


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


def both(lib, *calls, rounds=1500):
    """Every call over and over in a thread and on a stream of its own. The per-kernel timing is on and read by another
    thread, which holds calls up between their preparation and their launch."""
    errors, start, left = [], threading.Barrier(len(calls)), [len(calls)]

    def go(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(rounds):
                    call()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
        left[0] -= 1

    def read():
        while left[0] > 0 and not errors:
            lib.gla_profile_read(None, None, None, 0)

    threads = [threading.Thread(target=go, args=(c,)) for c in calls] + [threading.Thread(target=read)]
    gla.gla_profile_enable(True)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        gla.gla_profile_enable(False)
        gla.gla_profile_reset()
    assert not errors, errors


@pytest.mark.gpu
def test_scan_from_two_threads(lib):
    """One kernel, two shapes: 16 blocks a cluster ask for more shared memory than one block alone."""
    calls, outs = [], []
    for L in (1024, 64):
        t = ts.make(1, 1, L, 64, torch.bfloat16, "channel", seed=L)
        d = {n: v.cuda() for n, v in t.items()}
        ws = scan.scan_workspace(d["x"])
        h, hT = torch.empty_like(d["x"]), torch.empty_like(d["h0"])
        out = {"dx": torch.empty_like(h), "dlog_a": torch.empty_like(d["z"]), "dh0": torch.empty_like(hT)}

        def call(d=d, ws=ws, h=h, hT=hT, out=out):
            scan.scan_fwd(d["x"], d["z"], d["h0"], h=h, hT=hT, workspace=ws)
            scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], workspace=ws, ws_from_fwd=True, out=out)

        calls.append(call)
        outs.append((dict(h=h, hT=hT, **out), ts.run(t, None, "input", "channel")))
    torch.cuda.synchronize()
    both(lib, *calls)
    for got, want in outs:
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.gpu
def test_cache_from_two_threads(lib):
    """Two pools with different windows: the step's and the load's shared memory follow the window."""
    calls, outs = [], []
    for W in (64, 50):
        c, _, g = fill_pool(2, 1, 200, 128, W, "int8", torch.float32, seed=W)
        slots, lengths = pool_case(c, [1, 0], [3, W - 2])
        t = {n: x.cuda() for n, x in token(c, 2, g).items()}
        o, S = torch.empty(2, 1, 128, device="cuda"), torch.empty(2, 1, 200, 128, device="cuda")

        def call(c=c, t=t, slots=slots, lengths=lengths, o=o, S=S):
            gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths, o=o)
            gc.cache_load(c, slots, lengths, S=S)

        call()
        torch.cuda.synchronize()
        calls.append(call)
        outs.append((o, o.clone(), S, S.clone()))
    both(lib, *calls)
    for o, o1, S, S1 in outs:
        assert torch.equal(o, o1) and torch.equal(S, S1)


NAN = float("nan")


def refused(call, *a, **kw):
    with pytest.raises(gla.GlaError) as e:
        call(*a, **kw)
    assert e.value.status == _lib.GLA_ERR_INVALID_ARG and gla.gla_check_device_error() == _lib.GLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["channel", "preact"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_checks_of_packed_rows(lib, gate, dtype):
    """Rows outside every sequence may hold anything; the others are checked, their outputs too."""
    cu, T, H, D = [3, 40, 40, 200], 333, 2, 70
    t = ts.make(1, H, T, D, dtype, gate, cu=cu, seed=5)
    d = {n: v.cuda() for n, v in t.items()}
    for n in ("x", "z", "dh"):
        d[n][:, :, :3], d[n][:, :, 200:] = NAN, NAN
    o = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), write="leak", gate=gate,
             tau=ts.TAU if gate == "preact" else 0.0)
    full = lambda like: torch.full_like(like, NAN)  # noqa: E731
    ws = scan.scan_workspace(d["x"], o["cu_seqlens"], checks=True)
    h, hT = scan.scan_fwd(d["x"], d["z"], d["h0"], h=full(d["x"]), workspace=ws, checks=True, **o)
    b = scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], out={"dx": full(h), "dlog_a": full(d["z"])}, workspace=ws,
                      ws_from_fwd=True, checks=True, **o)
    h1, hT1 = scan.scan_fwd(d["x"], d["z"], d["h0"], **o)
    b1 = scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], **o)
    for g, g1 in ((h, h1), (b["dx"], b1["dx"]), (b["dlog_a"], b1["dlog_a"])):
        assert torch.equal(g[:, :, 3:200], g1[:, :, 3:200])
        assert bool(g[:, :, :3].isnan().all()) and bool(g[:, :, 200:].isnan().all())
    assert torch.equal(hT, hT1) and torch.equal(b["dh0"], b1["dh0"])
    # the first and the last row that belong to a sequence, in each input
    for n, row, bad in (("x", 3, NAN), ("x", 199, float("inf")), ("z", 199, 0.5), ("z", 3, NAN)):
        if n == "z" and gate == "preact" and bad == 0.5:
            continue  # every finite pre-activation is a gate
        p = dict(d, **{n: d[n].clone()})
        p[n][0, 1, row, 69] = bad
        refused(scan.scan_fwd, p["x"], p["z"], p["h0"], checks=True, **o)
    p = dict(d, dh=d["dh"].clone())
    p["dh"][0, 0, 100, 0] = NAN
    refused(scan.scan_bwd, p["x"], p["z"], p["dh"], p["h0"], p["dhT"], checks=True, **o)


@pytest.mark.gpu
def test_checks_of_padding_rows_in_a_scan_step(lib):
    B, D = 5, 40
    x, z = torch.randn(B, 1, D, device="cuda"), -torch.rand(B, 1, D, device="cuda")
    slots = torch.tensor([4, -1, 0, -7, 2], dtype=torch.int32, device="cuda")
    x[1], z[1], z[3] = NAN, NAN, 0.25
    h = scan.scan_step(x, z, torch.zeros(6, 1, D, device="cuda"), slots, checks=True)
    assert bool((h[[1, 3]] == 0).all()) and torch.equal(h[[0, 2, 4]], x[[0, 2, 4]])
    refused(scan.scan_step, x, z, torch.zeros(6, 1, D, device="cuda"), checks=True)  # without slots every row counts
    for b in (0, 4):
        zb = z.clone()
        zb[b, 0, D - 1] = 0.25
        refused(scan.scan_step, x, zb, torch.zeros(6, 1, D, device="cuda"), slots, checks=True)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["channel", "scalar"])
def test_checks_of_padding_rows_in_a_cached_step(lib, gate):
    c, S, g = fill_pool(4, 2, 32, 64, 4, "int8", torch.float32)
    t = {n: x.cuda() for n, x in token(c, 3, g, gate).items()}
    slots, lengths = pool_case(c, [3, -2, 0], [0, 0, 2])
    for x in t.values():
        x[1] = NAN
    gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths, gate=gate, checks=True)
    S = S.cuda()[:3].contiguous()
    S[1] = NAN
    gc.cache_store(c, S, slots, checks=True)
    gc.cache_load(c, slots, lengths, checks=True)
    S[2, 1, 31, 63] = NAN
    refused(gc.cache_store, c, S, slots, checks=True)
    t["log_a"][2, 1] = 0.25
    refused(gc.cache_step, c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths, gate=gate, checks=True)


@pytest.mark.gpu
def test_checks_still_report_refused_rows(lib):
    """A slot outside the pool has no row to check, and is reported."""
    x, z = torch.randn(2, 1, 40, device="cuda"), torch.full((2, 1, 40), NAN, device="cuda")
    z[0] = -1
    refused(scan.scan_step, x, z, torch.zeros(3, 1, 40, device="cuda"),
            torch.tensor([0, 3], dtype=torch.int32, device="cuda"), checks=True)
    # boundaries beyond the rows or out of order: nothing outside the tensors is read
    x = torch.randn(1, 1, 300, 64, device="cuda")
    for cu in ([-5, 100, 400], [250, 10, 20], [2**31 - 1, 5, -2**31]):
        scan.scan_fwd(x, -x.abs(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), hT=None, want_hT=False,
                      checks=True)


@pytest.fixture
def no_patience(lib):
    """Waits inside the kernels run out before they begin, until the fixture's function is called."""
    gla.gla_selftest_wait_limit(-1)
    yield lambda: gla.gla_selftest_wait_limit(0)
    gla.gla_selftest_wait_limit(0)
    gla.gla_check_device_error()


def timed_out():
    return gla.gla_check_device_error() == _lib.GLA_ERR_TIMEOUT and gla.gla_check_device_error() == _lib.GLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [None, [0, 1500, 1507, 4100]])
@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 33)])
def test_scan_writes_nothing_after_a_wait_that_ran_out(lib, no_patience, dtype, D, cu):
    """Several rounds of several blocks a sequence: the call ends, reports the timeout, leaves its outputs and the kept
    states as they were, and the next call is right."""
    t = ts.make(1, 2, 4100, D, dtype, "channel", cu=cu, seed=D)
    d = {n: v.cuda() for n, v in t.items()}
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    seven = lambda like: torch.full_like(like, 7)  # noqa: E731
    h, hT, ws = seven(d["x"]), seven(d["h0"]), scan.scan_workspace(d["x"], c).fill_(7)
    scan.scan_fwd(d["x"], d["z"], d["h0"], cu_seqlens=c, h=h, hT=hT, workspace=ws)
    assert timed_out()
    for x in (h, hT, ws[:2 * -(-4100 // 32) * D * 4]):  # (a guard block may follow the states)
        assert bool((x == 7).all())
    out = {"dx": seven(d["x"]), "dlog_a": seven(d["z"]), "dh0": seven(hT)}
    ws.zero_()
    scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], cu_seqlens=c, workspace=ws, ws_from_fwd=True, out=out)
    assert timed_out()
    for x in out.values():
        assert bool((x == 7).all())
    no_patience()
    ts.check(t, cu, "input", "channel")
    assert gla.gla_check_device_error() == _lib.GLA_OK


@pytest.mark.gpu
def test_scan_of_one_block_waits_for_nobody(lib, no_patience):
    ts.check(ts.make(2, 1, 30, 64, torch.float32, "channel"), None, "leak", "channel")
    assert gla.gla_check_device_error() == _lib.GLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("folds", ["some", "all"])
def test_cached_step_writes_nothing_after_a_wait_that_ran_out(lib, no_patience, folds):
    """Large heads for every SM: the parts of a block wait for one another. The call ends, reports the timeout, leaves
    its output and the pool as they were, and the next call is right."""
    c, _, g = fill_pool(42, 4, 256, 512, 16, "int8", torch.bfloat16)
    before = {n: getattr(c, n).clone() for n in ("codes", "scale", "k", "v", "log_a")}
    sl, ln = many_rows(40, 42, 16, g, folds)
    slots, lengths = pool_case(c, sl, ln)
    t = {n: x.cuda() for n, x in token(c, 40, g).items()}
    o = torch.full_like(t["v"], 7)
    gc.cache_step(c, t["q"], t["k"], t["v"], t["log_a"], slots, lengths, o=o)
    assert timed_out()
    assert bool((o == 7).all())
    for n, x in before.items():
        assert torch.equal(getattr(c, n), x), n
    no_patience()
    check_step(c, sl, ln, "channel", g)


def exchange(c, names=("codes", "scale", "k", "v", "log_a")):
    """New storage with the same values behind a pool's tensors; returns the old storage, which stays alive."""
    old = {}
    for n in names:
        t = getattr(c, n)
        old[n] = t.detach()
        t.data = t.clone()
    return old


@pytest.mark.gpu
@pytest.mark.parametrize("names", [("codes", "scale", "k", "v", "log_a"), ("scale",), ("v",)])
def test_pool_with_exchanged_storage(lib, names):
    """A pool is where its tensors are at the time of the call."""
    c, _, g = fill_pool(4, 2, 32, 160, 4, "int8", torch.bfloat16)
    ref, S, _ = fill_pool(4, 2, 32, 160, 4, "int8", torch.bfloat16)
    t = {n: x.cuda() for n, x in token(c, 3, g).items()}
    slots, lengths = pool_case(c, [3, 1, 0], [3, 0, 2])
    S = S[:3].contiguous().cuda()
    for call in (lambda p: gc.cache_step(p, t["q"], t["k"], t["v"], t["log_a"], slots, lengths),
                 lambda p: gc.cache_load(p, slots, lengths), lambda p: gc.cache_store(p, S, slots)):
        old = exchange(c, names)
        before = {n: x.clone() for n, x in old.items()}
        got, want = call(c), call(ref)
        assert got is None or torch.equal(got, want)
        for n, x in old.items():
            assert torch.equal(x, before[n]), n
        for n in ("codes", "scale", "k", "v", "log_a"):
            assert torch.equal(getattr(c, n), getattr(ref, n)), n


def test_pool_with_storage_that_does_not_fit(lib):
    c = gc.StateCache.empty(4, 1, 8, 16, device="cpu")
    s = torch.zeros(2, dtype=torch.int32)
    for n, other in (("scale", torch.zeros(3, 1, 8, 1)), ("k", torch.zeros(4, 1, 16, 4, dtype=torch.bfloat16)),
                     ("log_a", torch.zeros(4, 1, 16, 16)[..., ::2])):
        t = getattr(c, n)
        was, t.data = t.data, other
        with pytest.raises(ValueError, match=n):
            gc.cache_load(c, s, s)
        t.data = was
    with pytest.raises(ValueError, match="CUDA"):
        gc.cache_load(c, s, s)


def test_a_pool_keeps_a_limited_number_of_descriptors(lib):
    """Continuous batching calls with every number of rows, and the options are the caller's floats."""
    c = gc.StateCache.empty(4, 1, 8, 16, device="cpu")
    for i in range(1000):
        s = torch.zeros(i + 1, dtype=torch.int32)
        with pytest.raises(ValueError, match="CUDA"):
            gc.cache_load(c, s, s, S=torch.empty(i + 1, 1, 8, 16))
    assert all(len(x) <= 256 for x in vars(c).values() if isinstance(x, (dict, list, tuple)))


@pytest.mark.parametrize("wrong", [None, 0, 1, 2])
def test_checks_look_at_the_margins_of_outputs(lib, monkeypatch, wrong):
    """Every output that a binding allocates in checking mode lies between canaries (as gla_fwd's do). The library's call
    is left out here; in its place the margin behind one of the outputs is overwritten."""
    bufs = []

    def fake(*a):
        if wrong is not None:
            bufs[min(wrong, len(bufs) - 1)][-1] = 0

    for m in (scan, gc):
        guarded = m._guarded

        def record(shape, dtype, dev, guards, guarded=guarded):
            t = guarded(shape, dtype, dev, guards)
            bufs.append(guards[-1][0])
            return t

        monkeypatch.setattr(m, "_guarded", record)
        monkeypatch.setattr(m, "_enqueue", fake)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(gla, "gla_check_device_error", lambda: _lib.GLA_OK)
    x, z, s = torch.zeros(1, 1, 8, 4), torch.zeros(1, 1, 8, 4), torch.zeros(1, dtype=torch.int32)
    c = gc.StateCache.empty(4, 1, 8, 16, device="cpu", dtype=torch.float32)
    q, v = torch.zeros(1, 1, 8), torch.zeros(1, 1, 16)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for outputs, call in ((2, lambda: scan.scan_fwd(x, z, checks=True)), (2, lambda: scan.scan_fwd(x, z, cu_seqlens=cu, checks=True)),
                          (3, lambda: scan.scan_bwd(x, z, x, checks=True)),
                          (1, lambda: scan.scan_step(x[:, :, 0].contiguous(), z[:, :, 0].contiguous(), torch.zeros(1, 1, 4), checks=True)),
                          (1, lambda: gc.cache_load(c, s, s, checks=True)),
                          (1, lambda: gc.cache_step(c, q, q, v, q, s, s, checks=True))):
        bufs.clear()
        if wrong is None:
            call()
        else:
            with pytest.raises(gla.GlaError, match="canary"):
                call()
        assert len(bufs) == outputs
