"""Calls of the scan and of the state cache that their documentation allows: from two host threads at once, with a
pool whose storage was exchanged, and in checking mode with rows that take no part."""
import threading

import pytest
import torch

import chunkwise_linear_rnn_gla_b200 as gla
from chunkwise_linear_rnn_gla_b200 import _lib, build as gbuild, cache as gc, scan
from tests import test_scan as ts
from tests.test_state_cache import fill_pool, pool_case, token


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
