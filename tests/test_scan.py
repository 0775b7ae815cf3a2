"""Elementwise gated recurrence (scan_fwd / scan_bwd / scan_step) against a plain fp64 loop.

Tolerances come from a running error bound computed beside the fp64 values. With u = 2^-24 a step
h = a h' + w x in fp32 adds at most (ea + u) |a h'| + (ew + u) |w x| + u |h| to the error it carries on as a
times the old one, where ea and ew bound the relative errors of a and w: the exponential functions are off by
at most 2 ulp = 4u each, and a pre-activation gate adds the error of log a (the exponential in logsigmoid is
off by at most 2 + 1.173 |z| ulp, the logarithm and the scaling by 4u more), which a sees times |log a|.
Joining segments multiplies the same factors in another order, so the same bound holds with the step terms
doubled. The rounding of an output adds eps / 2 of its type.
"""
import ctypes

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gla_b200 as gla
from chunkwise_linear_rnn_gla_b200 import _lib, build as gbuild, scan

U = 2.0 ** -24
TAU = 16.0


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gates64(z, gate, leak):
    """log a, a, w and the relative error bounds of a and w."""
    if gate == "preact":
        la = (np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))) / TAU
        rel = (2 * (2 + 1.173 * np.abs(z)) + 12) * U
    else:
        la, rel = z, 0.0
    a = np.exp(np.maximum(la, -1e4))
    return a, (-np.expm1(np.maximum(la, -1e4)) if leak else np.ones_like(a)), 4 * U + rel * np.abs(np.maximum(la, -1e4)), \
        (4 * U + rel) if leak else 0.0


def reference(x, z, h0, cu, write, gate, dh=None, dhT=None):
    """fp64 loop over [B,H,L,D] (or [1,H,T,D] with cu): dict name -> (value, error bound before rounding)."""
    leak = write == "leak"
    H, L, D = x.shape[1:]
    a, w, ea, ew = gates64(z, gate, leak)
    N = x.shape[0] if cu is None else len(cu) - 1
    h, eh, hp, ehp = (np.zeros_like(x) for _ in range(4))
    hT, ehT = np.zeros((N, H, D)), np.zeros((N, H, D))
    spans = [(n, 0, L, n) for n in range(N)] if cu is None else [(0, int(cu[n]), int(cu[n + 1]), n) for n in range(N)]
    ea = np.broadcast_to(ea, x.shape)
    ew = np.broadcast_to(ew, x.shape)
    for b, lo, hi, n in spans:
        y = h0[n].copy()
        e = np.zeros((H, D))
        for t in range(lo, hi):
            i = (b, slice(None), t)
            hp[i], ehp[i] = y, e
            p, q = a[i] * y, w[i] * x[i]
            e = a[i] * e + 2 * ((ea[i] + U) * np.abs(p) + (ew[i] + U) * np.abs(q))
            y = p + q
            e = e + 2 * U * np.abs(y)
            h[i], eh[i] = y, e
        hT[n], ehT[n] = y, e
    res = {"h": (h, eh), "hT": (hT, ehT)}
    if dh is None:
        return res
    dx, edx, dla, edla = (np.zeros_like(x) for _ in range(4))
    dh0, edh0 = np.zeros((N, H, D)), np.zeros((N, H, D))
    zrel = 0.0
    if gate == "preact":
        sg = 1 / (1 + np.exp(z)) / TAU
        zrel = (2 * (2 + 1.173 * np.abs(z)) + 8) * U
    for b, lo, hi, n in spans:
        y = dhT[n].copy()
        e = np.zeros((H, D))
        for t in range(hi - 1, lo - 1, -1):
            i = (b, slice(None), t)
            g = dh[i] + y
            eg = e + 2 * U * (np.abs(g) + np.abs(y))
            dx[i], edx[i] = w[i] * g, w[i] * eg + (ew[i] + 2 * U) * np.abs(w[i] * g)
            y = a[i] * g
            e = a[i] * eg + 2 * (ea[i] + U) * np.abs(y)
            d = hp[i] - (x[i] if leak else 0)
            dla[i] = y * d
            edla[i] = e * np.abs(d) + np.abs(y) * (ehp[i] + 2 * U * np.abs(d)) + 2 * U * np.abs(y * d)
            if gate == "preact":
                dla[i] *= sg[i]
                edla[i] = edla[i] * sg[i] + zrel[i] * np.abs(dla[i])
        dh0[n], edh0[n] = y, e
    res.update(dx=(dx, edx), dlog_a=(dla, edla), dh0=(dh0, edh0))
    return res


def make(B, H, L, D, dtype, gate, cu=None, seed=0, z_mean=0.0, h0=True):
    g = torch.Generator().manual_seed(seed)
    lead = (B, H, L) if cu is None else (1, H, L)
    N = B if cu is None else len(cu) - 1
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    z = r(*lead, D) + z_mean
    t = dict(x=r(*lead, D).to(dtype), z=z if gate == "preact" else torch.nn.functional.logsigmoid(z) / TAU,
             dh=r(*lead, D).to(dtype), h0=r(N, H, D) if h0 else None, dhT=r(N, H, D) if h0 else None)
    return t


def f64(t, like=None):
    return np.zeros(like) if t is None else t.double().cpu().numpy()


def close(got, want, dtype=torch.float32):
    v, e = want
    got = f64(got)
    tol = e + half_step(dtype) * (np.abs(v) + e) * (dtype != torch.float32) + 1e-37
    bad = np.abs(got - v) > tol
    assert not bad.any(), "%d of %d off, worst %.3g times the bound" % (
        bad.sum(), bad.size, np.nanmax(np.abs(got - v) / tol))


def run(t, cu, write, gate, reuse=True, **kw):
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = dict(cu_seqlens=c, write=write, gate=gate, tau=TAU if gate == "preact" else 0.0, **kw)
    ws = scan.scan_workspace(d["x"], c)
    h, hT = scan.scan_fwd(d["x"], d["z"], d["h0"], workspace=ws if reuse else None, **o)
    if reuse:
        b = scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], workspace=ws, ws_from_fwd=True, **o)
    else:
        b = scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], **o)
    return dict(h=h, hT=hT, **b)


def check(t, cu, write, gate, reuse=True):
    got = run(t, cu, write, gate, reuse)
    N, H, D = got["hT"].shape
    want = reference(f64(t["x"]), f64(t["z"]), f64(t["h0"], (N, H, D)), cu, write, gate, f64(t["dh"]),
                     f64(t["dhT"], (N, H, D)))
    for n in ("h", "hT", "dx", "dlog_a", "dh0"):
        close(got[n], want[n], t["x"].dtype if n in ("h", "dx") else torch.float32)
    return got


# ---------------------------------------------------------------- numerics

SHAPES = [(1, 1, 1, 1), (1, 1, 2, 64), (2, 3, 127, 5), (1, 2, 128, 66), (3, 1, 129, 64), (2, 1, 333, 130), (1, 1, 1000, 33),
          (1, 1, 4100, 64), (5, 2, 64, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("gate,write", [("channel", "input"), ("channel", "leak"), ("preact", "input"),
                                        ("preact", "leak")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_dense(lib, shape, dtype, gate, write):
    check(make(*shape, dtype, gate, seed=sum(shape)), None, write, gate)


PACKS = [(1, [0, 1]), (7, [0, 0, 3, 3, 3, 7, 7]), (300, [0, 1, 2, 130, 256, 299]), (1100, [5, 5, 400, 401, 1090]),
         (64, [0, 0, 0]), (2500, [0, 128, 256, 2400, 2400]), (513, list(range(0, 501, 2)))]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(torch.float32, 33), (torch.bfloat16, 64)])
@pytest.mark.parametrize("T,cu", PACKS)
def test_scan_packed(lib, T, cu, dtype, D):
    t = make(1, 2, T, D, dtype, "channel", cu=cu, seed=T)
    got = check(t, cu, "leak", "channel")
    # each sequence on its own gives the same values: nothing leaks across a boundary
    for n in range(len(cu) - 1):
        lo, hi = cu[n], cu[n + 1]
        if lo == hi:
            assert torch.equal(got["hT"][n].cpu(), t["h0"][n]) and torch.equal(got["dh0"][n].cpu(), t["dhT"][n])


@pytest.mark.gpu
def test_scan_packed_leaves_other_rows(lib):
    cu, T, H, D = [3, 40, 40, 200], 333, 2, 70
    t = make(1, H, T, D, torch.bfloat16, "preact", cu=cu, seed=5)
    d = {k: v.cuda() for k, v in t.items()}
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h = torch.full((1, H, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dla = h.clone(), torch.full((1, H, T, D), 7.0, device="cuda")
    # what stands in the rows outside does not matter either
    for n in ("x", "z", "dh"):
        d[n][:, :, :3] = float("nan")
        d[n][:, :, 200:] = float("inf")
    o = dict(cu_seqlens=c, write="leak", gate="preact", tau=TAU)
    _, hT = scan.scan_fwd(d["x"], d["z"], d["h0"], h=h, **o)
    b = scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], out={"dx": dx, "dlog_a": dla}, **o)
    for g in (h, dx, dla):
        assert bool((g[:, :, :3] == 7).all()) and bool((g[:, :, 200:] == 7).all())
        assert bool(torch.isfinite(g).all())
    assert bool(torch.isfinite(hT).all()) and bool(torch.isfinite(b["dh0"]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_packed_sequences_do_not_reach_each_other(lib, bad):
    """One sequence full of NaN or infinities: its neighbours' results are those without it, bit for bit."""
    cu, T, D = [0, 37, 300, 1500, 1507], 1507, 64
    t = make(1, 1, T, D, torch.float32, "channel", cu=cu, seed=12)
    want = run(t, cu, "leak", "channel")
    for n in ("x", "z", "dh"):
        p = dict(t, **{n: t[n].clone()})
        p[n][:, :, 37:300] = bad if n != "z" else -bad
        p["h0"], p["dhT"] = t["h0"].clone(), t["dhT"].clone()
        p["h0"][1], p["dhT"][1] = bad, bad
        got = run(p, cu, "leak", "channel")
        for m in ("h", "dx", "dlog_a"):
            assert torch.equal(got[m][:, :, :37], want[m][:, :, :37]) and torch.equal(got[m][:, :, 300:], want[m][:, :, 300:])
        for m in ("hT", "dh0"):
            assert torch.equal(got[m][[0, 2, 3]], want[m][[0, 2, 3]])
        assert not bool(torch.isfinite(got["dx"][:, :, 37:300]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [None, [0, 100, 700]])
def test_scan_without_states_and_without_reuse(lib, cu):
    t = make(2, 1, 700, 40, torch.float32, "channel", cu=cu, seed=3, h0=False)
    one = check(t, cu, "input", "channel", reuse=False)
    two = run(t, cu, "input", "channel", reuse=True)
    for n in one:
        assert torch.equal(one[n], two[n]), n


@pytest.mark.gpu
def test_scan_zero_gates_and_slow_decay(lib):
    t = make(1, 1, 3000, 64, torch.float32, "channel", seed=9, z_mean=6.0)
    t["z"][:, :, 500] = -1e30  # a zero gate forgets everything before it
    t["z"][:, :, 1000:1100, ::2] = 0.0  # and a gate of one keeps everything
    got = check(t, None, "input", "channel")
    assert torch.equal(got["h"][:, :, 500].cpu(), t["x"][:, :, 500])
    check(t, None, "leak", "channel")


@pytest.mark.gpu
def test_scan_gradient_against_differences(lib):
    """Central differences of the fp32 call itself: step s = 2^-6, so the difference quotient of the (bi)linear
    loss is off by the gate's third derivative times s^2 / 6 < 5e-5 of the gradient's scale and by 2 u |loss| / s."""
    B, H, L, D = 1, 1, 40, 3
    t = make(B, H, L, D, torch.float32, "preact", seed=11)
    d = {k: v.cuda() for k, v in t.items()}
    o = dict(write="leak", gate="preact", tau=TAU)
    g = scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], **o)

    def loss(**r):
        e = {**d, **r}
        h, hT = scan.scan_fwd(e["x"], e["z"], e["h0"], **o)
        return float((h.double() * d["dh"].double()).sum() + (hT.double() * d["dhT"].double()).sum())

    rng = np.random.RandomState(0)
    s = 2.0 ** -6
    for name, grad in (("x", g["dx"]), ("z", g["dlog_a"]), ("h0", g["dh0"])):
        for _ in range(6):
            i = tuple(rng.randint(n) for n in d[name].shape)
            up, dn = d[name].clone(), d[name].clone()
            up[i] += s
            dn[i] -= s
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * s)
            # |loss| sums to under 2^7; each h is off by under 40 u, so the quotient by under 2^7 * 40 * u / s < 0.02
            assert abs(num - float(grad[i])) < 0.02 + 1e-3 * abs(num), (name, i, num, float(grad[i]))


@pytest.mark.gpu
def test_scan_split_sequence_continues(lib):
    t = make(2, 1, 400, 64, torch.float32, "channel", seed=4)
    d = {k: v.cuda() for k, v in t.items()}
    h, hT = scan.scan_fwd(d["x"], d["z"], d["h0"])
    cut = lambda n, a, b: d[n][:, :, a:b].contiguous()  # noqa: E731
    h1, m = scan.scan_fwd(cut("x", 0, 150), cut("z", 0, 150), d["h0"])
    h2, e = scan.scan_fwd(cut("x", 150, 400), cut("z", 150, 400), m)
    want = reference(f64(t["x"]), f64(t["z"]), f64(t["h0"]), None, "input", "channel")
    close(torch.cat([h1, h2], 2), want["h"])
    close(e, want["hT"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,D,pool", [(1, 1, 1, 1), (3, 2, 77, 9), (70, 1, 256, 128), (300, 1, 64, 300)])
def test_scan_step(lib, B, H, D, pool, dtype):
    for gate, write in (("channel", "input"), ("preact", "leak")):
        t = make(B, H, 1, D, dtype, gate, seed=B)
        g = torch.Generator().manual_seed(1)
        state = torch.randn(pool, H, D, generator=g)
        slots = torch.randperm(pool, generator=g)[:B].to(torch.int32)
        if B > 2:
            slots[1] = -1  # a padding row
        st, x, z = state.cuda(), t["x"][:, :, 0].contiguous().cuda(), t["z"][:, :, 0].contiguous().cuda()
        h = scan.scan_step(x, z, st, slots.cuda(), write=write, gate=gate, tau=TAU if gate == "preact" else 0.0)
        live = (slots >= 0).numpy()
        at = slots.numpy()[live]
        want = reference(f64(t["x"]), f64(t["z"]), f64(state[slots.clamp(min=0).long()]), None, write, gate)
        v, e = want["hT"]
        close(st.cpu()[torch.from_numpy(at).long()], (v[live], e[live]))
        close(h.cpu()[torch.from_numpy(live)], (v[live], e[live]), dtype)
        assert bool((h[~torch.from_numpy(live).cuda()] == 0).all())
        rest = np.setdiff1d(np.arange(pool), at)
        assert torch.equal(st.cpu()[rest], state[rest])
        assert gla.gla_check_device_error() == _lib.GLA_OK


@pytest.mark.gpu
def test_scan_step_iterated_equals_forward(lib):
    t = make(3, 2, 50, 96, torch.float32, "preact", seed=2)
    d = {k: v.cuda() for k, v in t.items()}
    o = dict(write="leak", gate="preact", tau=TAU)
    st = d["h0"].clone()
    hs = [scan.scan_step(d["x"][:, :, i].contiguous(), d["z"][:, :, i].contiguous(), st, **o) for i in range(50)]
    want = reference(f64(t["x"]), f64(t["z"]), f64(t["h0"]), None, "leak", "preact")
    close(torch.stack(hs, 2), want["h"])
    close(st, want["hT"])


@pytest.mark.gpu
def test_scan_step_refuses_bad_slots(lib):
    """The kernel bounds-checks the slots itself: a bad row is skipped and reported."""
    B, D, pool = 6, 40, 5
    x, z = torch.randn(B, 1, D, device="cuda"), -torch.rand(B, 1, D, device="cuda")
    for bad in ([0, 1, 5, 2, -1, 3], [0, 1, 2**31 - 1, 2, -7, 3], [0, 1, 0, 2, -1, 3]):
        st = torch.ones(pool, 1, D, device="cuda")
        h = scan.scan_step(x, z, st, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert gla.gla_check_device_error() == _lib.GLA_ERR_INVALID_ARG
        assert gla.gla_check_device_error() == _lib.GLA_OK
        assert bool((h[2] == 0).all()) and bool((h[4] == 0).all()) and bool((st[4] == 1).all())
        for b in (0, 1, 3, 5):
            assert torch.equal(h[b], st[bad[b]])
            assert not bool((st[bad[b]] == 1).all())


@pytest.mark.gpu
def test_scan_on_another_stream_and_in_a_graph(lib):
    t = make(2, 1, 300, 64, torch.bfloat16, "channel", seed=6)
    d = {k: v.cuda() for k, v in t.items()}
    ref = run(t, None, "input", "channel")
    ws = [scan.scan_workspace(d["x"]) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both(w):
        h, hT = scan.scan_fwd(d["x"], d["z"], d["h0"], workspace=w)
        return dict(h=h, hT=hT, **scan.scan_bwd(d["x"], d["z"], d["dh"], d["h0"], d["dhT"], workspace=w,
                                                ws_from_fwd=True))

    with torch.cuda.stream(side):
        one = both(ws[0])
    torch.cuda.synchronize()
    graphs = []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(w)
        graphs.append((g, out))
    d["x"].mul_(2)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    t2 = dict(t, x=t["x"] * 2)
    ref2 = run(t2, None, "input", "channel")
    for n in ref:
        assert torch.equal(one[n], ref[n]), n
        for _, out in graphs:
            assert torch.equal(out[n], ref2[n]), n


@pytest.mark.gpu
def test_scan_bad_boundaries_stay_inside(lib):
    """Boundaries outside the rows or out of order: the values are meaningless, the accesses are not. The output
    margins stay as they were."""
    T, D = 300, 64
    for cu in ([-5, 100, 400], [0, 200, 100, 300], [250, 10, 20], [2**31 - 1, 5, -2**31]):
        N = len(cu) - 1
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        x, z = torch.randn(1, 1, T, D, device="cuda"), -torch.rand(1, 1, T, D, device="cuda")
        buf = torch.full((T * D + 512,), 7.0, device="cuda")
        h = buf[256:256 + T * D].view(1, 1, T, D)
        tb = torch.full((N * D + 512,), 7.0, device="cuda")
        hT = tb[256:256 + N * D].view(N, 1, D)
        scan.scan_fwd(x, z, torch.zeros(N, 1, D, device="cuda"), cu_seqlens=c, h=h, hT=hT)
        scan.scan_bwd(x, z, x, None, None, cu_seqlens=c)
        torch.cuda.synchronize()
        assert gla.gla_check_device_error() == _lib.GLA_OK
        for m, n in ((buf, T * D), (tb, N * D)):
            assert bool((m[:256] == 7).all()) and bool((m[256 + n:] == 7).all())


@pytest.mark.gpu
def test_scan_checks(lib):
    x, z = torch.randn(1, 1, 200, 64, device="cuda"), -torch.rand(1, 1, 200, 64, device="cuda")
    ws = scan.scan_workspace(x, checks=True)
    h, hT = scan.scan_fwd(x, z, workspace=ws, checks=True)
    scan.scan_bwd(x, z, x, workspace=ws, ws_from_fwd=True, checks=True)
    scan.scan_step(x[:, :, 0].contiguous(), z[:, :, 0].contiguous(), hT, checks=True)
    z[0, 0, 77, 3] = 0.5
    with pytest.raises(gla.GlaError):
        scan.scan_fwd(x, z, checks=True)


# ---------------------------------------------------------------- refusals (no GPU needed)


def desc(**kw):
    d = dict(B=1, H=1, L=64, Dk=64, Dv=1, dtype=0, chunk=0, subchunk=0, state_mode=0, impl=0, flags=0, gate=0,
             gate_tau=0.0)
    d.update(kw)
    return _lib.GlaDesc(**d)


@pytest.mark.parametrize("bad,want", [(dict(B=0), 1), (dict(L=0), 1), (dict(Dk=0), 1), (dict(H=-1), 1), (dict(dtype=4), 1),
                                      (dict(flags=0x40), 1), (dict(gate=9), 1), (dict(gate=3), 1), (dict(gate=1), 2),
                                      (dict(gate=2), 2), (dict(chunk=64), 2), (dict(state_mode=1), 2), (dict(impl=2), 2),
                                      (dict(L=1 << 31), 2)])
def test_scan_bad_descriptor(lib, bad, want):
    d = ctypes.byref(desc(**bad))
    assert lib.gla_scan_workspace_size(d, 0) == 0
    assert lib.gla_scan_fwd(d, 0, 16, 16, None, None, 16, None, None, 0, None) == want
    assert lib.gla_scan_bwd(d, 0, 16, 16, None, None, 16, None, 16, 16, None, 256, 1 << 40, None) == want
    if "L" not in bad:
        assert lib.gla_scan_step(d, 0, 16, 16, None, 1, 16, 16, None) == want


def test_scan_bad_pointers_and_workspace(lib):
    d = ctypes.byref(desc())
    ok = [0, 16, 16, None, None, 16, None, None, 0, None]
    for i in (1, 2, 5):
        for p in (None, 24):
            a = list(ok)
            a[i] = p
            assert lib.gla_scan_fwd(d, *a) == 1, (i, p)
    assert lib.gla_scan_fwd(d, 2, *ok[1:]) == 1  # no such write kind
    assert lib.gla_scan_fwd(None, *ok) == 1
    assert lib.gla_scan_fwd(d, 0, 16, 16, 18, None, 16, None, None, 0, None) == 1  # boundaries off a 4-byte address
    assert lib.gla_scan_fwd(d, 0, 16, 16, None, None, 16, None, 256, 8, None) == 3
    assert lib.gla_scan_fwd(ctypes.byref(desc(flags=1)), *ok) == 1  # a forward reuses nothing
    n = lib.gla_scan_workspace_size(d, 0)
    assert n > 0
    for ws, size in ((None, 0), (256, n - 1), (128, n)):
        assert lib.gla_scan_bwd(d, 0, 16, 16, None, None, 16, None, 16, 16, None, ws, size, None) == 3
    assert lib.gla_scan_step(d, 0, 16, 16, None, 0, 16, 16, None) == 1  # an empty pool
    assert lib.gla_scan_step(ctypes.byref(desc(B=4)), 0, 16, 16, None, 3, 16, 16, None) == 1  # fewer entries than rows
    assert lib.gla_scan_step(d, 0, 16, 16, 18, 4, 16, 16, None) == 1


def test_scan_binding_refuses(lib):
    x, z = torch.zeros(2, 1, 8, 4), torch.zeros(2, 1, 8, 4)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(ValueError):
        scan.scan_fwd(x[0], z)
    with pytest.raises(ValueError):
        scan.scan_fwd(x, z, cu_seqlens=cu)  # packed rows have no batch axis
    with pytest.raises(ValueError):
        scan.scan_fwd(x.transpose(2, 3), z)
    with pytest.raises(ValueError):
        scan.scan_fwd(x, z[:, :, :4])
    with pytest.raises(TypeError):
        scan.scan_fwd(x, z.double())
    with pytest.raises(TypeError):
        scan.scan_fwd(x.half(), z)
    with pytest.raises(ValueError):
        scan.scan_fwd(x, z, torch.zeros(1, 1, 4))
    with pytest.raises(TypeError):
        scan.scan_fwd(x[:1], z[:1], cu_seqlens=cu.long())
    with pytest.raises(ValueError):
        scan.scan_fwd(x[:1], z[:1], cu_seqlens=cu[:1])
    with pytest.raises(ValueError):
        scan.scan_bwd(x, z, x, ws_from_fwd=True)
    with pytest.raises(ValueError):
        scan.scan_step(x[:, :, 0].contiguous(), z[:, :, 0].contiguous(), torch.zeros(1, 1, 4))
    with pytest.raises(ValueError):
        scan.scan_step(x[:, :, 0].contiguous(), z[:, :, 0].contiguous(), torch.zeros(3, 1, 4),
                       torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        scan.scan_fwd(x, z, write="add")


@pytest.mark.gpu
@pytest.mark.parametrize("N", [255, 256, 257, 700])  # on both sides of a power of two, for the search of a row's sequence
def test_scan_packed_many_sequences(lib, N):
    g = torch.Generator().manual_seed(N)
    cu = [2] + (2 + torch.randint(0, 4, (N,), generator=g).cumsum(0)).tolist()  # some empty, rows in front and behind
    check(make(1, 1, cu[-1] + 5, 34, torch.float32, "channel", cu=cu, seed=N), cu, "leak", "channel")


# several rounds with sixteen rows a warp: one and two channels a lane, blocks of four warps and of eight, a ragged end
LONG = [(1, 1, 2077, 64), (1, 2, 4100, 33), (3, 7, 1100, 71), (1, 40, 1500, 37)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", LONG)
def test_scan_long_dense(lib, shape, dtype):
    check(make(*shape, dtype, "preact", seed=sum(shape)), None, "leak", "preact")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,D", [(1, 64), (2, 33), (40, 37)])
def test_scan_long_packed(lib, H, D, dtype):
    cu = [3, 15, 16, 16, 17, 31, 33, 900, 1057, 1057, 1999, 2060]
    check(make(1, H, 2077, D, dtype, "channel", cu=cu, seed=H + D), cu, "input", "channel")
